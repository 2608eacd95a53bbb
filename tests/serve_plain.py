"""Plain CPU implementations of the serving operators: the codes and scales
in IEEE binary32 steps as the formats define them, everything else in 64
bits. Shared by the GPU tests; nothing here calls the library."""
import numpy as np
import torch

F = np.float32


def quantize_rows(x):
    """x float32 [n, k] -> codes int8 [n, k up to 128s], scales float32 [n]."""
    n, k = x.shape
    codes = np.zeros((n, -(-k // 128) * 128), dtype=np.int8)
    scales = np.zeros(n, dtype=F)
    for r in range(n):
        row = x[r].astype(F)
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        amax = F(np.max(np.abs(row)))
        with np.errstate(all="ignore"):
            inv = F(127) / amax
            if np.isfinite(inv):
                scales[r] = amax / F(127)
                codes[r, :k] = np.rint(row * inv).astype(np.int8)
    return codes, scales


def product(w, wd, x, xd, bias=None):
    """(y, magnitude) in 64 bits."""
    s = x.astype(np.float64) @ w.astype(np.float64).T
    y = s * xd.astype(np.float64)[:, None] * wd.astype(np.float64)[None, :]
    mag = np.abs(y)
    if bias is not None:
        y = y + bias.astype(np.float64)
        mag = mag + np.abs(bias.astype(np.float64))
    return y, mag


class PlainCache:
    """codes [2][n_blocks, n_heads, block, dim] int8 (keys, values),
    scales [2][n_blocks, n_heads]."""

    def __init__(self, n_blocks, n_heads, dim, block):
        self.block, self.n_blocks = block, n_blocks
        self.codes = [np.zeros((n_blocks, n_heads, block, dim), dtype=np.int8) for _ in range(2)]
        self.scales = [np.zeros((n_blocks, n_heads), dtype=F) for _ in range(2)]

    def place(self, table_row, p):
        slot = p // self.block
        if p < 0 or slot >= len(table_row) or not 0 <= table_row[slot] < self.n_blocks:
            return None
        return table_row[slot], p % self.block

    def append(self, kv, cu, kv_len, table):
        """kv: keys and values float32 [n_tok, n_heads, dim]."""
        for s in range(len(kv_len)):
            n = cu[s + 1] - cu[s]
            first = kv_len[s] - n
            byblock = {}
            for i in range(n):
                at = self.place(table[s], first + i)
                if at is not None:
                    byblock.setdefault(at[0], []).append((at[1], cu[s] + i))
            for b, items in byblock.items():
                t0 = items[0][0]
                rows = [r for _, r in items]
                for j in range(2):
                    new = kv[j][rows].astype(F)                      # [m, h, d]
                    for h in range(new.shape[1]):
                        self._write(j, b, h, t0, new[:, h])

    def _write(self, j, b, h, t0, new):
        with np.errstate(all="ignore"):
            old = self.scales[j][b, h] if t0 > 0 else F(0)
            codes = self.codes[j][b, h]
            if not np.all(np.isfinite(new)) or np.isnan(old):
                self.scales[j][b, h] = np.nan
                codes[t0:t0 + len(new)] = 0
                return
            cand = F(np.max(np.abs(new))) / F(127)
            if not np.isfinite(F(1) / cand):
                cand = F(0)
            d = max(old, cand)
            if t0 > 0 and d > old:
                codes[:t0] = np.rint(codes[:t0].astype(F) * (old / d)).astype(np.int8)
            inv = F(1) / d
            if not np.isfinite(inv):
                inv = F(0)
            codes[t0:t0 + len(new)] = np.clip(np.rint(new * inv), -127, 127).astype(np.int8)
            self.scales[j][b, h] = d

    def values(self, table_row, n):
        """(keys, values, present) of positions 0..n-1 in 64 bits."""
        h, dim = self.codes[0].shape[1], self.codes[0].shape[3]
        out = [np.zeros((n, h, dim)) for _ in range(2)]
        present = np.zeros(n, dtype=bool)
        for p in range(n):
            at = self.place(table_row, p)
            if at is None:
                continue
            present[p] = True
            for j in range(2):
                out[j][p] = self.codes[j][at[0], :, at[1]].astype(np.float64) * \
                    self.scales[j][at[0]].astype(np.float64)[:, None]
        return out[0], out[1], present

    def device_tensors(self):
        """k, v, kd, vd laid out as qrow_kv8.h states, on the CPU."""
        k = torch.from_numpy(self.codes[0].copy())
        v = torch.from_numpy(self.codes[1].copy())
        nb, h, bt, d = v.shape
        # token t = 32 a + 8 b + c, channel 2 e + f -> [a][e][b][f][c]
        v = v.view(nb, h, bt // 32, 4, 8, d // 2, 2).permute(0, 1, 2, 5, 3, 6, 4).contiguous()
        return k, v, torch.from_numpy(self.scales[0].copy()), torch.from_numpy(self.scales[1].copy())


def attention(q, cache, cu, kv_len, table, scale, window, fp16_weights):
    """(out, bound) in 64 bits for the rows cu covers; other rows are NaN in
    out. q float64 [n_tok, n_q, dim].

    The bound counts the kernel's roundings, u = 2^-24 being fp32's and
    2^-11 fp16's:
     - a score is D products added in fp32, at most 2 u each relative to the
       sum of magnitudes A, three scalings and, for fp32 queries, the 2^-22
       that two fp16 parts leave of an element: (2 D + 8 + 4) u A;
     - exp2 of a difference: u of its size (at most |s - max| log2 e + 9),
       and 2 u of its own;
     - each of the g groups of 32 tokens rescales the sums (2 u) and adds to
       them (1 u), 32 products per group (2 u each): (3 g + 80) u; the joins
       of waves and splits add 4 u for each of at most 132 parts;
     - weights in fp16: 2^-11 (two parts: 2^-22), and 2^-25 of 2^10 times the
       largest weight where they (or the second parts) are subnormal.
    They enter the weighted sum of |v| and, through the sum of weights, |o|.
    """
    n_tok, n_q, dim = q.shape
    u = 2.0 ** -24
    out = np.full(q.shape, np.nan)
    bound = np.zeros(q.shape)
    for s in range(len(kv_len)):
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        length = max(0, kv_len[s])
        k, v, present = cache.values(table[s], length)
        g = n_q // k.shape[1]
        for i in range(n):
            p = kv_len[s] - n + i
            lo = max(0, p - window + 1) if window else 0
            idx = np.arange(lo, p + 1) if p >= lo else np.zeros(0, int)
            idx = idx[present[idx]]
            r = cu[s] + i
            if len(idx) == 0:
                out[r] = 0.0
                continue
            for h in range(n_q):
                kk, vv = k[idx, h // g], v[idx, h // g]
                sc = scale * (kk @ q[r, h])
                mag = np.max(abs(scale) * (np.abs(kk) @ np.abs(q[r, h])))
                w = np.exp(sc - np.max(sc))
                tot = np.sum(w)
                o = (w @ vv) / tot
                out[r, h] = o
                groups = len(idx) // 32 + 2
                spread = min(np.max(sc) - np.min(sc), 200.0)
                e = (2 * dim + 12) * u * mag + u * (spread * 1.5 + 9 + 2) + (3 * groups + 80 + 528) * u
                e += 2.0 ** -11 if fp16_weights else 2.0 ** -22
                # weights' floor, relative to their sum
                floor = len(idx) * 2.0 ** -35 / tot
                bound[r, h] = e * ((w @ np.abs(vv)) / tot + np.abs(o)) + floor * np.max(np.abs(vv), axis=0)
    return out, bound


def table_for(lens, block, n_blocks, rng, width=None):
    """A table that scatters every sequence's blocks."""
    per = [-(-max(0, n) // block) for n in lens]
    assert sum(per) <= n_blocks
    order = rng.permutation(n_blocks)
    width = width or max(max(per), 1)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, m in enumerate(per):
        table[s, :m] = order[at:at + m]
        at += m
    return table


def offsets(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


