"""Plain CPU implementations of the 8-bit layer's operators (norm, product with
epilogue, router, experts): the steps that the headers fix in their 32 or 64
bits, sums and everything else in 64. Shared by the GPU tests; nothing here
calls the library."""
import numpy as np
import torch

F, D = np.float32, np.float64
U = 2.0 ** -24            # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACT_ERROR = 8 * U         # of an activation, relative to its argument


def rounded(x, dtype):
    """float32 values rounded to dtype, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(dtype).float().numpy()


def code_rule(v):
    """(codes, scales) of the rows (last dimension) of float32 v: max / 127 and
    rint(v * (127 / max)); zero codes where there is no number to make them of,
    and the products before their rounding to a code."""
    with np.errstate(all="ignore"):
        top = np.max(np.abs(v), axis=-1, keepdims=True)
        top = np.where(np.isfinite(v).all(axis=-1, keepdims=True), top, F(np.inf)).astype(F)
        inv = F(127) / top
        d = top / F(127)
        none = ~np.isfinite(inv)
        d = np.where(none, F(0), d)
        inv = np.where(none, F(0), inv)
        bad = ~np.isfinite(top)
        d = np.where(bad, F(np.nan), d).astype(F)
        inv = np.where(bad, F(0), inv).astype(F)
        p = np.where(bad, F(0), v * inv).astype(F)
    return np.rint(p).astype(np.int8), d[..., 0], p


def norm(x, residual, weight, eps, dtype):
    """x, residual (or None), weight (or None) float32 -> (total, y) float32
    before y's rounding to dtype."""
    total = None
    s = x.astype(F)
    with np.errstate(all="ignore"):
        if residual is not None:
            total = s = rounded((s + residual.astype(F)).astype(F), dtype)
        s64 = s.astype(D)
        f = 1.0 / np.sqrt(np.sum(s64 * s64, axis=1, keepdims=True) / x.shape[1] + eps)
        y = (s64 * f).astype(F)
        if weight is not None:
            y = (y * weight.astype(F)).astype(F)
    return total, y


def erfc(x):
    return torch.special.erfc(torch.from_numpy(np.asarray(x, dtype=D))).numpy()


def act(name, x):
    """In 64 bits."""
    with np.errstate(all="ignore"):
        if name == "relu":
            return np.where(x > 0, x, np.where(np.isnan(x), x, 0.0))
        if name == "silu":
            return x / (1.0 + np.exp(-x))
        if name == "gelu":
            return x * 0.5 * erfc(-x / np.sqrt(2.0))
        if name == "gelu_tanh":
            return x / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))
    return x


def linear(w, wd, x, xd, bias):
    """(product, its error in fp32): four roundings of |product| + |bias|."""
    s = (x.astype(D) @ w.astype(D).T) * xd.astype(D)[:, None] * wd.astype(D)[None, :]
    mag = np.abs(s)
    if bias is not None:
        s = s + bias.astype(D)
        mag = mag + np.abs(bias.astype(D))
    return s, 4 * U * mag


def product(w, wd, x, xd, bias, name, up, residual, dtype):
    """(y, bound) of qr_matmul_i8_ex. up: None or (codes, scales, bias). An
    activation passes an error of its argument on by at most 1.13 (GELU's
    steepest slope)."""
    p, e = linear(w, wd, x, xd, bias)
    y = act(name, p)
    if name != "none":
        e = 1.13 * e + (0 if name == "relu" else ACT_ERROR) * np.abs(p) + 2.0 ** -110
    if up is not None:
        u, eu = linear(up[0], up[1], x, xd, up[2])
        e = e * (np.abs(u) + eu) + np.abs(y) * eu
        y = y * u
        e = e + U * (np.abs(y) + e)
    if residual is not None:
        y = y + residual.astype(D)
        e = e + U * (np.abs(y) + e)
    return y, e + HALF[dtype] * (np.abs(y) + e) + 2.0 ** -130


def route(x, w, top_k, score, bias, renorm, factor):
    """(ids, weights in 64 bits); x, w float64."""
    with np.errstate(all="ignore"):
        logit = x @ w.T
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-logit))
        else:
            top = np.where(np.isnan(logit), -np.inf, logit).max(axis=1, keepdims=True)
            s = np.exp(logit - top)
            s = s / s.sum(axis=1, keepdims=True)
        by = s + (0 if bias is None else bias.astype(D)[None, :])
        # a NaN before everything, then the largest, the lowest index among equals
        order = np.lexsort((np.broadcast_to(np.arange(w.shape[0]), by.shape), np.where(np.isnan(by), 0.0, -by),
                            ~np.isnan(by)), axis=1)
    ids = np.full((len(x), top_k), -1, dtype=np.int64)
    wt = np.zeros((len(x), top_k))
    off = np.zeros(w.shape[0], dtype=bool) if bias is None else bias == -np.inf
    for t in range(len(x)):
        mine = [e for e in order[t] if not off[e]][:top_k]
        ids[t, :len(mine)] = mine
        wt[t, :len(mine)] = s[t, mine]
    if renorm:
        with np.errstate(all="ignore"):
            tot = wt.sum(axis=1, keepdims=True)
            wt = np.where(tot == 0.0, 0.0, wt / tot)
    wt = wt * np.where(ids < 0, 0.0, factor)
    return ids, np.where(ids < 0, 0.0, wt)


def hidden(gate, gated, up, upd, x, xd, name):
    """Hidden rows of one expert as their codes stand for them: values
    [n, blocks, 64] in 64 bits, float32 scales. gate, up int8 [n_mid, n_in]."""
    with np.errstate(all="ignore"):
        one = lambda w, wd: (((x.astype(D) @ w.astype(D).T).astype(F) * xd[:, None]).astype(F) * wd[None, :]).astype(F)
        g, u = one(gate, gated).astype(D), one(up, upd).astype(D)
        h = (act(name, g) * u).astype(F)
        pad = -h.shape[1] % 64
        h = np.pad(h, ((0, 0), (0, pad))).reshape(len(x), -1, 64)
        codes, d, _ = code_rule(h)
        return codes.astype(D) * d.astype(D)[..., None]


def experts(layer, x, xd, ids, weights, name, residual, dtype):
    """(y, bound) of qr_moe_i8. layer: dict of int8 arrays gate, up, down
    [n_experts, rows, n] (row tails cut off) and float32 gated, upd, downd.

    An expert's output is a sum over blocks in fp32: two roundings a block of
    what it has added up by then, at most (2 blocks + 8 parts) U of the sum of
    magnitudes, its scale and weight one more each; a token's slots one each."""
    n_tok, k = ids.shape
    n_in = layer["down"].shape[1]
    y = np.zeros((n_tok, n_in))
    e = np.zeros((n_tok, n_in))
    mag = np.zeros((n_tok, n_in))
    with np.errstate(all="ignore"):
        for ex in range(layer["gate"].shape[0]):
            t, j = np.nonzero(ids == ex)
            if len(t) == 0:
                continue
            h = hidden(layer["gate"][ex], layer["gated"][ex], layer["up"][ex], layer["upd"][ex], x[t], xd[t], name)
            down = layer["down"][ex].astype(D)
            down = np.pad(down, ((0, 0), (0, h.shape[1] * 64 - down.shape[1]))).reshape(n_in, -1, 64)
            part = np.einsum("nbc,rbc->nrb", h, down) * layer["downd"][ex].astype(D)[None, :, None]
            wt = weights[t, j].astype(D)[:, None]
            o = part.sum(axis=2) * wt
            m = np.abs(part).sum(axis=2) * np.abs(wt)
            np.add.at(y, t, o)
            np.add.at(mag, t, m)
            np.add.at(e, t, (2 * h.shape[1] + 8 + 3) * U * m)
        e = e + k * U * (mag + e)
        if residual is not None:
            y = y + residual.astype(D)
            e = e + U * (np.abs(y) + e)
        return y, e + HALF[dtype] * (np.abs(y) + e) + 2.0 ** -130
