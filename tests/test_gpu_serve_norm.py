"""The norm that makes 8-bit rows on the GPU, against the plain form: totals bit
for bit; scales, codes and normed rows too, but where the last bits of a 64-bit
sum could move a value across a rounding (within 2^-20 of one, of which 2^-52
times a sum of up to 2^17 terms is a small part)."""
import numpy as np
import pytest

import serve_layer_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


def rows(n, k, seed, dtype, size=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, k)).astype(F) * np.exp(rng.standard_normal((n, 1))).astype(F)
    x[:, rng.random(k) < 0.01] *= 20
    return torch.from_numpy(x * F(size)).to(dtype)


def check(got, x, residual, weight, eps, want_y):
    """got: what the call returned; x, residual, weight: CPU tensors."""
    codes, scales, total, y = got
    np_of = lambda t: None if t is None else t.float().cpu().numpy()
    n = x.shape[1]
    t64, y64 = plain.norm(np_of(x), np_of(residual), np_of(weight), eps, x.dtype)
    if residual is None:
        assert total is None
    else:
        assert total.dtype == x.dtype and np.array_equal(np_of(total).view(np.int32), t64.view(np.int32))
    c, d, p = plain.code_rule(y64)
    got_d, got_c = scales.cpu().numpy(), codes.cpu().numpy()
    assert np.array_equal(np.isnan(got_d), np.isnan(d))
    fine = ~np.isnan(d)
    assert np.all(np.abs(got_d[fine] - d[fine]) <= 2.0 ** -23 * d[fine])
    assert got_c.shape == (x.shape[0], -(-n // 128) * 128) and not got_c[:, n:].any()
    off = got_c[:, :n].astype(int) - c
    near = np.abs(np.abs(p.astype(np.float64) - np.floor(p)) - 0.5) < 2.0 ** -13   # 2^-20 of a code of up to 127
    assert not off[~near].any() and np.abs(off).max(initial=0) <= 1 and np.count_nonzero(off) <= 1 + off.size // 100000
    if want_y:
        assert y.dtype == x.dtype
        w = plain.rounded(y64, x.dtype)
        g = np_of(y)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        ok = ~np.isnan(w)
        step = 2.0 ** -23 if x.dtype == torch.float32 else 2.0 ** -7
        differ = g[ok] != w[ok]
        assert np.count_nonzero(differ) <= 1 + differ.size // 100000
        assert np.all(np.abs(g[ok][differ] - w[ok][differ]) <= step * np.abs(w[ok][differ]) + 2.0 ** -140)
    else:
        assert y is None


SIZES = [(1, 1), (3, 7), (5, 128), (4, 129), (9, 511), (6, 512), (2, 513), (17, 1000), (2, 2048), (3, 2049), (1, 4096),
         (5, 4100), (3, 7168), (2, 8192), (3, 8200), (2, 11008), (2, 16384), (2, 16392), (1, 40001), (1, 131072),
         (600, 96), (70, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,k", SIZES)
def test_norm(sv, n, k, dtype):
    say(f"norm {n}x{k} {dtype}")
    x, r = rows(n, k, n * 3 + k, dtype), rows(n, k, n * 5 + k, dtype, 3.0)
    for wtype, residual, y in ((dtype, r, True), (torch.float32, None, False), (torch.bfloat16, r, False),
                               (None, None, True)):
        w = None if wtype is None else (1 + 0.2 * rows(1, k, k, torch.float32)[0]).to(wtype)
        cuda = lambda t: None if t is None else t.cuda()
        got = sv.qr_norm_rows_i8(x.cuda(), cuda(w), 1e-5, residual=cuda(residual), y=y)
        check(got, x, residual, w, 1e-5, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [100, 4000, 20000])
def test_in_place(sv, k, dtype):
    say(f"in place {k} {dtype}")
    x, r = rows(3, k, 1, dtype), rows(3, k, 2, dtype)
    w = rows(1, k, 3, dtype)[0]
    for which in ("total is x", "total is residual", "y is x", "y is residual", "total is residual, y is x",
                  "total is x, y is residual"):
        gx, gr = x.cuda(), r.cuda()
        kw = {}
        for part in which.split(", "):
            name, of = part.split(" is ")
            kw[name] = gx if of == "x" else gr
        got = sv.qr_norm_rows_i8(gx, w.cuda(), 0.0, residual=gr, **kw)
        for name, t in kw.items():
            assert got[2 if name == "total" else 3] is t
        check(got, x, r, w, 0.0, "y" in kw)
        for t, before, name in ((gx, x, "x"), (gr, r, "residual")):   # what is no output is as it was
            if all(of is not t for of in kw.values()):
                assert torch.equal(t.cpu(), before), name
    gx = x.cuda()
    check(sv.qr_norm_rows_i8(gx, w.cuda(), 0.0, y=gx), x, None, w, 0.0, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [1, 3, 8, 40])
def test_strided_rows(sv, pad, dtype):
    say(f"strided pad={pad} {dtype}")
    k = 700
    whole = [rows(6, k + pad, s, dtype) for s in range(4)]
    gpu = [t.cuda() for t in whole]
    for first in (0, min(pad, 5)):
        part = [t[:, first:first + k] for t in gpu]
        got = sv.qr_norm_rows_i8(part[0], None, 1e-6, residual=part[1], total=part[2], y=part[3])
        check(got, whole[0][:, first:first + k], whole[1][:, first:first + k], None, 1e-6, True)
        for t, before in zip(gpu[2:], whole[2:]):   # nothing beside the rows was written
            keep = torch.ones(k + pad, dtype=torch.bool)
            keep[first:first + k] = False
            assert torch.equal(t.cpu()[:, keep], before[:, keep])
        gpu[2].copy_(whole[2]), gpu[3].copy_(whole[3])


def test_values_out_of_the_ordinary(sv):
    say("special values")
    k = 600
    x = rows(12, k, 9, torch.float32)
    x[0] = 0                                   # eps alone
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] *= 1e38 / x[3].abs().max()            # squares beyond fp32
    x[4] *= 1e-40 / x[4].abs().max()           # subnormal values
    x[5] = 3e38
    x[6, 1:] = 0                               # one value
    x[7] = -1e-30
    x[8, 3] = float("-inf")
    w = torch.ones(k)
    w[11] = 0.0
    got = sv.qr_norm_rows_i8(x.cuda(), w.cuda(), 1e-12, y=True)
    check(got, x, None, w, 1e-12, True)
    assert got[1][0].item() == 0.0 and torch.isnan(got[1][[1, 2, 8]]).all() and not torch.isnan(got[1][[3, 4, 5, 6, 7]]).any()
    got = sv.qr_norm_rows_i8(x.cuda(), w.cuda(), 0.0)
    check(got, x, None, w, 0.0, False)
    assert torch.isnan(got[1][0]).item()       # 0 / 0
    # a sum that overflows, a weight that is no number, one that overflows the row
    big = torch.full((2, k), 3e38)
    got = sv.qr_norm_rows_i8(big.cuda(), None, 1e-6, residual=big.cuda())
    assert torch.isinf(got[2]).all() and torch.isnan(got[1]).all() and not got[0].any()
    w[3] = float("nan")
    assert torch.isnan(sv.qr_norm_rows_i8(x[9:].cuda(), w.cuda())[1]).all()
    x[9] = 0
    x[9, 0] = 1
    w[3], w[0] = 1.0, 3e38
    got = sv.qr_norm_rows_i8(x[9:10].cuda(), w.cuda())
    assert torch.isnan(got[1]).all() and not got[0].any()


def test_largest_rows_and_none(sv):
    say("rows 0 and 70000")
    got = sv.qr_norm_rows_i8(torch.empty((0, 64), device="cuda"), None)
    assert got[0].shape == (0, 128) and got[1].shape == (0,)
    x = rows(70000, 33, 4, torch.bfloat16)
    check(sv.qr_norm_rows_i8(x.cuda(), None, 1e-6, y=True), x, None, None, 1e-6, True)


def test_graph_and_stream(sv):
    say("graph")
    x, r, w = (t.cuda() for t in (rows(5, 4096, 1, torch.bfloat16), rows(5, 4096, 2, torch.bfloat16),
                                  rows(1, 4096, 3, torch.bfloat16)[0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.qr_norm_rows_i8(x, w, residual=r, y=True, stream=side)
    side.synchronize()
    check(got, x.cpu(), r.cpu(), w.cpu(), 1e-6, True)
    out = [t.clone() for t in got]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_norm_rows_i8(x, w, residual=r, total=out[2], y=out[3], codes=out[0], scales=out[1])
    for seed in (5, 6, 7):
        nx = rows(5, 4096, seed, torch.bfloat16)
        x.copy_(nx)
        g.replay()
        torch.cuda.synchronize()
        check(out, nx, r.cpu(), w.cpu(), 1e-6, True)
        eager = sv.qr_norm_rows_i8(x, w, residual=r, y=True)
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
