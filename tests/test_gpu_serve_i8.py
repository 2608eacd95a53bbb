"""8-bit rows with one scale each and their product on the GPU, through the
C-ABI, against the plain CPU forms: codes and scales bit for bit, products
within the bound that the header states (four fp32 roundings, and half a step
of bf16 where that is the output type)."""
import numpy as np
import pytest

import serve_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


def rows(n, k, seed, bf16):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, k)).astype(np.float32) * np.exp(rng.standard_normal((n, 1))).astype(np.float32)
    x[:, rng.random(k) < 0.01] *= 20
    t = torch.from_numpy(x)
    return t.to(torch.bfloat16) if bf16 else t


def check_quantized(codes, scales, x):
    c, d = plain.quantize_rows(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy().view(np.int32), d.view(np.int32))
    assert np.array_equal(codes.cpu().numpy(), c)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 7), (5, 128), (4, 129), (17, 1000), (2, 2048), (3, 2049), (1, 4096),
                                 (7, 11008), (2, 12289), (2, 40000), (1, 131072), (600, 96)])
def test_quantize_rows(sv, n, k, bf16):
    say(f"quantize {n}x{k} bf16={bf16}")
    x = rows(n, k, n * 7 + k, bf16)
    codes, scales = sv.qr_quantize_rows_i8(x.cuda())
    check_quantized(codes, scales, x)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("pad", [1, 3, 8, 56])
def test_quantize_strided_rows(sv, pad, bf16):
    say(f"quantize strided pad={pad}")
    x = rows(9, 500 + pad, pad, bf16)
    for first in (0, min(pad, 5)):
        part = x.cuda()[:, first:first + 500]
        codes, scales = sv.qr_quantize_rows_i8(part)
        check_quantized(codes, scales, x[:, first:first + 500])


def test_quantize_edge_rows(sv):
    say("quantize edge rows")
    x = rows(12, 700, 3, False)
    x[0] = 0
    x[1] = 1e-45                       # 127 / amax overflows
    x[2] = 3.4e38
    x[3, 5] = float("inf")
    x[4, 699] = float("nan")
    x[5] = float("-inf")
    x[6] = 0
    x[6, 300] = -2.0
    x[7] = 1e-37
    x[8] = torch.arange(700) - 350.5   # halves: ties to even
    x[9] = 127.0
    x[9, ::2] = 0.5
    codes, scales = sv.qr_quantize_rows_i8(x.cuda())
    c, d = plain.quantize_rows(x.numpy())
    got = scales.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(d)) and np.isnan(got[[3, 4, 5]]).all()
    assert np.array_equal(got[~np.isnan(d)].view(np.int32), d[~np.isnan(d)].view(np.int32))
    assert np.array_equal(codes.cpu().numpy(), c)


def check_product(sv, n_out, n_tok, n_in, dtype, bias, seed, out=None, extreme=False):
    rng = np.random.default_rng(seed)
    pitch = -(-n_in // 128) * 128
    w = np.zeros((n_out, pitch), np.int8)
    x = np.zeros((n_tok, pitch), np.int8)
    lo, hi = (-127, 128)
    w[:, :n_in] = 127 if extreme else rng.integers(lo, hi, (n_out, n_in))
    x[:, :n_in] = -127 if extreme else rng.integers(lo, hi, (n_tok, n_in))
    wd = np.exp(rng.standard_normal(n_out)).astype(np.float32) * np.float32(1e-3)
    xd = np.exp(rng.standard_normal(n_tok)).astype(np.float32) * np.float32(1e-2)
    b = rng.standard_normal(n_out).astype(np.float32) if bias else None
    cu = lambda a: None if a is None else torch.from_numpy(a).cuda()
    y = sv.qr_matmul_i8(cu(w), cu(wd), cu(x), cu(xd), n_in, bias=cu(b), dtype=dtype, out=out)
    ref, mag = plain.product(w, wd, x, xd, b)
    got = y.float().cpu().numpy().astype(np.float64)
    bound = 4 * 2.0 ** -24 * mag
    if y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside the bound, first at {np.argwhere(bad)[0]}"
    return y


SHAPES = [(1, 1, 1), (5, 1, 64), (17, 3, 129), (64, 64, 128), (65, 63, 256), (200, 1, 4096), (333, 16, 1000),
          (129, 17, 640), (256, 31, 2048), (100, 32, 2500), (40, 33, 384), (130, 100, 1024), (500, 64, 4096), (257, 129, 512),
          (300, 333, 1100), (512, 512, 256), (1000, 700, 640), (77, 2000, 192), (2304, 520, 384), (1900, 1801, 520), (3700, 3901, 200), (6200, 40, 300),
          (6145, 64, 1300), (4100, 200, 300), (2500, 2200, 140), (4096, 50, 300), (2048, 64, 700)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_out,n_tok,n_in", SHAPES)
def test_product(sv, n_out, n_tok, n_in, dtype):
    say(f"product {n_out}x{n_tok}x{n_in} {dtype}")
    check_product(sv, n_out, n_tok, n_in, dtype, (n_out + n_tok) % 2 == 0, n_out + 3 * n_tok + n_in)


@pytest.mark.parametrize("n_out,n_tok", [(70, 1), (70, 13), (70, 20), (140, 150), (6200, 30)])
def test_product_longest_sum(sv, n_out, n_tok):
    # 131072 products of 127 * -127: the whole range of the int32 sum
    say(f"product longest {n_out}x{n_tok}")
    check_product(sv, n_out, n_tok, 131072, torch.float32, False, 5, extreme=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_out,n_tok,pad,first", [(65, 3, 5, 0), (256, 70, 8, 8), (130, 300, 3, 1), (512, 512, 64, 0),
                                                    (4101, 200, 3, 1), (2049, 1800, 8, 4)])
def test_product_strided_output(sv, n_out, n_tok, pad, first, dtype):
    say(f"product strided {n_out}x{n_tok} pad={pad}")
    big = torch.full((n_tok, n_out + pad), 7.0, dtype=dtype, device="cuda")
    out = big[:, first:first + n_out]
    check_product(sv, n_out, n_tok, 300, dtype, True, 11, out=out)
    rest = torch.cat([big[:, :first], big[:, first + n_out:]], dim=1)
    assert bool((rest == 7.0).all())


def test_product_reproducible_and_independent_of_the_batch(sv):
    # the sum is exact: a token's outputs are the same bits in any batch
    say("product batch independence")
    w, wd = sv.qr_quantize_rows_i8(rows(2300, 1000, 1, True).cuda())
    x, xd = sv.qr_quantize_rows_i8(rows(2200, 1000, 2, True).cuda())
    full = sv.qr_matmul_i8(w, wd, x, xd, 1000, dtype=torch.float32)
    for n in (1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 128, 129, 256, 257, 500, 1000, 1500):
        part = sv.qr_matmul_i8(w, wd, x[:n].contiguous(), xd[:n].contiguous(), 1000, dtype=torch.float32)
        assert torch.equal(part, full[:n]), n


def test_nan_rows_stay_apart(sv):
    say("product NaN rows")
    a, b = rows(70, 300, 5, False), rows(40, 300, 6, False)
    b[7, 3] = float("nan")
    a[11, 0] = float("inf")
    w, wd = sv.qr_quantize_rows_i8(a.cuda())
    for n in (40, 9):
        x, xd = sv.qr_quantize_rows_i8(b[:n].cuda())
        y = sv.qr_matmul_i8(w, wd, x, xd, 300, dtype=torch.float32).cpu()
        nan = torch.isnan(y)
        want = torch.zeros_like(nan)
        want[7] = True
        want[:, 11] = True
        assert torch.equal(nan, want)


def test_empty_calls(sv):
    say("empty")
    c, d = sv.qr_quantize_rows_i8(torch.zeros((0, 64), device="cuda"))
    assert c.shape == (0, 128) and d.shape == (0,)
    w, wd = sv.qr_quantize_rows_i8(torch.ones((3, 64), device="cuda"))
    assert sv.qr_matmul_i8(w, wd, c, d, 64).shape == (0, 3)
    assert sv.qr_matmul_i8(c, d, w, wd, 64).shape == (3, 0)


def test_other_stream_and_graph(sv):
    say("stream and graph")
    a = rows(200, 640, 8, True).cuda()
    w, wd = sv.qr_quantize_rows_i8(a)
    for n_tok in (1, 20, 150):
        src = [rows(n_tok, 640, 20 + i, True).cuda() for i in range(3)]
        x = src[0].clone()
        y = torch.empty((n_tok, 200), dtype=torch.bfloat16, device="cuda")
        codes, scales = sv.qr_quantize_rows_i8(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            sv.qr_quantize_rows_i8(x, codes, scales)
            sv.qr_matmul_i8(w, wd, codes, scales, 640, out=y)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.qr_quantize_rows_i8(x, codes, scales)
            sv.qr_matmul_i8(w, wd, codes, scales, 640, out=y)
        for s in src + src[:1]:
            x.copy_(s)
            y.fill_(-1)
            g.replay()
            torch.cuda.synchronize()
            c, d = sv.qr_quantize_rows_i8(s)
            assert torch.equal(y, sv.qr_matmul_i8(w, wd, c, d, 640))
