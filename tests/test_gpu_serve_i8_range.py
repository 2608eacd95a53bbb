"""Products of 8-bit rows whose scales lie near the ends of fp32, against
64-bit arithmetic: an output is finite wherever its value is."""
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


# one of each tile: up to 16 tokens, 32, 64, and the LDS tiles
SHAPES = [(70, 3), (200, 30), (4100, 40), (130, 100), (1000, 700), (2500, 2200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_out,n_tok", SHAPES)
def test_scales_near_the_ends_of_fp32(sv, n_out, n_tok, dtype):
    """Four fp32 roundings of the magnitude, half a step of the smallest fp32
    value for each of the last two (what is below 2^-126), and bf16's half
    step, whose smallest is 2^-134."""
    say(f"range {n_out}x{n_tok} {dtype}")
    rng = np.random.default_rng(n_out)
    n_in = 300
    w = np.zeros((n_out, 384), np.int8)
    x = np.zeros((n_tok, 384), np.int8)
    w[:, :n_in] = rng.integers(-127, 128, (n_out, n_in))
    x[:, :n_in] = rng.integers(-127, 128, (n_tok, n_in))
    # 2^-128 .. 2^121: the scales that the row quantizer can give
    xd = np.float32(2.0) ** rng.integers(-127, 121, n_tok).astype(np.float32) * rng.uniform(1, 2, n_tok).astype(np.float32)
    wd = np.float32(2.0) ** rng.integers(-127, 121, n_out).astype(np.float32) * rng.uniform(1, 2, n_out).astype(np.float32)
    xd[:3] = np.array([2.0 ** 121, 2.0 ** -128, 2.0 ** 96.5], np.float32)[:min(3, n_tok)]
    wd[:4] = np.array([2.0 ** -30, 2.0 ** 121, 2.0 ** -128, 1.0], np.float32)
    b = rng.standard_normal(n_out).astype(np.float32)
    cu = lambda a: torch.from_numpy(a).cuda()
    for bias in (None, b):
        y = sv.qr_matmul_i8(cu(w), cu(wd), cu(x), cu(xd), n_in, bias=None if bias is None else cu(bias), dtype=dtype)
        got = y.double().cpu().numpy()
        ref, mag = plain.product(w, wd, x, xd, bias)
        bound = 4 * 2.0 ** -24 * mag + 2 * 2.0 ** -150
        most = float(torch.finfo(dtype).max)
        if dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -134
        assert not np.isnan(got).any()
        inside = np.abs(ref) + bound < most
        assert inside.any() and not inside.all()
        assert np.all(np.abs(got - ref)[inside] <= bound[inside])
        assert np.all(np.abs(got)[np.abs(ref) - bound > most * (1 + 2.0 ** -8)] == np.inf)


def test_loud_tokens_from_the_quantizer(sv):
    say("loud tokens")
    g = torch.Generator().manual_seed(1)
    x = torch.randn((20, 500), generator=g)
    x[3] *= 5e37 / x[3].abs().max()
    x[4] *= 3.3e38 / x[4].abs().max()
    a = torch.randn((90, 500), generator=g) * 0.001
    w, wd = sv.qr_quantize_rows_i8(a.cuda())
    codes, d = sv.qr_quantize_rows_i8(x.cuda())
    for n in (20, 9):
        y = sv.qr_matmul_i8(w, wd, codes[:n].contiguous(), d[:n].contiguous(), 500, dtype=torch.float32).cpu()
        ref, mag = plain.product(w.cpu().numpy(), wd.cpu().numpy(), codes[:n].cpu().numpy(), d[:n].cpu().numpy())
        assert torch.isfinite(y).all()
        assert np.all(np.abs(y.double().numpy() - ref) <= 4 * 2.0 ** -24 * mag)
