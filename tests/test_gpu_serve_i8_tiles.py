"""Every tile of the 8-bit product with what its epilogue has to carry through
LDS: ragged channels and tokens, rows far apart, scales of every size, a NaN,
and nothing written behind the last token or channel."""
import numpy as np
import pytest

from test_gpu_serve_i8_ex import call, case, check, dev, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


# 64x64 in four parts, 64x128 and 128x128 in two, 128x128, 256x256: one round
# of it that is half full, and more; a single step of the sum, and several
TILES = [(70, 1001, 90), (130, 6003, 300), (500, 5002, 130), (1290, 4003, 90), (1500, 5701, 257), (3001, 6401, 70)]
KINDS = [("none", False, False), ("relu", False, True), ("silu", True, False), ("gelu_tanh", True, True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,r,k", TILES)
def test_tiles(sv, t, r, k, dtype):
    for i, (act, up, residual) in enumerate(KINDS):
        if i % 2 and t * r > 5000000:
            continue
        say(f"tile {t}x{r}x{k} {dtype} {act} up={up} residual={residual}")
        c = case(t, r, k, dtype, up, i % 2 == 0, residual, seed=i)
        c["x"][1][:: 17] *= np.float32(2.0 ** -60)
        if act in ("none", "relu"):
            c["x"][1][5:: 29] *= np.float32(2.0 ** 110)
        c["x"][1][3:: 41] = 0.0
        first, pad = i % 3, 3 + i
        big = torch.full((t + 2, r + first + pad), 7.0, dtype=dtype, device="cuda")
        out = big[1:t + 1, first:first + r]
        args = dict(out=out)
        if residual:
            out.copy_(dev(c["residual"]))
            args["residual"] = out
        y = call(sv, c, k, act, dtype, **args)
        check(y, c, k, act, dtype)
        big[1:t + 1, first:first + r] = 7.0
        assert torch.equal(big, torch.full_like(big, 7.0))


@pytest.mark.parametrize("t,r,k", [(70, 1001, 90), (500, 5002, 130), (1500, 5701, 257)])
def test_a_scale_that_is_no_number(sv, t, r, k):
    for act, up in (("none", False), ("silu", True)):
        say(f"nan {t}x{r}x{k} {act}")
        c = case(t, r, k, torch.float32, up, False, False)
        want = call(sv, c, k, act, torch.float32)
        bad = [0, 31, 32, t // 2, t - 1]
        c["x"][1][bad] = np.nan
        y = call(sv, c, k, act, torch.float32)
        assert torch.isnan(y[bad]).all()
        y[bad] = want[bad]
        assert torch.equal(y, want)


def test_the_same_sums_in_every_tile(sv):
    """One row of x among few and many tokens: the same bits."""
    say("tiles agree")
    k, r = 700, 3001
    c = case(3000, r, k, torch.float32, True, True, False)
    row = call(sv, {**c, "x": (c["x"][0][:1].copy(), c["x"][1][:1].copy())}, k, "silu", torch.float32)[0]
    for t in (2, 20, 40, 64, 100, 400, 900, 3000):
        x = (c["x"][0][:t].copy(), c["x"][1][:t].copy())
        x[0][t - 1], x[1][t - 1] = c["x"][0][0], c["x"][1][0]
        y = call(sv, {**c, "x": x}, k, "silu", torch.float32)
        assert torch.equal(y[0], row) and torch.equal(y[t - 1], row), t
