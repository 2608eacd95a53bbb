"""The 8-bit product with an epilogue on the GPU, against 64 bits: products
within four fp32 roundings, an activation within 8 * 2^-24 of its argument, a
rounding for the gate's product, the residual and the output each."""
import itertools

import numpy as np
import pytest

import serve_layer_plain as plain
import serve_plain

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


def codes(n, k, seed, size=1.0):
    rng = np.random.default_rng(seed)
    c = np.zeros((n, -(-k // 128) * 128), dtype=np.int8)
    c[:, :k] = rng.integers(-127, 128, (n, k))
    d = (size * np.exp(0.5 * rng.standard_normal(n)) / 127 / 73 / np.sqrt(k)).astype(np.float32)
    return c, d


def case(t, r, k, dtype, up, bias, residual, seed=0):
    rng = np.random.default_rng(seed + 17)
    x, xd = codes(t, k, seed + 1)
    xd = (xd * 127 * 2).astype(np.float32)
    c = {"x": (x, xd), "w": codes(r, k, seed + 2, 127.0), "bias": None, "up": None, "residual": None}
    vec = lambda: rng.standard_normal(r).astype(np.float32)
    if bias:
        c["bias"] = vec()
    if up:
        c["up"] = codes(r, k, seed + 3, 127.0) + ((vec() if bias else None),)
    if residual:
        c["residual"] = torch.from_numpy(rng.standard_normal((t, r)).astype(np.float32)).to(dtype)
    return c


def dev(a):
    return None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()


def call(sv, c, k, act, dtype, **kw):
    up = c["up"] or (None, None, None)
    kw.setdefault("residual", dev(c["residual"]))
    return sv.qr_matmul_i8_ex(dev(c["w"][0]), dev(c["w"][1]), dev(c["x"][0]), dev(c["x"][1]), k, bias=dev(c["bias"]),
                              act=act, up=dev(up[0]), upd=dev(up[1]), up_bias=dev(up[2]), dtype=dtype, **kw)


def check(y, c, k, act, dtype):
    cut = lambda p: None if p is None else (p[0][:, :k],) + tuple(p[1:])
    w, x, up = cut(c["w"]), cut(c["x"]), cut(c["up"])
    want, bound = plain.product(w[0], w[1], x[0], x[1], c["bias"], act, up,
                                None if c["residual"] is None else c["residual"].float().numpy(), dtype)
    got = y.float().cpu().numpy().astype(np.float64)
    assert y.dtype == dtype and got.shape == want.shape
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


# every kernel that the rule chooses, with ragged edges: few tokens, tiles in
# four and two parts, whole tiles up to 256 x 256
SHAPES = [(1, 1, 1), (1, 3, 130), (5, 30, 200), (16, 100, 4100), (17, 33, 64), (33, 130, 700), (48, 4097, 128),
          (64, 1000, 300), (20, 3001, 1000), (65, 200, 129), (100, 2050, 384), (129, 3001, 256), (300, 4100, 520),
          (700, 2000, 100), (1030, 4001, 140), (2500, 5000, 90)]
KINDS = [("silu", True, False, False), ("none", False, True, True), ("gelu", False, True, False),
         ("gelu_tanh", True, True, True), ("relu", False, False, True), ("none", True, False, False)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,r,k", SHAPES)
def test_product_with_epilogue(sv, t, r, k, dtype):
    for act, up, bias, residual in KINDS if t * r < 3000000 else KINDS[:2]:
        say(f"{t}x{r}x{k} {dtype} {act} up={up} bias={bias} residual={residual}")
        c = case(t, r, k, dtype, up, bias, residual)
        check(call(sv, c, k, act, dtype), c, k, act, dtype)


def test_without_an_epilogue_it_is_the_plain_product(sv):
    say("plain")
    for t, r, k in ((3, 40, 300), (200, 700, 300)):
        c = case(t, r, k, torch.float32, False, True, False)
        args = [dev(c["w"][0]), dev(c["w"][1]), dev(c["x"][0]), dev(c["x"][1])]
        a = sv.qr_matmul_i8(*args, k, bias=dev(c["bias"]), dtype=torch.float32)
        assert torch.equal(a, call(sv, c, k, "none", torch.float32))
        # an epilogue changes nothing in the products themselves
        zero = torch.zeros((t, r), device="cuda")
        assert torch.equal(a, call(sv, c, k, "none", torch.float32, residual=zero))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,r", [(4, 50), (70, 300), (600, 2000)])
def test_residual_in_place_and_strides(sv, t, r, dtype):
    say(f"in place {t}x{r} {dtype}")
    k = 150
    c = case(t, r, k, dtype, True, False, True)
    y = dev(c["residual"]).clone()
    assert call(sv, c, k, "silu", dtype, residual=y, out=y) is y
    check(y, c, k, "silu", dtype)
    wide = torch.full((t, r + 7), 3.0, dtype=dtype, device="cuda")
    wide[:, 3:3 + r] = dev(c["residual"])
    call(sv, c, k, "silu", dtype, residual=wide[:, 3:3 + r], out=wide[:, 3:3 + r])
    check(wide[:, 3:3 + r], c, k, "silu", dtype)
    assert (wide[:, :3] == 3).all() and (wide[:, 3 + r:] == 3).all()
    # side by side in one buffer
    both = torch.full((t, 2 * r + 5), 3.0, dtype=dtype, device="cuda")
    both[:, :r] = dev(c["residual"])
    call(sv, c, k, "silu", dtype, residual=both[:, :r], out=both[:, r:2 * r])
    check(both[:, r:2 * r], c, k, "silu", dtype)
    assert torch.equal(both[:, :r], dev(c["residual"])) and (both[:, 2 * r:] == 3).all()


def test_activations_over_their_whole_range(sv):
    """One channel of code 1 and scale 1: p is the token's scale times its code."""
    say("range")
    v = np.concatenate([np.linspace(-110, 110, 4001), np.linspace(-4, 4, 4001), 10.0 ** np.linspace(-40, 38, 200),
                        -10.0 ** np.linspace(-40, 38, 200)]).astype(np.float32)
    t = len(v)
    x = np.zeros((t, 128), dtype=np.int8)
    x[:, 0] = 1
    w = np.zeros((3, 128), dtype=np.int8)
    w[:, 0] = 1
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        for n in (t, 16):
            y = sv.qr_matmul_i8_ex(dev(w), torch.ones(3, device="cuda"), dev(x[:n]), dev(v[:n]), 1, act=act,
                                   dtype=torch.float32)
            want = plain.act(act, v[:n].astype(np.float64))
            bound = plain.ACT_ERROR * np.abs(v[:n].astype(np.float64)) + 2.0 ** -110
            assert np.all(np.abs(y.cpu().numpy()[:, 1] - want) <= bound), act


def test_infinities_and_nan_stay_in_their_token(sv):
    say("inf, nan")
    t, r, k = 40, 60, 100
    c = case(t, r, k, torch.float32, True, False, True)
    c["x"][1][3] = np.nan
    c["x"][1][5] = np.inf
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        y = call(sv, c, k, act, torch.float32).cpu()
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[5]).any()
        keep = [i for i in range(t) if i not in (3, 5)]
        assert torch.isfinite(y[keep]).all()
    # an infinite product: silu and gelu let it through
    x = np.zeros((1, 128), dtype=np.int8)
    x[0, 0] = 127
    y = sv.qr_matmul_i8_ex(dev(x), torch.full((1,), 3e38, device="cuda"), dev(x), torch.ones(1, device="cuda"), 1,
                           act="silu", dtype=torch.float32)
    assert torch.isinf(y).all()


def test_graph_and_stream(sv):
    say("graph")
    t, r, k = 20, 500, 1000
    c = case(t, r, k, torch.bfloat16, True, True, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(call(sv, c, k, "silu", torch.bfloat16, stream=side), c, k, "silu", torch.bfloat16)
    args = [dev(c["w"][0]), dev(c["w"][1]), dev(c["x"][0]), dev(c["x"][1])]
    kw = dict(bias=dev(c["bias"]), act="silu", up=dev(c["up"][0]), upd=dev(c["up"][1]), up_bias=dev(c["up"][2]),
              residual=dev(c["residual"]), out=torch.empty((t, r), dtype=torch.bfloat16, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_matmul_i8_ex(*args, k, **kw)
    for seed in (7, 8, 9):
        c["x"] = (codes(t, k, seed)[0], c["x"][1])
        args[2].copy_(torch.from_numpy(c["x"][0]))
        g.replay()
        torch.cuda.synchronize()
        check(kw["out"], c, k, "silu", torch.bfloat16)
        assert torch.equal(kw["out"], sv.qr_matmul_i8_ex(*args, k, **{**kw, "out": None}))
