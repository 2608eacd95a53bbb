"""The router and the experts on the GPU, against 64 bits: the choice equal, its
weights within one rounding to fp32 (and 2^-40 for sums and exp in 64 bits), the
experts' output within the bound that serve_layer_plain.experts derives."""
import numpy as np
import pytest

import serve_layer_plain as plain

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


def dev(a):
    return None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()


# --------------------------------------------------------------------------
# the router

def route_case(t, e, k, seed, xtype=torch.float32, wtype=torch.float32):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).to(xtype)
    w = torch.from_numpy((rng.standard_normal((e, k)) * 2 / np.sqrt(k)).astype(np.float32)).to(wtype)
    return x, w, (0.2 * rng.standard_normal(e)).astype(np.float32)


def check_route(got, x, w, top_k, score, bias, renorm, factor):
    ids, weights = got
    want, wt = plain.route(x.double().numpy(), w.double().numpy(), top_k, score, bias, renorm, np.float32(factor))
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want)
    g = weights.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(wt))
    assert np.all((np.abs(g - wt) <= (plain.U + 2.0 ** -40) * np.abs(wt) + 2.0 ** -150) | np.isnan(wt))


ROUTES = [(1, 1, 1, 1), (1, 2, 33, 2), (1, 256, 7168, 8), (2, 5, 100, 3), (3, 64, 31, 6), (15, 65, 1000, 4),
          (16, 16, 64, 16), (17, 300, 129, 8), (33, 1000, 96, 64), (40, 1024, 500, 1), (130, 100, 2000, 6),
          (300, 256, 640, 8), (1500, 160, 72, 8), (5000, 8, 40, 2), (600, 520, 257, 5)]


@pytest.mark.parametrize("t,e,k,top_k", ROUTES)
def test_route(sv, t, e, k, top_k):
    types = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32),
             (torch.float32, torch.bfloat16)]
    for i, (xt, wt) in enumerate(types):
        score, renorm, factor = ("softmax", "sigmoid")[i % 2], i < 2, (1.0, 2.5)[i // 2]
        say(f"route {t}x{e}x{k} top {top_k} {xt} {wt} {score}")
        x, w, b = route_case(t, e, k, 10 * i + e, xt, wt)
        b = b if i in (1, 2) else None
        got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(b), renorm=renorm, factor=factor)
        check_route(got, x, w, top_k, score, b, renorm, factor)


@pytest.mark.parametrize("t", [3, 900])
def test_equal_scores_go_to_the_lowest_index(sv, t):
    say(f"ties {t}")
    x, w, _ = route_case(t, 40, 200, 3)
    w = w[torch.arange(40) % 8].contiguous()       # five of each
    got = sv.qr_moe_route(x.cuda(), w.cuda(), 12)
    check_route(got, x, w, 12, "softmax", None, True, 1.0)
    zero = torch.zeros_like(x)
    got = sv.qr_moe_route(zero.cuda(), w.cuda(), 7, score="sigmoid")
    assert (got[0].cpu() == torch.arange(7)).all() and torch.allclose(got[1].cpu(), torch.full((t, 7), 1 / 7))


def test_experts_that_are_switched_off(sv):
    say("off")
    x, w, b = route_case(9, 12, 50, 4)
    b[[0, 3, 4, 5, 7, 9, 10, 11]] = -np.inf
    for renorm in (False, True):
        got = sv.qr_moe_route(x.cuda(), w.cuda(), 6, bias=dev(b), renorm=renorm)
        check_route(got, x, w, 6, "softmax", b, renorm, 1.0)
        assert (got[0][:, 4:] == -1).all() and (got[1][:, 4:] == 0).all()
    b[:] = -np.inf
    got = sv.qr_moe_route(x.cuda(), w.cuda(), 6, bias=dev(b))
    assert (got[0] == -1).all() and (got[1] == 0).all()


def test_rows_that_are_no_numbers(sv):
    say("nan")
    x, w, b = route_case(6, 20, 70, 5)
    x[1, 3] = float("nan")
    x[2, 4] = float("inf")
    x[4] *= 1e30                                    # exp of far apart logits
    for score in ("softmax", "sigmoid"):
        got = sv.qr_moe_route(x.cuda(), w.cuda(), 4, score=score)
        check_route(got, x, w, 4, score, None, True, 1.0)
        assert torch.isnan(got[1][1]).all() and (got[0] >= 0).all()
    # scores that all underflow: weights of zero, not 0 / 0
    far = torch.full((1, 70), -1e6)
    got = sv.qr_moe_route(far.cuda(), torch.ones((5, 70), device="cuda"), 2, score="sigmoid")
    assert (got[1] == 0).all() and got[0].tolist() == [[0, 1]]


def test_route_strided_rows_and_none(sv):
    say("strided")
    x, w, _ = route_case(20, 30, 115, 6, torch.bfloat16, torch.bfloat16)
    w = w[:, :100].contiguous()
    for first in (0, 1, 15):
        part = x[:, first:first + 100]
        check_route(sv.qr_moe_route(x.cuda()[:, first:first + 100], w.cuda(), 3), part, w, 3, "softmax", None, True, 1.0)
    ids, wt = sv.qr_moe_route(x[:0, :100].cuda(), w.cuda(), 3)
    assert ids.shape == (0, 3) and wt.shape == (0, 3)


@pytest.mark.parametrize("t", [2, 300])
def test_route_graph_and_stream(sv, t):
    say(f"route graph {t}")
    x, w, b = route_case(t, 64, 512, 8)
    gx, gw, gb = x.cuda(), w.cuda(), dev(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.qr_moe_route(gx, gw, 4, bias=gb, stream=side)
    side.synchronize()
    check_route(got, x, w, 4, "softmax", b, True, 1.0)
    ws = torch.empty(sv.qr_moe_route_workspace_bytes(64, t, 512), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(o) for o in got]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_moe_route(gx, gw, 4, bias=gb, ids=out[0], weights=out[1], workspace=ws)
    for seed in (1, 2, 3):
        nx = route_case(t, 64, 512, seed)[0]
        gx.copy_(nx)
        ws.fill_(255)                              # what scratch memory holds does not matter
        g.replay()
        torch.cuda.synchronize()
        check_route(out, nx, w, 4, "softmax", b, True, 1.0)


# --------------------------------------------------------------------------
# the experts

def rows(rng, shape, n, size):
    c = np.zeros(shape + (-(-n // 128) * 128,), dtype=np.int8)
    c[..., :n] = rng.integers(-127, 128, shape + (n,))
    return c, (size * np.exp(0.3 * rng.standard_normal(shape)) / (73 * np.sqrt(n))).astype(np.float32)


class Case:
    def __init__(self, t, e, k, n_in, n_mid, seed=0, stacked=False):
        rng = np.random.default_rng(seed)
        self.n_in, self.n_mid = n_in, n_mid
        full, self.layer = {}, {}
        for name, r, n in (("gate", n_mid, n_in), ("up", n_mid, n_in), ("down", n_in, n_mid)):
            full[name], self.layer[name + "d"] = rows(rng, (e, r), n, 1.0)
            self.layer[name] = full[name][..., :n]
        self.layer["gated"], self.layer["upd"], self.layer["downd"] = (self.layer[n + "d"] for n in ("gate", "up", "down"))
        self.x, self.xd = rows(rng, (t,), n_in, 1.0)
        self.xd = (self.xd * np.float32(np.sqrt(n_in))).astype(np.float32)
        self.ids = np.stack([rng.permutation(e)[:k] for _ in range(t)]).astype(np.int32).reshape(t, k)
        self.weights = rng.random((t, k)).astype(np.float32)
        self.residual = rng.standard_normal((t, n_in)).astype(np.float32)
        self.full, self.stacked = full, stacked

    def experts(self, sv):
        g, u = dev(self.full["gate"]), dev(self.full["up"])
        gd, ud = dev(self.layer["gated"]), dev(self.layer["upd"])
        if self.stacked:
            both, scales = torch.cat([g, u], dim=1), torch.cat([gd, ud], dim=1)
            g, u, gd, ud = both[:, :self.n_mid], both[:, self.n_mid:], scales[:, :self.n_mid], scales[:, self.n_mid:]
        return sv.MoeExperts(g, gd, u, ud, dev(self.full["down"]), dev(self.layer["downd"]), self.n_in, self.n_mid)

    def run(self, sv, dtype, act="silu", residual=True, **kw):
        res = torch.from_numpy(self.residual).to(dtype).cuda() if residual else None
        kw.setdefault("residual", res)
        return sv.qr_moe_i8(dev(self.x), dev(self.xd), self.experts(sv), dev(self.ids), dev(self.weights), act=act,
                            dtype=dtype, **kw)

    def check(self, y, dtype, act="silu", residual=True):
        res = plain.rounded(self.residual, dtype) if residual else None
        want, bound = plain.experts(self.layer, self.x[:, :self.n_in], self.xd, self.ids, self.weights, act, res, dtype)
        got = y.float().cpu().numpy().astype(np.float64)
        assert y.dtype == dtype and got.shape == want.shape
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.all(np.abs(got[ok] - want[ok]) <= bound[ok]), np.max(np.abs(got[ok] - want[ok]) / bound[ok])


EXPERTS = [(1, 1, 1, 1, 1), (1, 2, 1, 100, 64), (1, 16, 8, 300, 70), (1, 300, 8, 128, 128), (2, 4, 2, 130, 200),
           (3, 8, 8, 129, 63), (5, 7, 3, 1000, 65), (16, 8, 2, 256, 512), (17, 5, 1, 400, 129), (23, 8, 2, 260, 1100),
           (33, 2, 2, 140, 300), (64, 32, 8, 200, 192), (70, 3, 1, 333, 100), (130, 4, 4, 100, 260), (65, 64, 6, 150, 64),
           (9, 1024, 64, 64, 64), (250, 40, 4, 80, 130)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,e,k,n_in,n_mid", EXPERTS)
def test_experts(sv, t, e, k, n_in, n_mid, dtype):
    say(f"experts {t} tokens, {k} of {e}, {n_in}x{n_mid} {dtype}")
    c = Case(t, e, k, n_in, n_mid, seed=t + e, stacked=t % 2 == 1)
    c.check(c.run(sv, dtype), dtype)
    c.check(c.run(sv, dtype, residual=False), dtype, residual=False)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
def test_activations(sv, act):
    say(f"experts {act}")
    c = Case(7, 5, 2, 200, 150, seed=3)
    c.check(c.run(sv, torch.float32, act=act), torch.float32, act=act)


@pytest.mark.parametrize("t,e,k", [(5, 6, 3), (70, 9, 4), (40, 3, 12)])
def test_absent_and_repeated_experts(sv, t, e, k):
    """Ids outside the experts add nothing, whatever their weight; the same
    expert twice counts twice."""
    say(f"absent {t} {e} {k}")
    c = Case(t, e, min(k, e), 150, 100, seed=k)
    rng = np.random.default_rng(1)
    c.ids = rng.integers(-2, e + 2, (t, k)).astype(np.int32)
    c.ids[0] = -1                                  # a padded token
    c.ids[1] = e - 1                               # one expert in every slot
    c.ids[2, 0], c.ids[2, -1] = 2 ** 31 - 1, -2 ** 31
    c.weights = rng.random((t, k)).astype(np.float32)
    c.weights[(c.ids < 0) | (c.ids >= e)] = np.nan
    c.check(c.run(sv, torch.float32), torch.float32)
    c.ids[:] = -1
    y = c.run(sv, torch.bfloat16)
    assert torch.equal(y.cpu(), torch.from_numpy(c.residual).to(torch.bfloat16))
    assert not c.run(sv, torch.float32, residual=False).any()


def test_all_tokens_at_one_expert(sv):
    say("one expert")
    for t, k in ((200, 1), (100, 5)):
        c = Case(t, 20, 1, 130, 200, seed=2)
        c.ids = np.full((t, k), 13, dtype=np.int32)
        c.weights = np.random.default_rng(1).random((t, k)).astype(np.float32)
        c.check(c.run(sv, torch.float32), torch.float32)


def test_most_pairs(sv):
    say("8192 pairs")
    for t, e, k in ((1024, 16, 8), (128, 64, 64), (8192, 5, 1)):
        c = Case(t, e, k, 64, 64, seed=4)
        c.check(c.run(sv, torch.float32), torch.float32)


def test_infinities_and_nan_stay_in_their_token(sv):
    say("inf, nan")
    c = Case(20, 6, 2, 200, 150, seed=5)
    c.xd[3], c.xd[7], c.weights[11, 1] = np.nan, np.inf, np.nan
    y = c.run(sv, torch.float32)
    c.check(y, torch.float32)
    bad = torch.isnan(y).all(dim=1).cpu()
    assert bad.nonzero().flatten().tolist() == [3, 7, 11] and torch.isfinite(y[~bad.cuda()]).all()
    c = Case(4, 3, 2, 200, 150, seed=6)
    c.layer["gated"][1, 5] = np.inf
    c.layer["upd"][2] = 0                          # blocks of zeros
    c.layer["downd"][0, 3] = np.nan
    c.check(c.run(sv, torch.float32), torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_strides_and_workspace(sv, dtype):
    say(f"in place {dtype}")
    c = Case(10, 6, 3, 200, 150, seed=7)
    wide = torch.full((10, 209), 3.0, dtype=dtype, device="cuda")
    wide[:, 4:204] = torch.from_numpy(c.residual).to(dtype).cuda()
    ex = c.experts(sv)
    ws = torch.full((sv.qr_moe_i8_workspace_bytes(ex, 10, 3),), 255, dtype=torch.uint8, device="cuda")
    y = sv.qr_moe_i8(dev(c.x), dev(c.xd), ex, dev(c.ids), dev(c.weights), residual=wide[:, 4:204], out=wide[:, 4:204],
                     workspace=ws)
    c.check(y, dtype)
    assert (wide[:, :4] == 3).all() and (wide[:, 204:] == 3).all()
    assert sv.qr_moe_i8(dev(c.x[:0]), dev(c.xd[:0]), ex, dev(c.ids[:0]), dev(c.weights[:0])).shape == (0, 200)


@pytest.mark.parametrize("t", [1, 6, 80])
def test_experts_graph_and_stream(sv, t):
    say(f"experts graph {t}")
    c = Case(t, 12, 3, 200, 300, seed=8)
    ex, x, xd, ids, wt = c.experts(sv), dev(c.x), dev(c.xd), dev(c.ids), dev(c.weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = sv.qr_moe_i8(x, xd, ex, ids, wt, dtype=torch.float32, stream=side)
    side.synchronize()
    c.check(y, torch.float32, residual=False)
    ws = torch.empty(sv.qr_moe_i8_workspace_bytes(ex, t, 3), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_moe_i8(x, xd, ex, ids, wt, out=y, workspace=ws)
    for seed in (1, 2, 3):
        n = Case(t, 12, 3, 200, 300, seed=seed)
        c.ids, c.x = n.ids, n.x
        ids.copy_(torch.from_numpy(c.ids)), x.copy_(torch.from_numpy(c.x))
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        c.check(y, torch.float32, residual=False)
        assert torch.equal(y, sv.qr_moe_i8(x, xd, ex, ids, wt, dtype=torch.float32))
