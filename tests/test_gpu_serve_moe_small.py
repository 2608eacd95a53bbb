"""The router of few experts on the GPU, whose call is one launch: against the
definition, on both sides of the sizes where it takes over."""
import numpy as np
import pytest

from test_gpu_serve_moe import check_route, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


def rows(t, e, k, xt, wt, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32)).to(xt)
    w = torch.from_numpy((rng.standard_normal((e, k)) / np.sqrt(k)).astype(np.float32)).to(wt)
    return x, w, (0.1 * rng.standard_normal(e)).astype(np.float32)


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("t,e,k,top_k", [(1, 1, 1, 1), (2, 2, 7, 2), (3, 8, 511, 2), (256, 8, 512, 8), (257, 8, 513, 1), (5, 9, 1030, 3),
                                         (7, 16, 4096, 4), (7, 16, 4097, 4), (4, 17, 300, 17), (30, 15, 2000, 15), (1, 1, 65536, 1),
                                         (2, 1, 65537, 1), (3, 8, 8192, 2)])
def test_few_experts(sv, t, e, k, top_k, xt, wt):
    x, w, b = rows(t, e, k, xt, wt, t + e + k)
    for score, bias, renorm, factor in (("softmax", None, True, 1.0), ("softmax", None, False, 2.0), ("sigmoid", b, True, 2.5),
                                        ("softmax", b, False, 1.0), ("sigmoid", None, False, 1.0)):
        say(f"route {t}x{e}x{k} top {top_k} {xt} {wt} {score}")
        got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(bias), renorm=renorm, factor=factor)
        check_route(got, x, w, top_k, score, bias, renorm, factor)


def test_ties_and_rows_of_every_kind(sv):
    say("kinds")
    x, w, b = rows(9, 12, 700, torch.bfloat16, torch.bfloat16, 3)
    w = w[torch.arange(12) % 3].contiguous()
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 6] = float("nan")
    x[4] = (x[4].float() * 1e-39).to(torch.bfloat16)
    x[5] = (x[5].float() * 1e36).to(torch.bfloat16)
    off = np.where(np.arange(12) % 5 == 0, -np.inf, np.repeat(b[:3], 4)).astype(np.float32)
    for score, bias in (("softmax", None), ("sigmoid", None), ("sigmoid", off)):
        got = sv.qr_moe_route(x.cuda(), w.cuda(), 12, score=score, bias=dev(bias))
        check_route(got, x, w, 12, score, bias, True, 1.0)
    ids = sv.qr_moe_route(x.cuda()[:1], w.cuda(), 12)[0].cpu().numpy()[0].reshape(3, 4)
    assert (np.diff(ids, axis=1) == 3).all()      # (equal rows: the lowest index first)


def test_strided_rows_and_a_graph(sv):
    say("graph")
    x, w, b = rows(20, 8, 1024, torch.bfloat16, torch.bfloat16, 4)
    wide = torch.zeros((20, 1100), dtype=torch.bfloat16, device="cuda")
    gx, gw = wide[:, 37:37 + 1024], w.cuda()
    gx.copy_(x)
    out = sv.qr_moe_route(gx, gw, 2)
    check_route(out, x, w, 2, "softmax", None, True, 1.0)
    ws = torch.empty(sv.qr_moe_route_workspace_bytes(8, 20, 1024), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_moe_route(gx, gw, 2, ids=out[0], weights=out[1], workspace=ws)
    for seed in (5, 6, 7):
        nx = rows(20, 8, 1024, torch.bfloat16, torch.bfloat16, seed)[0]
        gx.copy_(nx)
        g.replay()
        torch.cuda.synchronize()
        check_route(out, nx, w, 2, "softmax", None, True, 1.0)
