"""The router of many tokens on the GPU, where its logits come from fp32 sums
first and the choice is settled with exact ones: the choice equal to the one of
64-bit logits throughout, the weights as near, whatever the rows hold."""
import numpy as np
import pytest

from test_gpu_serve_moe import check_route, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def say(*a):
    print(*a, flush=True)


def rows(t, e, k, seed, loud=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((t, k)).astype(np.float32)
    if loud:
        x[:, rng.random(k) < 0.01] *= 12
    x, w = torch.from_numpy(x).to(BF16), torch.from_numpy((rng.standard_normal((e, k)) * 1.5 / np.sqrt(k)).astype(np.float32)).to(BF16)
    assert t * e * k > 2 ** 30
    return x, w, (0.1 * rng.standard_normal(e)).astype(np.float32)


@pytest.mark.parametrize("t,e,k,top_k", [(2100, 256, 2048, 8), (2049, 257, 2049, 8), (1300, 1000, 1000, 4), (12000, 120, 1100, 1),
                                         (700, 512, 3001, 16), (40000, 300, 100, 3), (5000, 1024, 300, 64), (90000, 200, 63, 5)])
def test_choice_and_weights(sv, t, e, k, top_k):
    x, w, b = rows(t, e, k, e)
    for score, bias, factor in (("softmax", None, 1.0), ("sigmoid", b, 2.5), ("sigmoid", None, 1.0)):
        say(f"route {t}x{e}x{k} top {top_k} {score} bias={bias is not None}")
        got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(bias), factor=factor)
        check_route(got, x, w, top_k, score, bias, True, factor)
    got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score="sigmoid", renorm=False)
    check_route(got, x, w, top_k, "sigmoid", None, False, 1.0)


def test_experts_that_fp32_sums_do_not_tell_apart(sv):
    """Rows of the router that differ in the last place of one small value, and
    equal ones: ties go to the lowest index."""
    say("near ties")
    t, e, k = 3000, 240, 1500
    x, w, b = rows(t, e, k, 1)
    w = w[torch.arange(e) % 12].contiguous()
    bits = w.view(torch.int16)
    for i in range(24, e):
        bits[i, (37 * i) % k] += 1
    for score, bias in (("softmax", None), ("sigmoid", b), ("sigmoid", None)):
        if bias is not None:
            bias = np.repeat(bias[:12], 20)
        got = sv.qr_moe_route(x.cuda(), w.cuda(), 6, score=score, bias=dev(bias))
        check_route(got, x, w, 6, score, bias, True, 1.0)


def test_rows_of_every_kind(sv):
    """Zeros (a padded token), one value, subnormal values, values whose products
    leave fp32, infinities and NaN, far apart logits, all in one call."""
    say("kinds")
    t, e, k = 2500, 256, 1700
    x, w, b = rows(t, e, k, 2)
    x[::7] = 0
    x[1, 1:] = 0
    x[2] = (x[2].float() * 1e-39).to(BF16)
    x[3] = (x[3].float() * 1e36).to(BF16)
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6] = x[6] * 300
    x[8] = 1.0
    x[9] = (x[9].float() * 1e-30).to(BF16)
    for score, bias in (("softmax", None), ("sigmoid", b), ("sigmoid", None)):
        got = sv.qr_moe_route(x.cuda(), w.cuda(), 8, score=score, bias=dev(bias))
        check_route(got, x, w, 8, score, bias, True, 1.0)
    big = (w.float() * 1e30).to(BF16)
    got = sv.qr_moe_route(x.cuda(), big.cuda(), 8, score="sigmoid")
    check_route(got, x, big, 8, "sigmoid", None, True, 1.0)
    zero = torch.zeros_like(w)
    got = sv.qr_moe_route(x.cuda(), zero.cuda(), 3)
    check_route(got, x, zero, 3, "softmax", None, True, 1.0)


def test_scores_that_round_together(sv):
    """Sigmoids that all round to one, and biases that leave nothing of a score:
    the lowest indices, as far as the 64-bit scores are equal."""
    say("saturated")
    t, e, k = 2300, 240, 2000
    x, w, b = rows(t, e, k, 9, loud=False)
    x[:, 0], w[:, 0] = 8.0, 100.0           # (every logit near 800)
    ids, wt = sv.qr_moe_route(x.cuda(), w.cuda(), 8, score="sigmoid")
    assert (ids.cpu().numpy() == np.arange(8)).all() and (wt.cpu().numpy() == 0.125).all()
    x, w, b = rows(t, e, k, 10)
    bias = np.where(np.arange(e) % 3 == 1, 2.0 ** 60, 0).astype(np.float32)
    ids, wt = sv.qr_moe_route(x.cuda(), w.cuda(), 8, score="sigmoid", bias=dev(bias))
    assert (ids.cpu().numpy() == 3 * np.arange(8) + 1).all()
    w = w * 0.0
    w[100:, 0], x[:, 0] = -100.0, 16.0      # (all but a hundred scores are zero)
    got = sv.qr_moe_route(x.cuda(), w.cuda(), 8)
    assert (got[0].cpu().numpy() == np.arange(8)).all()
    w[3:100, 0] = -100.0
    got = sv.qr_moe_route(x.cuda(), w.cuda(), 8)
    assert (got[0].cpu().numpy() == np.arange(8)).all()
    assert (got[1].cpu().numpy()[:, 3:] == 0).all()


def test_experts_switched_off(sv):
    say("off")
    t, e, k = 3000, 240, 1600
    x, w, b = rows(t, e, k, 3)
    b[np.random.default_rng(1).random(e) < 0.985] = -np.inf
    assert 0 < np.isfinite(b).sum() < 8
    got = sv.qr_moe_route(x.cuda(), w.cuda(), 8, score="sigmoid", bias=dev(b))
    check_route(got, x, w, 8, "sigmoid", b, True, 1.0)
    assert (got[0] == -1).any()


def test_strided_rows(sv):
    say("strided")
    t, e, k = 2300, 250, 2000
    x, w, _ = rows(t, e, k + 37, 4)
    w = w[:, :k].contiguous()
    for first in (0, 1, 37):
        got = sv.qr_moe_route(x.cuda()[:, first:first + k], w.cuda(), 5)
        check_route(got, x[:, first:first + k], w, 5, "softmax", None, True, 1.0)


def test_graph(sv):
    say("graph")
    t, e, k = 2200, 256, 2048
    x, w, b = rows(t, e, k, 5)
    gx, gw, gb = x.cuda(), w.cuda(), dev(b)
    ws = torch.empty(sv.qr_moe_route_workspace_bytes(e, t, k), dtype=torch.uint8, device="cuda")
    out = sv.qr_moe_route(gx, gw, 4, score="sigmoid", bias=gb, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.qr_moe_route(gx, gw, 4, score="sigmoid", bias=gb, ids=out[0], weights=out[1], workspace=ws)
    for seed in (6, 7, 8):
        nx = rows(t, e, k, seed)[0]
        gx.copy_(nx)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        check_route(out, nx, w, 4, "sigmoid", b, True, 1.0)
