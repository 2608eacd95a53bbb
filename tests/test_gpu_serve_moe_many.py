"""The router's choice among more than 256 experts on the GPU, in 64 bits
throughout and from fp32 sums: equal scores go to the lowest index, experts that
are switched off are never chosen."""
import numpy as np
import pytest

from test_gpu_serve_moe import check_route, dev, route_case
from test_gpu_serve_moe_prompts import rows, say, sv  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
KINDS = [("softmax", False), ("sigmoid", True), ("sigmoid", False)]


def equal_rows(x, w):
    """x and w of the same logits for check_route, with one sum for rows of w that
    are equal: a library's product may round columns at the end of a block
    otherwise, and no two of them are equal in the oracle then."""
    some, index = np.unique(w.double().numpy(), axis=0, return_inverse=True)
    logits = x.double().numpy() @ some.T
    return torch.from_numpy(logits[:, index.ravel()]), torch.eye(w.shape[0], dtype=torch.float64)


def off(bias, on, seed):
    """A bias that leaves `on` of the experts, the first and the last among them."""
    keep = np.concatenate([[0, len(bias) - 1], 1 + np.random.default_rng(seed).permutation(len(bias) - 2)[:on - 2]])
    out = np.full_like(bias, -np.inf)
    out[keep] = bias[keep]
    return out


@pytest.mark.parametrize("t,e,top_k", [(1, 300, 12), (30, 512, 64), (7, 513, 9), (40, 1024, 33), (3, 1000, 64)])
def test_ties(sv, t, e, top_k):  # noqa: F811
    say(f"ties {t} tokens, {top_k} of {e}")
    for xt in (torch.float32, BF16):
        x, w, b = route_case(t, e, 90, e, xt, xt)
        w = w[torch.arange(e) % 37].contiguous()
        b = np.repeat(b[:37], -(-e // 37))[:e]
        for score, bias in KINDS + [("softmax", True)]:
            bias = b if bias else None
            check_route(sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(bias)), *equal_rows(x, w), top_k, score,
                        bias, True, 1.0)
        zero = torch.zeros_like(x).cuda()
        ids = sv.qr_moe_route(zero, w.cuda(), top_k)[0]
        assert (ids.cpu() == torch.arange(top_k)).all()


@pytest.mark.parametrize("t,e,top_k,on", [(1, 300, 8, 5), (30, 512, 64, 64), (7, 513, 9, 2), (40, 1024, 33, 20)])
def test_switched_off(sv, t, e, top_k, on):  # noqa: F811
    say(f"off {t} tokens, {top_k} of {e}, {on} on")
    x, w, b = route_case(t, e, 90, e)
    b = off(b, on, 1)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(b), renorm=renorm)
            check_route(got, x, w, top_k, score, b, renorm, 1.0)
            assert (got[0][:, on:] == -1).all() and (got[0][:, :min(on, top_k)] >= 0).all()
    b[:] = -np.inf
    assert (sv.qr_moe_route(x.cuda(), w.cuda(), top_k, bias=dev(b))[0] == -1).all()


# rough logits are taken from more than 64 + 7 top_k experts and 2^30 products on
MANY = [(2300, 300, 1600, 8), (1400, 520, 1500, 12), (1100, 1024, 1000, 40)]


@pytest.mark.parametrize("t,e,k,top_k", MANY)
def test_ties_of_many_tokens(sv, t, e, k, top_k):  # noqa: F811
    say(f"ties {t} tokens, {top_k} of {e}")
    x, w, b = rows(t, e, k, e)
    w = w[torch.arange(e) % 37].contiguous()
    bits = w.view(torch.int16)
    for i in range(e // 2, e):                  # half of them off by the last place of one value
        bits[i, (37 * i) % k] += 1
    x[::9] = 0
    b = np.repeat(b[:37], -(-e // 37))[:e]
    for score, bias in KINDS:
        bias = b if bias else None
        check_route(sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(bias)), *equal_rows(x, w), top_k, score, bias,
                    True, 1.0)


@pytest.mark.parametrize("t,e,k,top_k", MANY)
def test_switched_off_for_many_tokens(sv, t, e, k, top_k):  # noqa: F811
    x, w, b = rows(t, e, k, e + 1)
    for on in (top_k - 3, top_k, top_k + 1):
        say(f"off {t} tokens, {top_k} of {e}, {on} on")
        c = off(b, on, on)
        got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score="sigmoid", bias=dev(c))
        check_route(got, x, w, top_k, "sigmoid", c, True, 1.0)
        assert (got[0][:, on:] == -1).all()
