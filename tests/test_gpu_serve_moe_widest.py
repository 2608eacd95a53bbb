"""The router's widest choices on the GPU: 64 experts of each token, one per lane,
out of as many or some more, with equal scores and experts switched off."""
import numpy as np
import pytest

from test_gpu_serve_moe import check_route, dev, route_case
from test_gpu_serve_moe_many import equal_rows
from test_gpu_serve_moe_prompts import rows, say, sv  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,e", [(1, 64), (5, 64), (3, 65), (2, 128), (33, 192), (4, 256), (700, 64)])
def test_64_experts(sv, t, e):  # noqa: F811
    say(f"64 of {e}, {t} tokens")
    x, w, b = route_case(t, e, 130, e)
    b[[0, e // 2, e - 1]] = -np.inf
    for score, bias, renorm in (("softmax", None, True), ("sigmoid", b, True), ("softmax", b, False)):
        check_route(sv.qr_moe_route(x.cuda(), w.cuda(), 64, score=score, bias=dev(bias), renorm=renorm), x, w, 64, score, bias,
                    renorm, 1.0)
    w = w[torch.arange(e) % 9].contiguous()
    check_route(sv.qr_moe_route(x.cuda(), w.cuda(), 64), *equal_rows(x, w), 64, "softmax", None, True, 1.0)


@pytest.mark.parametrize("t,e,k,top_k", [(3000, 256, 1500, 27), (2000, 513, 1100, 64), (9000, 72, 1700, 1)])
def test_most_that_rough_logits_take(sv, t, e, k, top_k):  # noqa: F811
    """At most (n_experts - 65) / 7 of them."""
    say(f"{top_k} of {e}, {t} tokens")
    x, w, b = rows(t, e, k, e)
    for score, bias in (("softmax", None), ("sigmoid", b)):
        check_route(sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score=score, bias=dev(bias)), x, w, top_k, score, bias, True, 1.0)
