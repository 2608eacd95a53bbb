"""The router of many tokens on the GPU where scores are of no size, or are no
numbers: its choice and weights stay those of 64-bit logits throughout."""
import numpy as np
import pytest

from test_gpu_serve_moe import check_route, dev
from test_gpu_serve_moe_prompts import rows, say, sv  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [-100.0, -88.5, -87.5])
def test_sigmoids_that_vanish(sv, first):  # noqa: F811
    """Logits around -800, -708 and -700: below -709.8 exp(-logit) leaves 64 bits
    and a score is zero, so that the lowest indices come first."""
    say(f"vanishing sigmoids {8 * first}")
    t, e, k = 2300, 240, 2000
    x, w, _ = rows(t, e, k, 11, loud=False)
    x[:, 0], w[:, 0] = 8.0, first
    for some in (False, True):
        if some:                                # (three experts have scores that count)
            w[[50, 120, 200], 0] = 0.0
        for renorm in (False, True):
            got = sv.qr_moe_route(x.cuda(), w.cuda(), 8, score="sigmoid", renorm=renorm)
            check_route(got, x, w, 8, "sigmoid", None, renorm, 1.0)
            if first == -100.0:
                assert (got[0].cpu().numpy()[:, 3 * some:] == np.arange(8 - 3 * some)).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("top_k", [1, 8])
def test_zeros_against_a_row_of_no_numbers(sv, top_k, value):  # noqa: F811
    """One expert is left to choose from, and zero times its infinite weight is no
    number: a token of zeros has that weight too."""
    say(f"zeros and {value}, top {top_k}")
    t, e, k = 3000, 240, 1600
    x, w, b = rows(t, e, k, 12)
    x[::2] = 0
    w[17:19, 5] = value
    b[:] = -np.inf
    b[17] = 0.25
    got = sv.qr_moe_route(x.cuda(), w.cuda(), top_k, score="sigmoid", bias=dev(b))
    check_route(got, x, w, top_k, "sigmoid", b, True, 1.0)
    assert (got[0][:, 0] == 17).all() and (got[0][:, 1:] == -1).all() and torch.isnan(got[1][::2, 0]).all()
