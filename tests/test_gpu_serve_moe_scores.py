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
