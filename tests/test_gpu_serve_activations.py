"""The activations of the 8-bit product's epilogue on the GPU, relative to their
results: what is left of SiLU and GELU at negative arguments keeps its bits.

Derived with u = 2^-24 (half a step of fp32), for results of 2^-110 and more:

SiLU, x / d with d = 1 + exp(-x): exp2 is good to a step (2u), the bits that
-x log2(e) loses are carried on by one fma (u), d is rounded once (u), and the
quotient, mended by one step, once (u, and 9 u^2 of the reciprocal's step and
the first quotient's rounding): 5u, and less than 1u for what is left out. 8u.

GELU_TANH, x / (1 + exp(t)), t = x (A - B x^2): the rounded constants count u
each, the three products u each, the sum u; both terms have one sign, so t is off
by 5u of its size, which the quotient passes on in full at most (and by less
than 2u at negative t): (8 + 5 |t|) u.

GELU, x / 2 * erfc(z), z = -x / sqrt(2): constant and product leave z off by 2u,
of which erfc passes on |z| 2/sqrt(pi) exp(-z^2) / erfc(z) <= 2 z^2 + 1 = x^2 + 1;
erfc itself is good to 16 steps (32u, what OpenCL asks of it), and one rounding:
(36 + 2 x^2) u."""
import numpy as np
import pytest

import serve_layer_plain as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LEAST = 2.0 ** -110


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_row_amd import serve
    serve.load_library()
    return serve


def bound(act, x):
    if act == "silu":
        return np.full_like(x, 8 * U)
    if act == "gelu":
        return (36 + 2 * x * x) * U
    return (8 + 5 * np.abs(2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))) * U


def definition(act, x):
    """In 64 bits, also where one over a sum that has lost its bits is no good."""
    if act != "gelu":
        return plain.act(act, x)
    return x * 0.5 * plain.erfc(-x / np.sqrt(2.0))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t", [16, 60, 30000])
def test_relative_to_the_result(sv, act, t):
    """One channel of code 1 and scale 1: the token's scale is the argument, and
    no product rounds it."""
    print(f"{act} {t}", flush=True)
    rng = np.random.default_rng(t)
    low = {"silu": -80.0, "gelu": -12.5, "gelu_tanh": -8.0}[act]
    x = np.concatenate([rng.uniform(low, 0, t), rng.uniform(-1, 1, t // 2), rng.uniform(0, 90, t // 4),
                        np.exp(rng.uniform(-70, 0, t)) * rng.choice([-1, 1], t)]).astype(np.float32)
    x = rng.permutation(x)[:t]
    codes = np.zeros((t, 128), dtype=np.int8)
    codes[:, 0] = 1
    dev = lambda a: torch.from_numpy(a).cuda()
    y = sv.qr_matmul_i8_ex(dev(codes[:1].repeat(3, axis=0)), torch.ones(3, device="cuda"), dev(codes), dev(x), 1, act=act,
                           dtype=torch.float32)
    x = x.astype(np.float64)
    with np.errstate(over="ignore"):
        want = definition(act, x)
    got = y.cpu().numpy().astype(np.float64)
    counts = np.abs(want) >= LEAST
    assert counts.sum() > t // 2 and (want[counts] < 0).any()
    off = np.abs(got - want[:, None])[counts] / np.abs(want[counts])[:, None] / bound(act, x[counts])[:, None]
    print(f"  at most {off.max():.3f} of the bound", flush=True)
    assert off.max() <= 1
