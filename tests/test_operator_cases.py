"""perf/operators.py on the CPU: its listed and drawn cases are well formed,
and the plain forms agree with the definitions in 64 bits on small cases."""
import random

import pytest
import torch

from perf import operators


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(operators, "_DEV", "cpu")
    monkeypatch.setattr(operators, "own", False)


def test_cases_are_well_formed():
    cases = operators.listed()
    assert 4 <= len(cases) <= 12 and len({c["name"] for c in cases}) == len(cases)
    rng = random.Random(1)
    drawn = [operators.draw(rng) for _ in range(200)]
    most = max(operators.work(c)["flops"] for c in cases)
    for c in drawn:
        assert "name" not in c and 0 < operators.work(c)["flops"] <= most
        if c["op"] != "linear":
            lens, new = operators._lengths(c)
            assert all(1 <= b <= a for a, b in zip(lens, new))


CASES = [
    operators._linear("a", 5, 30, 200),
    operators._linear("b", 3, 17, 130, "f32", True),
    operators._attention("c", 3, 100, 7, 4, 2, 64, 32, window=20, dtype="f32"),
    operators._attention("d", 2, 70, 1, 6, 2, 64, 32),
    operators._cache("e", 3, 100, 7, 2, 64, 32),
    operators._cache("f", 2, 70, 70, 1, 64, 32, dtype="f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c["name"])
def test_plain_forms_agree_with_the_definitions(case):
    # fp32: sums of up to 200 products; bf16 outputs: half a step of 2^-8
    state = operators.prepare(case, 3)
    exact = operators.exact(case, 3)
    exact = exact if isinstance(exact, tuple) else (exact,)
    for _ in range(2):   # a pass may be repeated on its state
        out = operators.run(state)
        out = out if isinstance(out, tuple) else (out,)
        for a, b in zip(out, exact):
            assert a.shape == b.shape
            tol = 2.0 ** -8 * b.abs() if a.dtype == torch.bfloat16 else 0.0
            assert bool(((a.double() - b).abs() <= tol + 1e-5 * b.abs().max()).all())
