"""perf/more_operators.py on the CPU: its listed and drawn cases are well
formed, and the plain forms agree with the definitions in 64 bits on small
cases."""
import random

import pytest
import torch

from perf import more_operators as operators


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(operators, "_DEV", "cpu")
    monkeypatch.setattr(operators, "own", False)


def test_cases_are_well_formed():
    cases = operators.listed()
    assert 4 <= len(cases) <= 12 and len({c["name"] for c in cases}) == len(cases)
    rng = random.Random(1)
    drawn = [operators.draw(rng) for _ in range(300)]
    most = max(operators.work(c)["flops"] for c in cases)
    for c in drawn:
        assert "name" not in c and 0 < operators.work(c)["flops"] <= most and operators.work(c)["bytes"] > 0
    assert {c["op"] for c in drawn} == {c["op"] for c in cases} == {"norm", "product", "route", "experts"}


CASES = [
    operators._norm("a", 5, 300, y=True),
    operators._norm("b", 3, 130, "f32", False, True),
    operators._product("c", 5, 30, 200, act="silu", up=True, bias=True, residual=True),
    operators._product("d", 4, 33, 130, "f32", act="gelu"),
    operators._product("e", 3, 20, 100, "f32", act="gelu_tanh", up=True),
    operators._product("f", 3, 20, 100, act="relu", residual=True),
    operators._route("g", 7, 20, 100, 4),
    operators._route("h", 6, 33, 70, 5, "f32", "sigmoid", True, False),
    operators._experts("i", 5, 6, 2, 200, 70),
    operators._experts("j", 9, 4, 4, 130, 200, "f32", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c["name"])
def test_plain_forms_agree_with_the_definitions(case):
    # fp32: sums of up to 200 products; bf16 outputs: half a step of 2^-8
    state = operators.prepare(case, 3)
    many = lambda v: list(v) if isinstance(v, (list, tuple)) else [v]
    exact = many(operators.exact(case, 3))
    for _ in range(2):   # a pass may be repeated on its state
        out = many(operators.run(state))
        assert len(out) == len(exact)
        for a, b in zip(out, exact):
            assert a.shape == b.shape
            if not a.dtype.is_floating_point:
                assert torch.equal(a, b)
                continue
            tol = 2.0 ** -8 * b.abs() if a.dtype == torch.bfloat16 else 0.0
            assert bool(((a.double() - b).abs() <= tol + 1e-5 * b.abs().max()).all())
