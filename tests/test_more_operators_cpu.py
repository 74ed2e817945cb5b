"""The plain forms of perf/more_operators.py against its definitions in 64 bits, on small cases (CPU), and
the cases that it draws."""
import random

import pytest
import torch

from perf import more_operators as ops

HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
BASE = dict(dtype="bf16", cache="same", B=3, Hq=4, Hkv=2, D=128, bs=16, rows=1, packed=0, groups=0, plo=0, phi=0, lo=1, hi=70)
CASES = [dict(op="cross"), dict(op="cross", rows=5, dtype="f16", bs=33, lo=40), dict(op="cross", packed=11, D=256, cache="fp8"),
         dict(op="shared", groups=1, plo=30, phi=30), dict(op="shared", groups=2, B=7, plo=5, phi=60, rows=3, lo=3, dtype="f16"),
         dict(op="shared", groups=1, B=2, plo=33, phi=33, D=256, cache="fp8", bs=7)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the forms run on the GPU where there is one")
@pytest.mark.parametrize("case", CASES)
def test_plain_forms(case):
    case = dict(BASE, **case)
    assert not ops.own
    state = ops.prepare(case, 5)
    got, want = ops.run(state).double(), ops.exact(case, 5)
    assert got.shape == want.shape == state["q"].shape
    # The output's rounding; sums of up to 130 weighted values below 6 and scores below 10 with terms of up
    # to 200, each product and sum off by 2^-24 of it: 2^-24 (2 * 130 * 6 + 2 * 200 * 6) < 2^-11
    assert torch.all((got - want).abs() <= HALF_STEP[case["dtype"]] * want.abs() + 2.0 ** -11)
    again = ops.prepare(case, 5)
    assert all(torch.equal(state[k].view(torch.uint8), again[k].view(torch.uint8)) for k in ("q", "k_cache", "v_cache"))
    assert not torch.equal(ops.prepare(case, 6)["q"], state["q"])


def test_drawn_cases_stay_within_the_listed():
    most = max(ops.work(c)["flops"] for c in ops.listed())
    rng = random.Random(1)
    cases = [ops.draw(rng) for _ in range(60)]
    assert all(ops.work(c)["flops"] <= most for c in cases)
    assert {c["op"] for c in cases} == {"cross", "shared"} and {c["cache"] for c in cases} == {"same", "fp8"}
    assert len({(c["D"], c["bs"]) for c in cases}) == 5
