"""Randomised sweep of cross attention and decode behind shared prefixes against their definitions in 64
bits (GB300 only). Each case draws one point of what the calls accept from a fixed seed, so that a failing
one is reproduced by its index."""
import os
import random

import pytest

import attend_harness as ah
from test_cross_gpu import run as run_cross
from test_decode_shared_gpu import run as run_shared

# 60 of each by default; PA_RANDOM_ATTEND runs more draws of the same seeded generators
N_CASES = int(os.environ.get("PA_RANDOM_ATTEND", "60"))
BLOCKS = [1, 7, 8, 16, 24, 33, 40, 64, 128, 784]


def common(r):
    D = r.choice([128, 256])
    B = r.choice([1, 2, 3, 7, 16])
    return dict(D=D, G=r.randint(1, 16), Hkv=r.choice([1, 2, 3, 4, 8]), bs=r.choice(BLOCKS), B=B,
                dtype=r.choice(["bf16", "f16"]), cache=r.choice(["same", "same", "fp8"]), spread=r.choice([1.0, 1.0, 4.0]),
                most=r.choice([5, 60, 300, 1500, 4000]) // max(1, B // 4))


def draw_cross(idx):
    r = random.Random(31337 + idx)
    c = common(r)
    rows = max(1, 1500 // (c["B"] * c["G"] * c["Hkv"]))    # bounds the 64-bit work
    if r.random() < 0.4:
        counts = [r.choice([0, 1, 3, r.randint(1, 2 * rows)]) for _ in range(c["B"])]
        if not sum(counts):
            counts[-1] = 2
        pad = (r.randint(0, 3), r.randint(0, 3))
    else:
        counts, pad = [r.choice([1, 2, 5, rows])] * c["B"], None
    return dict(c, lens=[r.randint(0, c["most"]) for _ in range(c["B"])], counts=counts, pad=pad)


def draw_shared(idx):
    r = random.Random(27182 + idx)
    c = common(r)
    cuts = sorted(r.randint(0, c["B"]) for _ in range(r.randint(1, min(c["B"], 4)) + 1))
    lens, prefix = [r.randint(0, c["most"]) for _ in range(c["B"])], []
    for a, e in zip(cuts, cuts[1:]):
        P = r.randint(0, c["most"])
        for b in range(a, e):
            lens[b] = P + r.randint(0, max(1, c["most"] // 4))
        prefix.append(P if e > a else 0)
    rows = max(1, 1500 // (c["B"] * c["G"] * c["Hkv"]))
    return dict(c, lens=lens, groups=cuts, prefix=prefix, R=r.choice([1, 1, 2, 4, 9, rows]), own=r.random() < 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("idx", range(N_CASES))
def test_random_cross(cuda_lib, idx):
    c = draw_cross(idx)
    pool = ah.Pool(c["lens"], c["Hkv"], c["D"], c["bs"], c["dtype"], c["cache"], seed=idx, spread=c["spread"])
    Hq = c["G"] * c["Hkv"]
    if c["pad"] is None:
        run_cross(cuda_lib, pool, ah.queries((c["B"], c["counts"][0], Hq, c["D"]), c["dtype"], idx), c["counts"])
        return
    starts = [c["pad"][0]]
    for n in c["counts"]:
        starts.append(starts[-1] + n)
    q = ah.queries((starts[-1] + c["pad"][1], Hq, c["D"]), c["dtype"], idx)
    run_cross(cuda_lib, pool, q, c["counts"], starts)


@pytest.mark.gpu
@pytest.mark.parametrize("idx", range(N_CASES))
def test_random_decode_shared(cuda_lib, idx):
    c = draw_shared(idx)
    spans = [(a, e, P) for a, e, P in zip(c["groups"], c["groups"][1:], c["prefix"]) if e > a]
    pool = ah.Pool(c["lens"], c["Hkv"], c["D"], c["bs"], c["dtype"], c["cache"], seed=idx, prefixes=spans,
                   own_prefix=c["own"], spread=c["spread"])
    q = ah.queries((c["B"], c["R"], c["G"] * c["Hkv"], c["D"]), c["dtype"], idx)
    run_shared(cuda_lib, pool, q, c["groups"], c["prefix"], max_seq_len=pool.bt.shape[1] * c["bs"])


def test_draws_cover_the_space():
    cross, shared = ([f(i) for i in range(60)] for f in (draw_cross, draw_shared))
    for cases in (cross, shared):
        assert {c["D"] for c in cases} == {128, 256} and {c["cache"] for c in cases} == {"same", "fp8"}
        assert len({c["bs"] for c in cases}) >= 8 and len({c["G"] for c in cases}) >= 12
        assert any(max(c["lens"]) > 3000 for c in cases)
    assert any(c["pad"] for c in cross) and any(c["pad"] is None for c in cross)
    assert any(c["counts"][0] * c["G"] > 256 for c in cross)
    assert any(c["R"] * c["G"] > 128 for c in shared) and any(c["R"] == 1 for c in shared)
    assert any(len(c["groups"]) > 3 for c in shared) and {c["own"] for c in shared} == {True, False}
