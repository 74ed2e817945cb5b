"""Randomised sweeps of append, gather and decode over 4-bit caches against the float64 oracle
(GB300 only). Each case draws one point of what the calls accept from a fixed seed, so a
failing one is reproduced by its index."""
import os
import random

import numpy as np
import pytest
import torch

import rows_harness as rh
from test_int4_gpu import run_case
from test_rows_gpu import append, check_append, i32, make, rope_of, SCALES, views

# 60 of each by default; PA_RANDOM_ROWS runs more draws of the same seeded generators
N_CASES = int(os.environ.get("PA_RANDOM_ROWS", "60"))
BLOCKS = [1, 2, 7, 16, 31, 32, 33, 48, 100, 784, 1024]


def draw_lengths(r, B, most):
    kinds = [0, 1, r.randint(1, 40), r.randint(1, most), r.randint(1, most), r.randint(1, most)]
    return [r.choice(kinds) for _ in range(B)]


def draw_decode(idx):
    r = random.Random(777 + idx)
    D = r.choice([128, 256])
    rows = r.choice([1, 1, 1, 2, 3, 4])
    G = r.choice([g for g in (1, 2, 3, 4, 6, 8, 12, 16) if g * rows <= (32 if D == 128 else 16)])
    Hkv = r.choice([1, 2, 3, 8])
    B = r.randint(1, 6)
    return dict(D=D, rows=rows, Hq=G * Hkv, Hkv=Hkv, bs=r.choice(BLOCKS), lens=draw_lengths(r, B, 2500),
                window=r.choice([0, 0, 1, 40, 512]) if rows == 1 else 0, splits=r.choice([0, 0, 1, 2, 4, 11]),
                deterministic=r.random() < 0.4, dtype=r.choice(["bf16", "f16"]),
                step=r.choice([0.05, 0.3, 2.0]), k_scale=r.choice([1.0, 0.25]), v_scale=r.choice([1.0, 3.0]))


@pytest.mark.gpu
@pytest.mark.parametrize("idx", range(N_CASES))
def test_random_decode_int4(cuda_lib, idx):
    c = draw_decode(idx)
    kw = {k: c[k] for k in ("splits", "deterministic", "window", "k_scale", "v_scale", "step", "dtype", "rows")}
    run_case(cuda_lib, c["lens"], c["Hq"], c["Hkv"], c["D"], c["bs"], seed=idx,
             scale=0.3 / (c["step"] * c["k_scale"] * c["D"] ** 0.5), **kw)


def draw_rows(idx):
    r = random.Random(4242 + idx)
    D = r.choice([128, 256])
    Hkv, G = r.choice([1, 2, 3, 4, 8]), r.choice([1, 2, 3, 5, 8])
    B = r.randint(1, 9) if r.random() < 0.8 else r.randint(32, 100)
    lens = draw_lengths(r, B, 300)
    packed = r.random() < 0.5
    return dict(lens=lens, new=[r.randint(0, L + (r.random() < 0.2)) for L in lens] if packed else None,
                R=0 if packed else r.randint(1, 9), Hq=G * Hkv, Hkv=Hkv, D=D, bs=r.choice(BLOCKS),
                dtype=r.choice(["bf16", "f16"]), cache=r.choice(["same", "fp8", "int4", "int4"]),
                pad=(r.choice([0, 0, 3]), r.choice([0, 0, 7])), rot=16 * r.randint(0, D // 16),
                il=r.random() < 0.5, with_q=r.random() < 0.8,
                scaling=r.choice([{}, dict(kind="linear", factor=3.0), dict(kind="ntk", factor=2.0),
                                  dict(kind="yarn", factor=4.0, original_max=128),
                                  dict(kind="banded", factor=4.0, original_max=256, slow=1.0, fast=4.0)]))


@pytest.mark.gpu
@pytest.mark.parametrize("idx", range(N_CASES))
def test_random_append_and_gather(cuda_lib, idx):
    c = draw_rows(idx)
    x = make(c["lens"], c["new"], c["R"], c["Hq"], c["Hkv"], c["D"], c["bs"], c["dtype"], c["cache"],
             seed=idx, pad=c["pad"] if c["new"] is not None else (0, 0))
    if x["T"] == 0:
        return
    kw = c["scaling"] if c["rot"] > 16 else {}
    rope, f, amp = rope_of(cuda_lib, c["rot"], c["il"], **kw)
    qo, kc, vc = append(cuda_lib, x, rope, with_q=c["with_q"])
    check_append(x, f, amp, c["il"], qo, kc, vc)
    # the rows read back are the cache's values, once rounded
    ks, vs = SCALES[c["cache"]]
    rows = x["T"] if c["new"] is not None else c["R"]
    shape = (rows, c["Hkv"], c["D"]) if c["new"] is not None else (x["B"], rows, c["Hkv"], c["D"])
    outs = [torch.full(shape, 9.0, dtype=rh.DT[c["dtype"]], device="cuda") for _ in range(2)]
    cuda_lib.gather(kc, vc, x["bt"].cuda(), i32(x["lens"]), rows, starts=i32(x["starts"]),
                    dtype=rh.DT[c["dtype"]], k_out=outs[0], v_out=outs[1], k_scale=ks, v_scale=vs)
    for got, cache, s in ((outs[0], kc, ks), (outs[1], vc, vs)):
        want = torch.full((x["T"], c["Hkv"], c["D"]), 9.0, dtype=rh.DT[c["dtype"]])
        for r, b, p in rh.positions(x["lens"], x["starts"], c["R"], x["B"]):
            if p < 0:
                want[r] = 0
                continue
            raw = rh.cache_rows(cache, c["cache"], x["bt"], b, np.array([p]), c["bs"])
            want[r] = raw[0] if c["cache"] == "same" else \
                (torch.from_numpy(rh.values(raw, c["cache"])[0]).float() *
                 torch.tensor(s, dtype=torch.float32)).to(want.dtype)
        assert torch.equal(rh.bits(got.cpu().reshape(want.shape)), rh.bits(want))
    assert cuda_lib.read_device_errors(cuda_lib.default_workspace()) == 0


def test_draws_cover_the_space():
    d = [draw_decode(i) for i in range(N_CASES)]
    assert {c["D"] for c in d} == {128, 256} and any(c["rows"] > 1 for c in d) and any(c["window"] for c in d)
    assert any(0 in c["lens"] for c in d) and len({c["bs"] for c in d}) >= 6
    a = [draw_rows(i) for i in range(N_CASES)]
    assert {c["cache"] for c in a} == {"same", "fp8", "int4"} and any(c["new"] is None for c in a)
    assert any(c["rot"] == 0 for c in a) and any(c["rot"] % 64 for c in a) and any(len(c["lens"]) >= 32 for c in a)
