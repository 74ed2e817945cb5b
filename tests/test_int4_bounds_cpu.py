"""The bounds of test_int4_bounds_gpu.py see what they are for: references with a planted loss
fall outside them, and the reference's own rounding falls inside."""
import numpy as np
import pytest
import torch

import rows_harness as rh
from int4_bounds import Case
from oracle import decode_ref, decode_ref_rows
from oracle import int4 as o4

SHAPES = [([512, 1000], 4, 2, 128), ([2500, 37], 8, 2, 128), ([500, 3000], 6, 1, 256)]


@pytest.mark.parametrize("rows,window", [(1, 0), (3, 0), (1, 100)])
def test_reference_is_the_oracle(rows, window):
    c = Case([300, 0, 1, 37], 4, 2, 128, 16, rows=rows, window=window, heavy=(0, -1), seed=1, v_scale=3.0)
    K, V = ([o4.dequant(c.rows_of(x, b)) * s if L else np.zeros((0, 2, 128)) for b, L in enumerate(c.lens)]
            for x, s in ((c.kc, c.k_scale), (c.vc, c.v_scale)))
    ref, _ = c.reference()
    want = decode_ref(rh.f64(c.q), K, V, c.scale, window=window)[:, None] if rows == 1 else \
        decode_ref_rows(rh.f64(c.q), K, V, c.scale)
    assert np.allclose(ref, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("heavy", [(), (0, 31, 32, -1)])
def test_a_lost_token_or_tile_is_seen(dtype, shape, heavy):
    c = Case(*shape, 16, dtype=dtype, heavy=heavy, seed=2)
    ref, tol = c.reference()
    rounded = torch.from_numpy(ref).to(rh.DT[dtype]).double().numpy()
    worst, norm = c.errors(rounded, ref, tol)
    assert worst <= 1 and norm <= 1
    tile = lambda b, L: np.arange(L)[(np.arange(L) // 32) == (L // 32) // 2]
    for kw in (dict(drop=tile), dict(zero_v=tile), dict(drop=lambda b, L: np.arange(L)[-32:]),
               dict(zero_v=lambda b, L: np.arange(L)[:32])):
        _, norm = c.errors(c.reference(**kw)[0], ref, tol)
        assert norm > 1, kw
    if heavy:   # any of the four, alone
        for t in heavy:
            lost = c.reference(drop=lambda b, L: [t])[0]
            worst, norm = c.errors(lost, ref, tol)
            assert norm > 20 and worst > 1, t


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_of_a_thousand_equal_tokens_is_seen(dtype):
    c = Case([512], 4, 2, 128, 16, dtype=dtype, seed=3)
    ref, tol = c.reference()
    assert c.errors(c.reference(drop=lambda b, L: [L - 1])[0], ref, tol)[1] > 1
