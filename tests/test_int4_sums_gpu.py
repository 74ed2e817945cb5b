"""Decode over 4-bit caches: the sums themselves, held to bounds that follow each element's own
terms (GB300 only)."""
import numpy as np
import pytest
import torch

import rows_harness as rh
from oracle import int4 as o4

pytestmark = pytest.mark.gpu


def pool_of(codes, st, mn, bs):
    """(cache, block table) of one sequence's rows, codes [L, Hkv, G, 32]."""
    L, Hkv, G = codes.shape[:3]
    nb = -(-L // bs)
    rows = torch.from_numpy(o4.pack(codes, st, mn))
    cache = torch.zeros((nb * bs, Hkv, o4.row_bytes(32 * G)), dtype=torch.uint8)
    cache[:L] = rows
    cache = cache.view(nb, bs, Hkv, -1).transpose(1, 2).contiguous()
    return cache.cuda(), torch.arange(nb, dtype=torch.int32, device="cuda")[None], o4.dequant(rows.numpy())


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L", [16, 17, 32, 33, 64, 200])
@pytest.mark.parametrize("G", [1, 12, 16])
def test_equal_weights_average_the_values_exactly(cuda_lib, D, L, G):
    # a query of zeros: every weight is 1 and its product with a step exact, so that only the
    # fp32 sums and the output round. The sixteenth value of a group, from which every other
    # 16 tokens are summed, lies half an fp16 step between its neighbours (-1000 + 15 * 133.25):
    # rounded to fp16 it would move the average by up to 0.125
    rng = np.random.default_rng(L + D)
    Hkv, bs = 2, 16
    codes = rng.integers(0, 16, (L, Hkv, D // 32, 32))
    st = np.full((L, Hkv, D // 32), 133.25, np.float16)
    mn = np.full((L, Hkv, D // 32), -1000.0, np.float16)
    st[:, 1], mn[:, 1] = rng.random((L, D // 32)) * 0.5, rng.standard_normal((L, D // 32))
    vc, bt, V = pool_of(codes, st, mn, bs)
    q = torch.zeros((1, G * Hkv, D), dtype=torch.float16, device="cuda")
    ref = np.repeat(V.mean(0), G, axis=0)[None]
    # A product of the sums is at most 16 steps; a tensor-core sum of 16 products and what was
    # there, cut off at fp32's last place, is off by 17 * 2^-23 of its largest term at most, and
    # 4 of them a block of 16 tokens follow one another: the sum of L tokens is off by 4 (L / 16 + 1) * 17 *
    # 2^-23 * 16 L steps at most, the average by an Lth of that
    most = np.repeat(np.maximum(16 * st.astype(np.float64), np.abs(mn.astype(np.float64))).max(0), 32, -1)
    most = np.repeat(most.reshape(Hkv, D), G, axis=0)[None]
    tol = 2.0 ** -11 * np.abs(ref) + 4 * (L / 16 + 1) * 17 * 2.0 ** -23 * most
    for splits in (0, 1):
        out = cuda_lib.decode(q, vc, vc, bt, torch.tensor([L], dtype=torch.int32, device="cuda"), 0.088,
                              max_seq_len=L, splits=splits)
        assert np.all(np.abs(rh.f64(out) - ref) <= tol)
