"""Decode behind shared prefixes against its definition in 64 bits (GB300 only)."""
import numpy as np
import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(pa, pool, q, groups, prefix, errors=0, **kw):
    """Call and check every sequence over its whole context."""
    scale = float(np.float32(pool.D ** -0.5))
    kc, vc, bt, sl = pool.cuda()
    out = pa.decode_shared(q.cuda(), kc, vc, bt, sl, scale, i32(groups), i32(prefix), k_scale=pool.scale,
                           v_scale=pool.scale, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_errors(pa.default_workspace()) == errors
    R = q.shape[1] if q.dim() == 4 else 1
    rows = q.double().numpy().reshape(len(pool.lens), R, *q.shape[-2:])
    got = out.reshape(rows.shape)
    for b, L in enumerate(pool.lens):
        lim = [max(0, L - R + i + 1) for i in range(R)]
        ref, mag, size = ah.attend(rows[b], pool.K[b], pool.V[b], scale, lim)
        ah.check(got[b], ref, mag, size, pool, scale, f"sequence {b}")
    return out


@pytest.mark.parametrize("P", [1, 15, 16, 17, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("own_prefix", [True, False])
@pytest.mark.parametrize("dtype,D,cache", [("bf16", 128, "same"), ("f16", 256, "same"), ("bf16", 128, "fp8")])
def test_one_group(cuda_lib, P, own_prefix, dtype, D, cache):
    # with and without the prefix in the other sequences' own tables: it is read from the first's
    lens = [P, P + 1, P + 16, P + 200, P + 33]
    pool = ah.Pool(lens, 2, D, 16, dtype, cache, seed=P, prefixes=[(0, 5, P)], own_prefix=own_prefix)
    run(cuda_lib, pool, ah.queries((5, 8, D), dtype, P), [0, 5], [P])


@pytest.mark.parametrize("R", [1, 2, 4, 9])
@pytest.mark.parametrize("G", [1, 3, 16])
def test_groups_and_sequences_alone(cuda_lib, R, G):
    # sequence 0 and the last two belong to no group; one group is empty, one has one sequence
    lens = [40, 333, 340, 420, 90, 150, 151, 260, 20, R]
    groups, prefix = [1, 4, 4, 5, 8], [330, 77, 90, 145]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=R + G, prefixes=[(1, 4, 330), (5, 8, 145)])
    run(cuda_lib, pool, ah.queries((10, R, 2 * G, 128), "bf16", R), groups, prefix)


@pytest.mark.parametrize("bs", [8, 33, 64, 784])
@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (256, "fp8")])
def test_block_sizes(cuda_lib, bs, D, cache):
    lens = [900, 850, 801, 1200, 830, 100]
    pool = ah.Pool(lens, 4, D, bs, "f16", cache, seed=bs, prefixes=[(0, 5, 800)], own_prefix=False)
    run(cuda_lib, pool, ah.queries((6, 24, D), "f16", bs), [0, 5], [800])


def test_many_sequences_of_a_group(cuda_lib):
    # 600 sequences: more segments than the CTA has threads, more rows than an item
    rng = np.random.default_rng(5)
    lens = (64 + rng.integers(0, 40, 600)).tolist()
    pool = ah.Pool(lens, 1, 128, 16, "bf16", seed=5, prefixes=[(3, 590, 64)])
    run(cuda_lib, pool, ah.queries((600, 4, 128), "bf16", 5), [3, 590], [64])


def test_prefixes_longer_than_sequences(cuda_lib):
    # what is shared ends with the group's first sequence; shorter members see their part of it, an
    # empty one (a padded batch) nothing
    lens = [200, 120, 0, 260, 200, 3]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=9, prefixes=[(0, 6, 200)])
    run(cuda_lib, pool, ah.queries((6, 4, 128), "bf16", 9), [0, 6], [250], max_seq_len=272)
    # an empty first sequence: nothing is shared
    lens = [0, 120, 121]
    pool = ah.Pool(lens, 2, 128, 16, "bf16", seed=10)
    run(cuda_lib, pool, ah.queries((3, 4, 128), "bf16", 10), [0, 3], [100])


def test_no_groups(cuda_lib):
    pool = ah.Pool([77, 0, 1000], 2, 128, 16, "f16", seed=11)
    out = run(cuda_lib, pool, ah.queries((3, 4, 128), "f16", 11), [0], [])
    assert torch.all(out[1] == 0)
