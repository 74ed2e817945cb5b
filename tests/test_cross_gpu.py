"""Cross attention against its definition in 64 bits (GB300 only)."""
import numpy as np
import pytest
import torch

import attend_harness as ah

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(pa, pool, q, rows, starts=None, scale=None, **kw):
    """Call and check; rows: query rows of each sequence."""
    scale = float(np.float32(pool.D ** -0.5)) if scale is None else scale
    kc, vc, bt, sl = pool.cuda()
    out = pa.cross(q.cuda(), kc, vc, bt, sl, scale, starts=None if starts is None else i32(starts),
                   k_scale=pool.scale, v_scale=pool.scale, **kw)
    torch.cuda.synchronize()
    assert pa.read_device_errors(pa.default_workspace()) == 0
    flat = ah.f64(q) if hasattr(ah, "f64") else q.double().numpy()
    flat = flat.reshape(-1, *q.shape[-2:])
    got = out.reshape(flat.shape)
    at = 0 if starts is None else starts[0]
    for b, n in enumerate(rows):
        ref, mag, size = ah.attend(flat[at:at + n], pool.K[b], pool.V[b], scale)
        ah.check(got[at:at + n], ref, mag, size, pool, scale, f"sequence {b}")
        at += n
    return out


@pytest.mark.parametrize("L", [0, 1, 7, 16, 127, 128, 129, 500, 1500])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256)])
def test_one_row(cuda_lib, L, dtype, D):
    pool = ah.Pool([L], 2, D, 16, dtype, seed=L)
    run(cuda_lib, pool, ah.queries((1, 4, D), dtype, L), [1])


@pytest.mark.parametrize("rows", [1, 5, 31, 32, 33, 63, 65, 100, 300])
@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f16", 128, 3), ("bf16", 256, 6), ("f16", 256, 1)])
def test_rows_of_a_sequence(cuda_lib, rows, dtype, D, G):
    # below, at and above the row tiles of 128 (row, head) pairs
    pool = ah.Pool([200, 0, 431], 2, D, 16, dtype, seed=rows)
    run(cuda_lib, pool, ah.queries((3, rows, 2 * G, D), dtype, rows), [rows] * 3)


@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 33, 64, 128, 256, 784])
@pytest.mark.parametrize("D,cache", [(128, "same"), (256, "same"), (128, "fp8"), (256, "fp8")])
def test_block_sizes(cuda_lib, bs, D, cache):
    pool = ah.Pool([1, bs, 3 * bs + 1 if bs < 100 else 300, 777], 2, D, bs, "bf16", cache, seed=bs)
    run(cuda_lib, pool, ah.queries((4, 9, 8, D), "bf16", bs), [9] * 4)


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [1, 2, 7, 16])
def test_packed_rows(cuda_lib, cache, dtype, G):
    counts = [3, 0, 40, 1, 129, 0, 64]
    starts = np.concatenate([[2], 2 + np.cumsum(counts)]).tolist()   # two rows of padding before
    total = starts[-1] + 3                                            # and three behind
    pool = ah.Pool([130, 50, 257, 0, 640, 10, 33], 2, 128, 16, dtype, cache, seed=G)
    q = ah.queries((total, 2 * G, 128), dtype, G)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    run(cuda_lib, pool, q, counts, starts, out=out)
    assert torch.all(out[:2] == 7.0) and torch.all(out[starts[-1]:] == 7.0)
