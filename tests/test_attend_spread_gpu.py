"""Few rows over fp8 caches, whose tokens the four warps of a softmax group share (GB300 only): row
counts about its limits (16 rows, 32 rows), with enough tiles that a CTA holds long pieces, ends and
beginnings of items and, among them, short ones that one warp takes."""
import numpy as np
import pytest
import torch

import attend_harness as ah
from test_cross_gpu import run
from test_decode_shared_gpu import run as run_shared

pytestmark = pytest.mark.gpu

LENS = [2500, 1, 900, 3100, 0, 1408, 130, 2047, 768, 1537, 64, 2900, 897, 2304, 15, 1100]


@pytest.mark.parametrize("rows,G", [(1, 1), (1, 16), (2, 8), (17, 1), (5, 3), (4, 7), (8, 4), (32, 1), (2, 16), (33, 1)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256)])
def test_rows(cuda_lib, rows, G, dtype, D):
    pool = ah.Pool(LENS, 4, D, 16, dtype, "fp8", seed=rows * G)
    q = ah.queries((len(LENS), rows, 4 * G, D), dtype, rows)
    a = run(cuda_lib, pool, q, [rows] * len(LENS))
    b = run(cuda_lib, pool, q, [rows] * len(LENS))
    assert torch.equal(a, b)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 256)])
def test_raised_references(cuda_lib, dtype, D, sign):
    # scores that grow along the context raise every warp's reference many times
    pool = ah.Pool(LENS, 4, D, 33, dtype, "fp8", seed=9)
    kc = pool.caches[0].view(torch.uint8)
    for b, L in enumerate(LENS):
        t = torch.arange(L)
        k = pool.K[b] * 0.1
        k[..., 0] = (np.arange(L) / max(L, 1) * 4.0)[:, None]
        raw = torch.tensor(k / pool.scale).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        kc[pool.bt[b, t // 33].long(), t % 33] = raw.view(torch.uint8)
        pool.K[b] = ah.e4m3_to_float64(raw.view(torch.uint8).numpy()) * float(np.float32(pool.scale))
    q = ah.queries((len(LENS), 6, 8, D), dtype, 5)
    q[..., 0] = 8.0 * sign
    run(cuda_lib, pool, q, [6] * len(LENS), scale=sign)


@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256)])
def test_behind_prefixes(cuda_lib, dtype, D, rows):
    # members whose own contexts begin inside a tile, some of them short, some long
    prefixes = [(0, 3, 1500), (3, 5, 2000), (7, 12, 333)]
    lens = [2600, 1505, 3000, 2010, 3900, 1200, 4, 900, 3333, 340, 1800, 2500, 2048, 777]
    pool = ah.Pool(lens, 4, D, 16, dtype, "fp8", seed=rows, prefixes=prefixes)
    run_shared(cuda_lib, pool, ah.queries((len(lens), rows, 16, D), dtype, rows), [0, 3, 5, 7, 12], [1500, 2000, 0, 333])


def test_nan_rows_stay_apart(cuda_lib):
    pool = ah.Pool(LENS, 4, 128, 16, "bf16", "fp8", seed=3)
    q = ah.queries((len(LENS), 4, 16, 128), "bf16", 3)
    kc, vc, bt, sl = pool.cuda()
    call = lambda x: cuda_lib.cross(x.cuda(), kc, vc, bt, sl, 0.09, k_scale=pool.scale, v_scale=pool.scale)
    good = call(q)
    bad = q.clone()
    bad[3, 1, 2, 7] = float("nan")
    got = call(bad)
    assert torch.isnan(got[3, 1, 2]).all()
    got[3, 1, 2] = good[3, 1, 2]
    assert torch.equal(got, good)
