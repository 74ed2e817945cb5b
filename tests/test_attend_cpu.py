"""pa_cross and pa_decode_shared on a machine without a GPU: their refusals, and the definitions that
the GPU tests hold them to."""
import ctypes

import numpy as np
import pytest
import torch

import attend_harness as ah
import paged_kv_attention_pa_gb300 as pa
from oracle import decode_ref
from paged_kv_attention_pa_gb300 import build as pa_build

FAR = 1 << 40   # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


def cross_args(**kw):
    a = pa.CrossArgs()
    base = dict(q=FAR, k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, out=4 * FAR, q_stride=1024, B=2,
                rows=5, Hq=8, Hkv=8, D=128, block_size=16, num_blocks=64, max_blocks_per_seq=32, max_seq_len=512,
                scale=0.088, dtype=pa.PA_BF16, k_scale=1.0, v_scale=1.0)
    for k, v in dict(base, **kw).items():
        setattr(a, k, v)
    return a


SIZES = [
    (dict(B=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=12), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=34, Hkv=2), pa.PA_ERR_INVALID_ARG),                      # G = 17
    (dict(Hkv=0), pa.PA_ERR_INVALID_ARG),
    (dict(D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(block_size=0), pa.PA_ERR_INVALID_ARG),
    (dict(num_blocks=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), pa.PA_ERR_INVALID_ARG),
    (dict(dtype=2), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=pa.PA_KV_INT4), pa.PA_ERR_UNSUPPORTED),
    (dict(kv_dtype=7), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=pa.PA_KV_FP8_E4M3, k_scale=0.0), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=pa.PA_KV_FP8_E4M3, v_scale=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(num_blocks=1 << 30, block_size=16), pa.PA_ERR_UNSUPPORTED),   # 32-bit row numbers
    (dict(max_seq_len=513), pa.PA_ERR_OUT_OF_RANGE),
    (dict(max_seq_len=0, max_blocks_per_seq=1 << 28), pa.PA_ERR_OUT_OF_RANGE),
    (dict(q=0), pa.PA_ERR_INVALID_ARG),
    (dict(out=0), pa.PA_ERR_INVALID_ARG),
    (dict(k_cache=0), pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0), pa.PA_ERR_INVALID_ARG),
    (dict(seq_lens=0), pa.PA_ERR_INVALID_ARG),
    (dict(q=FAR + 8), pa.PA_ERR_INVALID_ARG),
    (dict(v_cache=3 * FAR + 2), pa.PA_ERR_INVALID_ARG),
    (dict(out=4 * FAR + 4), pa.PA_ERR_INVALID_ARG),
    (dict(out=FAR), pa.PA_ERR_INVALID_ARG),                            # over the queries
    (dict(), pa.PA_ERR_CUDA),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(rows=-1), pa.PA_ERR_INVALID_ARG),
    (dict(q_stride=1028), pa.PA_ERR_INVALID_ARG),                      # not a multiple of 8
    (dict(q_stride=1016), pa.PA_ERR_INVALID_ARG),                      # rows that overlap
    (dict(q_stride=0, B=1, rows=1), pa.PA_ERR_CUDA),                   # one row: any
    (dict(out=FAR + 2 * (9 * 4096 + 1024) - 16, q_stride=4096), pa.PA_ERR_INVALID_ARG),   # at the last row's end
    (dict(out=FAR + 2 * (9 * 4096 + 1024), q_stride=4096), pa.PA_ERR_CUDA),               # right behind it
    (dict(rows=1 << 28, starts=FAR), pa.PA_ERR_UNSUPPORTED),           # rows * Hq
    (dict(rows=0), pa.PA_OK),
    (dict(B=0), pa.PA_OK),
    (dict(B=0, starts=FAR), pa.PA_OK),
])
@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")
def test_cross_refusals(lib, kw, code):
    assert lib.pa_cross(ctypes.byref(cross_args(**kw)), 256, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(q_len=-1), pa.PA_ERR_INVALID_ARG),
    (dict(splits=2), pa.PA_ERR_UNSUPPORTED),
    (dict(window=16), pa.PA_ERR_UNSUPPORTED),
    (dict(flags=2), pa.PA_ERR_INVALID_ARG),
    (dict(total_tokens=-1), pa.PA_ERR_INVALID_ARG),
    (dict(flags=pa.PA_FLAG_DETERMINISTIC), pa.PA_ERR_CUDA),
    (dict(q_len=1000), pa.PA_ERR_CUDA),                                # any number of rows
    (dict(B=0), pa.PA_OK),
])
@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")
def test_decode_shared_refusals(lib, kw, code):
    a = pa.DecodeArgs()
    base = dict(q=FAR, k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, out=4 * FAR, B=4, Hq=8, Hkv=8,
                D=128, block_size=16, num_blocks=64, max_blocks_per_seq=32, max_seq_len=512, scale=0.088,
                dtype=pa.PA_BF16, k_scale=1.0, v_scale=1.0, q_len=1)
    for k, v in dict(base, **kw).items():
        setattr(a, k, v)
    assert lib.pa_decode_shared(ctypes.byref(a), FAR, FAR, 2, 256, 1 << 40, None) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")
def test_other_refusals(lib):
    assert lib.pa_cross(None, 256, 1 << 40, None) == pa.PA_ERR_INVALID_ARG
    a = cross_args()
    for ws in (0, 128):                                                # none, not 256-byte aligned
        assert lib.pa_cross(ctypes.byref(a), ws, 1 << 40, None) == pa.PA_ERR_WORKSPACE
    d = pa.DecodeArgs()
    for k, v in dict(q=FAR, k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, out=4 * FAR, B=4, Hq=8,
                     Hkv=8, D=128, block_size=16, num_blocks=64, max_blocks_per_seq=32, dtype=pa.PA_BF16).items():
        setattr(d, k, v)
    for groups, prefix, n, code in ((0, FAR, 2, pa.PA_ERR_INVALID_ARG), (FAR, 0, 2, pa.PA_ERR_INVALID_ARG),
                                    (FAR, FAR, -1, pa.PA_ERR_INVALID_ARG), (0, 0, 0, pa.PA_ERR_CUDA)):
        assert lib.pa_decode_shared(ctypes.byref(d), groups, prefix, n, 256, 1 << 40, None) == code
    assert lib.pa_decode_shared(None, FAR, FAR, 1, 256, 1 << 40, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_cross_workspace_bytes(ctypes.byref(cross_args(D=64))) == 0


def test_python_refuses_wrong_tensors(lib):
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    kc = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    bt, sl = torch.zeros(2, 4, dtype=torch.int32), i32(5, 6)
    cross = lambda q=q, kc=kc, bt=bt, sl=sl, **kw: pa.cross(q, kc, kc, bt, sl, 0.1, **kw)
    shared = lambda q=q, kc=kc, bt=bt, sl=sl, g=i32(0, 2), p=i32(3), **kw: pa.decode_shared(q, kc, kc, bt, sl, 0.1, g, p, **kw)
    for call in (cross, shared):
        for error, kw in [(ValueError, {}),                                    # CPU tensors
                          (TypeError, dict(q=q.float())), (TypeError, dict(kc=kc.half())),
                          (ValueError, dict(kc=kc[..., :64])), (TypeError, dict(sl=sl.long())),
                          (ValueError, dict(sl=i32(5))), (ValueError, dict(q=q[:1])),
                          (ValueError, dict(q=q[0])), (ValueError, dict(out=q[:1])), (TypeError, dict(out=q.half()))]:
            with pytest.raises(error):
                call(**kw)
    for error, kw in [(ValueError, dict(starts=i32(0, 2))), (TypeError, dict(starts=i32(0, 1, 2).long())),
                      (ValueError, dict(q=q[:, None], starts=i32(0, 1, 2)))]:
        with pytest.raises(error):
            cross(**kw)
    for error, kw in [(ValueError, dict(g=i32(0, 1, 2))), (TypeError, dict(p=i32(3).long())), (ValueError, dict(g=i32())),
                      (TypeError, dict(g=None))]:
        with pytest.raises(error):
            shared(**kw)


@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_the_harness_agrees_with_the_oracle(cache):
    # one definition of attention against the other, over pools with shared prefixes
    pool = ah.Pool([40, 55, 33], 2, 128, 16, "bf16", cache, seed=3, prefixes=[(0, 3, 33)])
    q = ah.queries((3, 4, 128), "bf16", 3).double().numpy()
    want = decode_ref(q, pool.K, pool.V, 0.1)
    for b in range(3):
        got, mag, _ = ah.attend(q[b][None], pool.K[b], pool.V[b], 0.1)
        assert np.allclose(got[0], want[b], rtol=0, atol=1e-12) and np.all(mag >= np.abs(got) - 1e-12)
    assert np.array_equal(pool.K[0][:33], pool.K[1][:33]) and torch.equal(pool.bt[0, :2], pool.bt[2, :2])
    # the causal limit, and rows that see nothing
    got, _, _ = ah.attend(q[:, :2][:, :, :], pool.K[0], pool.V[0], 0.1, [0, 1, 40])
    assert np.all(got[0] == 0) and np.allclose(got[1, 0], pool.V[0][0, 0])
