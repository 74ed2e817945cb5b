"""Sizes whose products pass 64 bits are refused by pa_cross and pa_decode_shared before anything is
computed from them (no GPU)."""
import ctypes

import pytest
import torch

import paged_kv_attention_pa_gb300 as pa
from test_attend_cpu import FAR, cross_args, lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")


@pytest.mark.parametrize("B,rows,Hq,Hkv", [(1 << 30, 1 << 30, 16, 8),       # 2^64: 0 in 64 bits
                                           (1 << 30, 1 << 30, 8, 8),        # 2^63: negative
                                           ((1 << 31) - 1, (1 << 31) - 1, 32, 16),
                                           (1 << 28, 1 << 28, 8, 8), (1, 1 << 28, 8, 8), (1 << 28, 1, 8, 8)])
def test_rows_in_all(lib, B, rows, Hq, Hkv):  # noqa: F811
    a = cross_args(B=B, rows=rows, Hq=Hq, Hkv=Hkv, q_stride=Hq * 128)
    assert lib.pa_cross(ctypes.byref(a), 256, 1 << 40, None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_cross_workspace_bytes(ctypes.byref(a)) == 0
    d = pa.DecodeArgs()
    for k, v in dict(q=FAR, k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, out=4 * FAR, B=B, Hq=Hq,
                     Hkv=Hkv, D=128, block_size=16, num_blocks=64, max_blocks_per_seq=32, dtype=pa.PA_BF16,
                     q_len=rows).items():
        setattr(d, k, v)
    assert lib.pa_decode_shared(ctypes.byref(d), FAR, FAR, 2, 256, 1 << 40, None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_decode_shared_workspace_bytes(ctypes.byref(d), 2) == 0


@pytest.mark.parametrize("stride,code", [(1 << 39, pa.PA_ERR_UNSUPPORTED),   # a tensor copy's strides: below 2^40 bytes
                                         (1 << 60, pa.PA_ERR_UNSUPPORTED),   # nine of them: 2^64 bytes and more
                                         ((1 << 63) - 8, pa.PA_ERR_UNSUPPORTED),
                                         ((1 << 39) - 8, pa.PA_ERR_CUDA)])
def test_strides(lib, stride, code):  # noqa: F811
    a = cross_args(q_stride=stride, out=FAR - (1 << 20))
    assert lib.pa_cross(ctypes.byref(a), 256, 1 << 40, None) == code
    a.B = a.rows = 1                                                        # one row: any
    assert lib.pa_cross(ctypes.byref(a), 256, 1 << 40, None) == pa.PA_ERR_CUDA
