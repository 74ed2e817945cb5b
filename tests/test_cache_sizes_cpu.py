"""Caches of more rows than 32 bits number are refused by every entry point, also where the count of
rows passes 64 bits (no GPU)."""
import ctypes

import pytest
import torch

import paged_kv_attention_pa_gb300 as pa
from test_attend_cpu import FAR, cross_args, lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are not there")

# blocks, tokens a block, KV heads: 2^64 rows (0 in 64 bits), 2^63, 2^32, and the most that is taken
SIZES = [(1 << 30, 1 << 30, 16), (1 << 30, 1 << 30, 8), (1 << 28, 2, 8), (3, 1431655765, 1)]


@pytest.mark.parametrize("num_blocks,block_size,Hkv", SIZES)
def test_rows_of_a_cache(lib, num_blocks, block_size, Hkv):  # noqa: F811
    beyond = num_blocks * block_size * Hkv >= 1 << 32
    sizes = dict(block_size=block_size, num_blocks=num_blocks, max_blocks_per_seq=1, Hkv=Hkv, D=128, B=2, dtype=pa.PA_BF16)
    refused = lambda code: code == pa.PA_ERR_UNSUPPORTED if beyond else code == pa.PA_ERR_CUDA

    def fill(a, **kw):
        for k, v in dict(sizes, **kw).items():
            setattr(a, k, v)
        return ctypes.byref(a)

    pointers = dict(q=FAR, k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, out=4 * FAR, Hq=Hkv)
    d = fill(pa.DecodeArgs(), **pointers)
    assert refused(lib.pa_decode_ex(d, 256, 1 << 40, None))
    assert refused(lib.pa_decode_shared(d, FAR, FAR, 2, 256, 1 << 40, None))
    c = fill(pa.CrossArgs(), **pointers, rows=3, q_stride=Hkv * 128)
    assert refused(lib.pa_cross(c, 256, 1 << 40, None))
    if beyond:  # with sizes that are taken these would launch
        rows = dict(k_cache=2 * FAR, v_cache=3 * FAR, block_tables=64, seq_lens=80, rows=1)
        a = fill(pa.AppendArgs(), **rows, k=FAR, v=FAR, k_stride=Hkv * 128, v_stride=Hkv * 128, k_scale=1.0, v_scale=1.0)
        assert refused(lib.pa_append(a, 256, 1 << 40, None))
        g = fill(pa.GatherArgs(), **rows, k_scale=1.0, v_scale=1.0)
        assert refused(lib.pa_gather(g, 256, 1 << 40, None))
