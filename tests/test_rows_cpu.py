"""Append, gather, rotary frequencies and 4-bit rows without a GPU: the oracle's own pins, the
frequencies the library computes, argument checks and refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_pa_gb300 as pa
from oracle import int4 as o4
from oracle import rope as orope
from paged_kv_attention_pa_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


# ---------------------------------------------------------------- oracle pins
@pytest.mark.parametrize("D", [128, 256])
def test_int4_pack_and_unpack_agree(D):
    rng = np.random.default_rng(0)
    G = D // 32
    codes = rng.integers(0, 16, (5, 2, G, 32))
    st = rng.random((5, 2, G)).astype(np.float16)
    mn = rng.standard_normal((5, 2, G)).astype(np.float16)
    rows = o4.pack(codes, st, mn)
    assert rows.shape == (5, 2, o4.row_bytes(D)) and pa.int4_row_bytes(D) == o4.row_bytes(D)
    c, s, m = o4.unpack(rows)
    assert np.array_equal(c, codes) and np.array_equal(s, st) and np.array_equal(m, mn)


def test_int4_word_order_by_hand():
    # D = 128: element d sits in word (d % 32 // 8) * 4 + d // 32, bits 4 (d % 8)
    for d in (0, 1, 7, 8, 31, 32, 77, 127):
        codes = np.zeros((1, 4, 32), dtype=np.int64)
        codes[0, d // 32, d % 32] = 9
        rows = o4.pack(codes, np.ones((1, 4), np.float16), np.zeros((1, 4), np.float16))
        words = rows[0, :64].copy().view("<u4")
        want = np.zeros(16, dtype=np.uint32)
        want[(d % 32 // 8) * 4 + d // 32] = 9 << (4 * (d % 8))
        assert np.array_equal(words, want), d


def test_int4_quantise_is_within_half_a_step():
    rng = np.random.default_rng(1)
    for scale in (1e-3, 1.0, 300.0):
        x = scale * rng.standard_normal((64, 128))
        rows = o4.quantise(x)
        _, st, _ = o4.unpack(rows)
        err = np.abs(o4.dequant(rows) - x).reshape(64, 4, 32)
        assert np.all(err <= st[..., None] * 0.5 * (1 + 1e-12))
    x = np.full((1, 128), 3.0)                      # no range: exact
    assert np.array_equal(o4.dequant(o4.quantise(x)), x)


def test_int4_quantise_saturates_within_fp16():
    # beyond +-65280 values saturate, and every value of a row, the sixteenth of each group
    # among them, rounds to a finite fp16
    rng = np.random.default_rng(0)
    x = rng.standard_normal((400, 128)) * np.exp(rng.uniform(5, 88, (400, 1)))
    x[:100] = np.sign(x[:100]) * 65280.0 * (1 - rng.uniform(0, 1e-2, (100, 128)))
    codes, steps, minima = o4.unpack(o4.quantise(x))
    assert steps.max() <= 8704 and np.abs(minima).max() <= 65280 + 32
    assert np.isfinite((minima + 15 * steps).astype(np.float16)).all()
    want = np.clip(x, -65280, 65280).reshape(400, 4, 32)
    got = minima[..., None] + steps[..., None] * codes
    assert np.all(np.abs(got - want) <= steps[..., None] / 2 * (1 + 1e-12))


def test_rotation_preserves_relative_positions():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f, _ = orope.frequencies(64)
    for il in (False, True):
        dots = [float((orope.rotate(q, [5 + s], f, il) * orope.rotate(k, [2 + s], f, il)).sum())
                for s in (0, 1, 1000, 10 ** 6)]
        # angles up to 1e6 rad in float64: 1e6 * 2^-53 * |q||k|
        assert max(dots) - min(dots) < 1e-7
        assert np.allclose(orope.rotate(q, [0], f, il), q)


# ---------------------------------------------------------------- frequencies
@pytest.mark.parametrize("kw", [
    dict(), dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
    dict(kind="yarn", factor=8.0, original_max=4096),
    dict(kind="yarn", factor=2.0, original_max=64, slow=0.5, fast=4.0),
    dict(kind="banded", factor=8.0, original_max=8192, slow=1.0, fast=4.0),
])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 10000.0), (64, 500000.0), (256, 1e6)])
def test_rope_turns(lib, rot, base, kw):
    o = dict(kw)
    r = pa.rope(rot, base=base, scaling=o.pop("kind", None), device="cpu", **o)
    f, amp = orope.frequencies(rot, base, **kw)
    turns = r.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # fp64 on both sides: pow, log and the blend cost a few units in the last place; the
    # fraction of a turn is cut to a multiple of 2^-64
    assert np.allclose(turns * 2 * math.pi, f, rtol=1e-13, atol=2 * math.pi * 2.0 ** -64)
    assert abs(r.amplitude - amp) <= 2.0 ** -24 * amp


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=272), dict(base=1.0), dict(base=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
    dict(scaling="banded", factor=2.0, original_max=64, slow=4.0, fast=4.0),
])
def test_rope_refusals(lib, kw):
    args = dict(rot_dim=64, base=10000.0, device="cpu")
    args.update(kw)
    with pytest.raises(pa.PAError):
        pa.rope(**args)


def test_rope_unknown_scaling(lib):
    with pytest.raises(ValueError):
        pa.rope(64, scaling="other", device="cpu")


# ---------------------------------------------------------------- C argument checks
def _append(**kw):
    a = pa.AppendArgs()
    base = dict(q=16, q_out=32, k=48, v=64, k_cache=80, v_cache=96, block_tables=4, seq_lens=8,
                rope_turns=8, q_stride=1024, k_stride=1024, v_stride=1024, B=2, rows=1, Hq=8,
                Hkv=8, D=128, block_size=16, num_blocks=8, max_blocks_per_seq=4,
                dtype=pa.PA_BF16, kv_dtype=0, k_scale=1.0, v_scale=1.0, rot_dim=128,
                rope_layout=0, rope_amplitude=1.0)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


def _gather(**kw):
    a = pa.GatherArgs()
    base = dict(k_cache=16, v_cache=32, block_tables=4, seq_lens=8, k_out=48, v_out=64, B=2,
                rows=3, Hkv=8, D=128, block_size=16, num_blocks=8, max_blocks_per_seq=4,
                dtype=pa.PA_F16, kv_dtype=0, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


SHARED = [
    (dict(B=-1), pa.PA_ERR_INVALID_ARG), (dict(rows=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hkv=0), pa.PA_ERR_INVALID_ARG), (dict(Hkv=65536), pa.PA_ERR_INVALID_ARG),
    (dict(D=64), pa.PA_ERR_UNSUPPORTED), (dict(D=0), pa.PA_ERR_INVALID_ARG),
    (dict(block_size=0), pa.PA_ERR_INVALID_ARG), (dict(num_blocks=0), pa.PA_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), pa.PA_ERR_INVALID_ARG), (dict(dtype=5), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=3), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=1, k_scale=0.0), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=2, v_scale=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(kv_dtype=2, v_scale=1e-45), pa.PA_ERR_INVALID_ARG),       # 1 / scale is infinite
    (dict(num_blocks=1 << 24, block_size=784), pa.PA_ERR_UNSUPPORTED),
    (dict(max_blocks_per_seq=1 << 28), pa.PA_ERR_OUT_OF_RANGE),     # positions past 2^31
    (dict(B=1 << 20, rows=1 << 12), pa.PA_ERR_INVALID_ARG),         # rows past 2^31
    (dict(k_cache=0), pa.PA_ERR_INVALID_ARG), (dict(v_cache=8), pa.PA_ERR_INVALID_ARG),
    (dict(block_tables=0), pa.PA_ERR_INVALID_ARG), (dict(seq_lens=0), pa.PA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(q_out=0), pa.PA_ERR_INVALID_ARG), (dict(q=0), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=0), pa.PA_ERR_INVALID_ARG), (dict(Hq=70000), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=24), pa.PA_ERR_INVALID_ARG), (dict(rot_dim=-16), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=144), pa.PA_ERR_INVALID_ARG), (dict(rope_turns=0), pa.PA_ERR_INVALID_ARG),
    (dict(rope_layout=2), pa.PA_ERR_INVALID_ARG),
    (dict(rope_amplitude=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(k_stride=1028), pa.PA_ERR_INVALID_ARG), (dict(v_stride=-1024), pa.PA_ERR_INVALID_ARG),
    (dict(q_stride=4), pa.PA_ERR_INVALID_ARG), (dict(k=0), pa.PA_ERR_INVALID_ARG),
    (dict(v=40), pa.PA_ERR_INVALID_ARG), (dict(q_out=24), pa.PA_ERR_INVALID_ARG),
])
def test_append_refusals(lib, kw, code):
    assert lib.pa_append(ctypes.byref(_append(**kw)), 256, 1 << 16, None) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(k_out=0), pa.PA_ERR_INVALID_ARG), (dict(v_out=72), pa.PA_ERR_INVALID_ARG),
])
def test_gather_refusals(lib, kw, code):
    assert lib.pa_gather(ctypes.byref(_gather(**kw)), 256, 1 << 16, None) == code


def test_rows_workspace_and_empty_calls(lib):
    for fn, a in ((lib.pa_append, _append), (lib.pa_gather, _gather)):
        assert fn(None, 256, 1 << 16, None) == pa.PA_ERR_INVALID_ARG
        assert fn(ctypes.byref(a()), 0, 1 << 16, None) == pa.PA_ERR_WORKSPACE
        assert fn(ctypes.byref(a()), 272, 1 << 16, None) == pa.PA_ERR_WORKSPACE
        assert fn(ctypes.byref(a()), 256, 256, None) == pa.PA_ERR_WORKSPACE
        assert fn(ctypes.byref(a(B=0)), 0, 0, None) == pa.PA_OK
        assert fn(ctypes.byref(a(rows=0)), 0, 0, None) == pa.PA_OK
        if not torch.cuda.is_available():
            assert fn(ctypes.byref(a()), 256, 1 << 16, None) == pa.PA_ERR_CUDA
    assert lib.pa_append(ctypes.byref(_append(q=0, q_out=0, Hq=0, rows=0)), 0, 0, None) == pa.PA_OK


# ---------------------------------------------------------------- decode over 4 bits, host side
def test_int4_decode_arguments(lib):
    a = pa.DecodeArgs()
    for k, v in dict(q=16, k_cache=32, v_cache=48, block_tables=64, seq_lens=80, out=96, B=1, Hq=8,
                     Hkv=8, D=128, block_size=16, num_blocks=64, max_blocks_per_seq=32,
                     max_seq_len=512, scale=0.088, dtype=pa.PA_BF16, kv_dtype=pa.PA_KV_INT4,
                     k_scale=1.0, v_scale=0.0).items():
        setattr(a, k, v)
    assert lib.pa_decode_ex(ctypes.byref(a), 256, 1 << 20, None) == pa.PA_ERR_INVALID_ARG
    a.v_scale = 1.0
    a.k_scale = float("inf")
    assert lib.pa_decode_ex(ctypes.byref(a), 256, 1 << 20, None) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("B,hkv,D,bs,L", [(1, 8, 128, 16, 512), (1, 4, 256, 784, 32768),
                                          (8, 8, 128, 16, 16384), (64, 8, 128, 33, 4096),
                                          (3, 1, 256, 1, 300000)])
def test_int4_plan_covers_the_context(lib, B, hkv, D, bs, L):
    for splits in (0, 1, 3, 7):
        S, P = pa.plan(B, 2 * hkv, hkv, D, bs, L, splits=splits, sm_count=152, kv_int4=True)
        assert P % 16 == 0 and S * P >= L and (S - 1) * P < L and 1 <= S <= 1024


# ---------------------------------------------------------------- Python refusals (CPU tensors)
def test_python_refuses_wrong_tensors(lib):
    k = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    c4 = torch.zeros(4, 8, 16, 80, dtype=torch.uint8)
    bt, sl = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.append(k, k, kc, kc, bt, sl)
    with pytest.raises(ValueError, match="CUDA"):
        pa.gather(kc, kc, bt, sl, 1)
    with pytest.raises(TypeError):
        pa.append(k.float(), k.float(), kc, kc, bt, sl)
    with pytest.raises(TypeError):
        pa.append(k, k, kc, kc.half(), bt, sl)
    with pytest.raises(ValueError):
        pa.append(k, k, kc, c4, bt, sl)
    with pytest.raises(TypeError):
        pa.append(k, k, kc, kc, bt.long(), sl)
    with pytest.raises(TypeError):
        pa.gather(c4, c4, bt, sl, 1)                       # the 16-bit dtype is needed
    with pytest.raises(ValueError):
        pa.gather(c4[..., :78], c4[..., :78], bt, sl, 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.append(k, k, kc, kc, bt[:1], sl)
    with pytest.raises(ValueError):
        pa.gather(kc, kc, bt, sl, 1, starts=torch.zeros(2, dtype=torch.int32))
