"""Calls at the edges of what the Python functions and the C entry points take, without a GPU."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_attention_pa_gb300 as pa
from paged_kv_attention_pa_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


@pytest.mark.parametrize("fn", [pa.decode_plain, pa.decode_noalloc])
def test_plain_calls_refuse_what_their_entry_points_cannot_tell(lib, fn):
    # pa_decode and pa_decode_noalloc take no cache type and no query rows: an fp8 or 4-bit cache
    # would be read as 16-bit rows, past its end
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    c4 = torch.zeros(4, 8, 16, pa.int4_row_bytes(128), dtype=torch.uint8)
    for k, v in ((c4, c4), (kc.to(torch.float8_e4m3fn),) * 2, (kc, c4), (kc.half(),) * 2):
        with pytest.raises(TypeError, match="dtype"):
            fn(q, k, v, bt, sl, 0.1)
    with pytest.raises(ValueError, match="B, Hq, D"):
        fn(q[:, None].expand(2, 3, 8, 128).contiguous(), kc, kc, bt, sl, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        fn(q, kc, kc, bt, sl, 0.1)


@pytest.mark.parametrize("kw", [{}, dict(kv_fp8=True), dict(kv_int4=True), dict(splits=3), dict(window=64)])
def test_plan_of_an_empty_batch(lib, kw):
    # nothing to split, and no division by the number of (sequence, KV head) pairs
    S, P = pa.plan(0, 8, 8, 128, 16, 512, sm_count=152, **kw)
    assert S == 1 and P >= 16


@pytest.mark.parametrize("B", [0, 1, 3])
def test_append_of_no_tokens_is_not_refused_for_its_strides(lib, B):
    # [B, 0, H, D]: the next check is the device's
    k, q = torch.zeros(B, 0, 2, 128).half(), torch.zeros(B, 0, 4, 128).half()
    kc = torch.zeros(4, 16, 2, 128).half()
    bt, sl = torch.zeros(B, 1, dtype=torch.int32), torch.ones(B, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pa.append(k, k, kc, kc, bt, sl, q=q)


def test_append_refuses_rows_that_are_not_evenly_spaced(lib):
    k = torch.zeros(3, 4, 2, 128).half()[:, :3]
    kc = torch.zeros(4, 16, 2, 128).half()
    bt, sl = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="evenly spaced"):
        pa.append(k, k, kc, kc, bt, sl)


def test_numbers_are_taken_as_int_and_float_take_them(lib):
    # whole numbers held as floats, arrays or tensors of one element; the next check is the device's
    q = torch.zeros(2, 8, 128).half()
    kc = torch.zeros(4, 16, 8, 128).half()
    bt, sl = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for n in (16, 16.0, np.float64(16), np.int32(16), torch.tensor(16), torch.tensor(16.0)):
        with pytest.raises(ValueError, match="CUDA"):
            pa.decode(q, kc, kc, bt, sl, np.float32(0.1), max_seq_len=n, splits=n, window=n, total_tokens=n)
        with pytest.raises(ValueError, match="CUDA"):
            pa.decode(q, kc, kc, bt, sl, torch.tensor(0.1), max_seq_len=n)
    for bad in ("sixteen", [16], torch.zeros(2), float("nan"), float("inf"), 2.0 ** 40):
        with pytest.raises((TypeError, ValueError, RuntimeError, OverflowError)) as e:
            pa.decode(q, kc, kc, bt, sl, 0.1, max_seq_len=bad)
        assert "CUDA" not in str(e.value)


def test_a_library_loaded_from_elsewhere_serves_every_call(lib, tmp_path):
    # one library is mapped, the one at the path given to load()
    other = str(tmp_path / "libpa_copy.so")
    shutil.copy(pa.LIB_PATH, other)
    code = ("import sys, torch, paged_kv_attention_pa_gb300 as pa\n"
            f"pa.load({other!r})\n"
            "maps = open('/proc/self/maps').read()\n"
            "assert 'libpa_copy.so' in maps and '/libpa.so' not in maps\n"
            "q, c = torch.zeros(2, 8, 128).half(), torch.zeros(4, 16, 8, 128).half()\n"
            "bt, sl = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)\n"
            "try:\n    pa.decode(q, c, c, bt, sl, 0.1)\n"
            "except ValueError as e:\n    assert 'CUDA' in str(e)\n"
            "else:\n    sys.exit(3)\n")
    root = os.path.dirname(os.path.dirname(pa.LIB_PATH))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


class FakeLib:
    """pa_read_device_errors on host memory."""

    def pa_set_device(self, index):
        return pa.PA_OK

    def pa_read_device_errors(self, ws, stream, flags):
        word = ctypes.c_uint32.from_address(ws)
        flags._obj.value, word.value = word.value, 0
        return pa.PA_OK


class FakeStream:
    cuda_stream = 77


capture = [0]  # the id of the capture under way


@pytest.fixture
def host_workspaces(monkeypatch):
    capture[0] = 0
    monkeypatch.setattr(pa, "load", FakeLib)
    monkeypatch.setattr(pa, "_capture_of", lambda stream_handle: capture[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capture[0]))
    monkeypatch.setattr(pa, "_workspaces", {})
    monkeypatch.setattr(pa, "_captured", {}, raising=False)
    monkeypatch.setattr(pa, "_outgrown", [])
    return lambda need: pa._workspace(need, torch.device("cpu"), FakeStream.cuda_stream)


def test_error_bits_survive_the_growth_of_a_workspace(host_workspaces):
    # append's kernel reports into the stream's workspace, decode replaces it by a larger one
    ws = host_workspaces(pa.PA_WORKSPACE_HEADER_BYTES)
    ws[0] = pa.PA_DEVERR_BLOCK_INDEX
    more = host_workspaces(ws.numel() + 1)
    more[0] = pa.PA_DEVERR_COPY
    most = host_workspaces(more.numel() + 1)
    most[0] = pa.PA_DEVERR_SEQ_LEN
    assert len({w.data_ptr() for w in (ws, more, most)}) == 3
    assert pa.read_device_errors(most, FakeStream) == 7
    assert pa.read_device_errors(most, FakeStream) == 0
    assert pa.read_device_errors(torch.zeros(64, dtype=torch.uint8), FakeStream) == 0


def test_a_capture_has_one_workspace_of_its_own(host_workspaces):
    eager = host_workspaces(1 << 16)
    capture[0] = 5
    mine = host_workspaces(1 << 16)
    assert mine is not eager                       # calls outside may run beside the graph's
    assert all(host_workspaces(n) is mine for n in (1, pa.PA_WORKSPACE_HEADER_BYTES, 1 << 16))
    grown = host_workspaces((1 << 16) + 1)
    assert grown.outgrown is mine and host_workspaces(1 << 16) is grown
    capture[0] = 6
    other = host_workspaces(1 << 16)
    assert other is not grown and other is not eager and not hasattr(other, "outgrown")
    capture[0] = 0
    assert host_workspaces(1 << 16) is eager and pa._outgrown == []


def test_no_capture_without_a_device(lib):
    assert pa._capture_of(0) == 0


def test_plan_knows_the_query_rows(lib):
    # unsplit short contexts run on short CTAs with at most eight columns: another cost, another plan
    kw = dict(sm_count=152, kv_int4=True, total_tokens=1600)
    one = pa.plan(10, 64, 16, 128, 16, 160, **kw)
    assert one == pa.plan(10, 64, 16, 128, 16, 160, rows=1, **kw) == pa.plan(10, 64, 16, 128, 16, 160, rows=2, **kw)
    assert one != pa.plan(10, 64, 16, 128, 16, 160, rows=4, **kw)
    with pytest.raises(pa.PAError):
        pa.plan(1, 32, 8, 128, 16, 512, sm_count=152, rows=9)


@pytest.mark.parametrize("kw,code", [
    (dict(q=32, q_out=32, q_stride=8 * 128), pa.PA_ERR_WORKSPACE),          # in place: the next check
    (dict(q=32, q_out=32, q_stride=24 * 128), pa.PA_ERR_INVALID_ARG),       # the heads of a projection's rows
    (dict(q=32, q_out=32, q_stride=24 * 128, B=1), pa.PA_ERR_WORKSPACE),    # one row: dense
    (dict(q=32, q_out=32, q_stride=24 * 128, rows=0), pa.PA_OK),
])
def test_append_in_place_needs_dense_queries(lib, kw, code):
    # q_out is dense: written over the strided rows of q, it would destroy rows not yet read
    a = pa.AppendArgs()
    base = dict(q=16, q_out=32, k=48, v=64, k_cache=80, v_cache=96, block_tables=4, seq_lens=8, q_stride=1024,
                k_stride=1024, v_stride=1024, B=2, rows=1, Hq=8, Hkv=8, D=128, block_size=16, num_blocks=8,
                max_blocks_per_seq=4, dtype=pa.PA_BF16, rope_amplitude=1.0)
    for k, v in dict(base, **kw).items():
        setattr(a, k, v)
    assert lib.pa_append(ctypes.byref(a), 0, 0, None) == code


def test_calls_run_on_their_tensors_device_and_leave_the_current_one(monkeypatch):
    # the current device may have changed since the last call, and belongs to the caller
    at = [0]

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before = at[0]
            if self.index >= 0:
                at[0] = self.index

        def __exit__(self, *_):
            at[0] = self.before

    class Lib(FakeLib):
        seen = []

        def pa_set_device(self, index):
            at[0] = index
            return pa.PA_OK

        def pa_read_device_errors(self, ws, stream, flags):
            self.seen.append(at[0])
            return pa.PA_OK

    class Workspace:
        def __init__(self, index):
            self.is_cuda, self.device = True, torch.device("cuda", index)

        def data_ptr(self):
            return 256

    monkeypatch.setattr(pa, "load", Lib)
    monkeypatch.setattr(torch.cuda, "device", device)
    for current in (0, 2):
        at[0] = current
        for index in (1, 0, 1):
            pa.read_device_errors(Workspace(index), FakeStream)
            assert Lib.seen[-1] == index and at[0] == current
