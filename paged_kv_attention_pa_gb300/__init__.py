"""Python binding of libpa.so: single-query paged-attention decode on GB300, and the
rows of its paged cache (append with rotary positions, gather).

Argument marshalling only (the hot calls' in csrc/binding.cpp): every step of the
computation runs in the CUDA kernels behind the C ABI declared in include/pa.h. PyTorch provides device
memory and the current stream. There is no CPU path: if the shared library is
missing, every call raises.

    import paged_kv_attention_pa_gb300 as pa
    out = pa.decode(q, k_cache, v_cache, block_tables, seq_lens, scale,
                    max_seq_len=4096)

A decode step of a layer, from the projection's output:

    rope = pa.rope(128, base=10000.0, device="cuda")
    q = pa.append(k, v, k_cache, v_cache, block_tables, seq_lens, q=q, rope=rope)
    out = pa.decode(q, k_cache, v_cache, block_tables, seq_lens, scale)
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional, Tuple

import torch

__version__ = "0.1.0"

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

# status codes (include/pa.h)
PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA, \
    PA_ERR_OUT_OF_RANGE = range(6)
PA_F16, PA_BF16 = 0, 1
PA_KV_AS_DTYPE, PA_KV_FP8_E4M3, PA_KV_INT4 = 0, 1, 2
PA_ROPE_HALF, PA_ROPE_INTERLEAVED = 0, 1
PA_DEVERR_BLOCK_INDEX, PA_DEVERR_SEQ_LEN, PA_DEVERR_COPY = 1, 2, 4
PA_FLAG_DETERMINISTIC = 1
PA_WORKSPACE_HEADER_BYTES = 8448
PA_NOALLOC_SCRATCH_BYTES = 32 << 20
MAX_GQA_GROUP = 16

# Every symbol include/pa.h declares, with its ctypes signature.
_c = ctypes
SIGNATURES = {
    "pa_decode_workspace_bytes": (_c.c_size_t, [_c.c_int] * 5),
    "pa_decode_ex_workspace_bytes": (_c.c_size_t, [_c.c_void_p]),
    "pa_decode": (_c.c_int, [_c.c_void_p] * 6 + [_c.c_int] * 8 +
                  [_c.c_float, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "pa_decode_ex": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "pa_decode_noalloc": (_c.c_int, [_c.c_void_p] * 6 + [_c.c_int] * 8 +
                          [_c.c_float, _c.c_int, _c.c_void_p]),
    "pa_decode_plan": (_c.c_int, [_c.c_void_p, _c.c_int, _c.c_void_p, _c.c_void_p]),
    "pa_decode_kernel_count": (_c.c_int, [_c.c_void_p, _c.c_void_p]),
    "pa_append": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "pa_gather": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "pa_rope_turns": (_c.c_int, [_c.c_int, _c.c_double, _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "pa_workspace_init": (_c.c_int, [_c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "pa_read_device_errors": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "pa_set_device": (_c.c_int, [_c.c_int]),
    "pa_status_string": (_c.c_char_p, [_c.c_int]),
    "pa_version": (_c.c_char_p, []),
}


class DecodeArgs(ctypes.Structure):
    """Mirror of pa_decode_args (include/pa.h)."""
    _fields_ = [
        ("q", _c.c_void_p), ("k_cache", _c.c_void_p), ("v_cache", _c.c_void_p),
        ("block_tables", _c.c_void_p), ("seq_lens", _c.c_void_p), ("out", _c.c_void_p),
        ("B", _c.c_int32), ("Hq", _c.c_int32), ("Hkv", _c.c_int32), ("D", _c.c_int32),
        ("block_size", _c.c_int32), ("num_blocks", _c.c_int32),
        ("max_blocks_per_seq", _c.c_int32), ("max_seq_len", _c.c_int32),
        ("scale", _c.c_float), ("dtype", _c.c_int32), ("splits", _c.c_int32),
        ("window", _c.c_int32), ("kv_dtype", _c.c_int32),
        ("k_scale", _c.c_float), ("v_scale", _c.c_float), ("q_len", _c.c_int32),
        ("flags", _c.c_uint32), ("total_tokens", _c.c_int64),
    ]


class AppendArgs(ctypes.Structure):
    """Mirror of pa_append_args (include/pa.h)."""
    _fields_ = [
        ("q", _c.c_void_p), ("q_out", _c.c_void_p), ("k", _c.c_void_p), ("v", _c.c_void_p),
        ("k_cache", _c.c_void_p), ("v_cache", _c.c_void_p), ("block_tables", _c.c_void_p),
        ("seq_lens", _c.c_void_p), ("starts", _c.c_void_p), ("rope_turns", _c.c_void_p),
        ("q_stride", _c.c_int64), ("k_stride", _c.c_int64), ("v_stride", _c.c_int64),
        ("B", _c.c_int32), ("rows", _c.c_int32), ("Hq", _c.c_int32), ("Hkv", _c.c_int32),
        ("D", _c.c_int32), ("block_size", _c.c_int32), ("num_blocks", _c.c_int32),
        ("max_blocks_per_seq", _c.c_int32), ("dtype", _c.c_int32), ("kv_dtype", _c.c_int32),
        ("k_scale", _c.c_float), ("v_scale", _c.c_float), ("rot_dim", _c.c_int32),
        ("rope_layout", _c.c_int32), ("rope_amplitude", _c.c_float),
    ]


class GatherArgs(ctypes.Structure):
    """Mirror of pa_gather_args (include/pa.h)."""
    _fields_ = [
        ("k_cache", _c.c_void_p), ("v_cache", _c.c_void_p), ("block_tables", _c.c_void_p),
        ("seq_lens", _c.c_void_p), ("starts", _c.c_void_p), ("k_out", _c.c_void_p),
        ("v_out", _c.c_void_p), ("B", _c.c_int32), ("rows", _c.c_int32), ("Hkv", _c.c_int32),
        ("D", _c.c_int32), ("block_size", _c.c_int32), ("num_blocks", _c.c_int32),
        ("max_blocks_per_seq", _c.c_int32), ("dtype", _c.c_int32), ("kv_dtype", _c.c_int32),
        ("k_scale", _c.c_float), ("v_scale", _c.c_float),
    ]


class RopeScaling(ctypes.Structure):
    """Mirror of pa_rope_scaling (include/pa.h)."""
    _fields_ = [("kind", _c.c_int32), ("original_max", _c.c_int32), ("factor", _c.c_double),
                ("slow", _c.c_double), ("fast", _c.c_double)]


class PAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = status_string(code) if _lib is not None else str(code)
        super().__init__(f"{where}: {msg} (status {code})")


_lib = None
_native = None  # the module of csrc/binding.cpp
_lib_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load libpa.so and the binding's module (built in-tree). Raises if one is missing: there
    is no fallback."""
    global _lib, _native
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m paged_kv_attention_pa_gb300.build`"
                    " (the decode path has no CPU fallback)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            from . import _binding
            _native = _binding
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().pa_status_string(int(code)).decode()


def version() -> str:
    return load().pa_version().decode()


_DT = {torch.float16: PA_F16, torch.bfloat16: PA_BF16}


def _ensure_device(lib, index: int):
    """Make a device current, for the library as for torch. (The calls below change it for
    their own duration only.)"""
    rc = lib.pa_set_device(index)
    if rc != PA_OK:
        raise PAError(rc, "pa_set_device")


def _device_of(t):
    """Context in which t's device is the current one."""
    return torch.cuda.device(t.device.index if t.is_cuda else -1)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: int, stream) -> int:
    """cudaStream_t of the given stream or the device's current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream_handle(torch.device("cuda", device), stream)


def _stream_handle(device: torch.device, stream) -> int:
    s = torch.cuda.current_stream(device) if stream is None else stream
    return int(s.cuda_stream)


def int4_row_bytes(D: int) -> int:
    """Bytes of one row (token and KV head) of a 4-bit cache: 5 bits per element."""
    return D // 8 * 5


def _cache_shape(k_cache, v_cache, dtype):
    """(kv_dtype, num_blocks, block_size, Hkv, D) of a pair of caches: [num_blocks,
    block_size, Hkv, D] in the q dtype or float8_e4m3fn, or 4 bits as uint8
    [num_blocks, Hkv, block_size, int4_row_bytes(D)]."""
    shape, cd = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be four-dimensional and of one shape")
    if v_cache.dtype != cd:
        raise TypeError("k_cache and v_cache must have one dtype")
    if cd == dtype:
        return (PA_KV_AS_DTYPE, *shape)
    if cd == torch.float8_e4m3fn:
        return (PA_KV_FP8_E4M3, *shape)
    if cd != torch.uint8:
        raise TypeError("the caches must both have the 16-bit dtype of the call, or both be "
                        "float8_e4m3fn, or both uint8 (4-bit rows)")
    nb, hkv, bs, row = shape
    if row % 5 != 0:
        raise ValueError("a 4-bit cache row has int4_row_bytes(D) bytes (80 or 160)")
    return PA_KV_INT4, nb, bs, hkv, row // 5 * 8


def make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale: float,
              max_seq_len: Optional[int] = None, splits: int = 0, window: int = 0,
              k_scale: float = 1.0, v_scale: float = 1.0,
              deterministic: bool = False, total_tokens: int = 0) -> DecodeArgs:
    """Check shapes / dtypes / devices and fill a pa_decode_args. q is [B, Hq, D], or
    [B, R, Hq, D] for R causal query rows per sequence."""
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, Hq, D] or [B, R, Hq, D]")
    if q.dim() == 4:
        B, R, Hq, D = q.shape
    else:
        (B, Hq, D), R = q.shape, 1
    if q.dtype not in _DT or out.dtype != q.dtype:
        raise TypeError("q and out must be float16 or bfloat16")
    kv, nb, bs, Hkv, Dk = _cache_shape(k_cache, v_cache, q.dtype)
    if Dk != D:
        raise ValueError("k_cache / v_cache / q shapes disagree")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("block_tables", block_tables), ("seq_lens", seq_lens), ("out", out)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    a = DecodeArgs()
    a.q, a.k_cache, a.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    a.block_tables, a.seq_lens, a.out = block_tables.data_ptr(), seq_lens.data_ptr(), out.data_ptr()
    a.B, a.Hq, a.Hkv, a.D = B, Hq, Hkv, D
    a.block_size, a.num_blocks = bs, nb
    a.max_blocks_per_seq = block_tables.shape[1]
    a.max_seq_len = 0 if max_seq_len is None else int(max_seq_len)
    a.scale = float(scale)
    a.dtype = _DT[q.dtype]
    a.splits = int(splits)
    a.window = int(window)
    a.q_len = R
    a.kv_dtype = kv
    a.k_scale, a.v_scale = (1.0, 1.0) if kv == PA_KV_AS_DTYPE else (float(k_scale), float(v_scale))
    a.flags = PA_FLAG_DETERMINISTIC if deterministic else 0
    a.total_tokens = int(total_tokens)
    return a


# One workspace per (device, stream), and per capture one of each stream that takes part in it;
# grown on demand, zero-filled when made. A captured call never uses the workspace of calls
# outside its graph: graphs, and calls beside them, may run at the same time. Made during a
# capture it lies in the graph's own memory and is zeroed once in every replay. Workspaces that
# were outgrown stay allocated: calls before may have left error bits in them.
_workspaces = {}
_captured = {}  # (device, stream) -> (id of its last capture, that capture's workspace)
_outgrown = []


def _capture_of(stream_handle: int) -> int:
    """The id of the capture that a stream takes part in, 0 outside one."""
    return _native.capture_id(stream_handle)


def _kept(key, capture: int) -> Optional[torch.Tensor]:
    """The workspace that a (device, stream) has, in a capture that capture's."""
    if not capture:
        return _workspaces.get(key)
    held = _captured.get(key)
    return held[1] if held is not None and held[0] == capture else None


def _default_workspace(dev: int, stream_handle: int) -> Optional[torch.Tensor]:
    return _kept((dev, stream_handle), _capture_of(stream_handle)) if dev >= 0 else None


def _workspace(need: int, device: torch.device, stream_handle: int, stream=None) -> torch.Tensor:
    key, capture = (device.index, stream_handle), _capture_of(stream_handle)
    ws = _kept(key, capture)
    if ws is not None and ws.numel() >= need:
        return ws
    if ws is not None:
        need = max(need, 2 * ws.numel())
    with torch.cuda.stream(stream):  # zeroed in the order of the call's stream
        new = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=device)
    if ws is not None:
        new.outgrown = ws  # its error word is read with the new one's
    if capture:
        _captured[key] = (capture, new)
        return new
    if ws is not None:
        _outgrown.append(ws)
    _workspaces[key] = new
    return new


def workspace_for(args: DecodeArgs, device: torch.device, stream_handle: int,
                  stream=None) -> torch.Tensor:
    with torch.cuda.device(device):  # the plan follows its number of SMs
        need = load().pa_decode_ex_workspace_bytes(ctypes.byref(args))
    if need == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_decode_ex_workspace_bytes")
    return _workspace(need, device, stream_handle, stream)


def _call_on(t: torch.Tensor, stream):
    """(device index, stream handle, stream) of a call on t's device; -1, 0 and None for a CPU
    tensor, which the call then refuses."""
    if _lib is None:
        load()
    dev = t.get_device()
    if dev < 0:
        return dev, 0, None
    sh = _stream_of(dev, stream)
    if stream is not None and not isinstance(stream, torch.Stream):  # another library's
        stream = torch.cuda.ExternalStream(sh, device=dev)
    return dev, sh, stream


def _rows_workspace(t: torch.Tensor, dev: int, sh: int, stream) -> Optional[torch.Tensor]:
    """The workspace whose error word append and gather use: any of the stream's."""
    ws = _default_workspace(dev, sh)
    if ws is None and dev >= 0:
        ws = _workspace(PA_WORKSPACE_HEADER_BYTES, t.device, sh, stream)
    return ws


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
           out: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
           splits: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
           window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
           deterministic: bool = False, total_tokens: int = 0) -> torch.Tensor:
    """out[b, h] = softmax(scale * q[b,h] . K_b^T) V_b over the paged context of sequence b.

    q [B, Hq, D]; k_cache, v_cache [num_blocks, block_size, Hkv, D]; block_tables
    [B, max_blocks] int32; seq_lens [B] int32; all on one CUDA device. max_seq_len
    bounds seq_lens (pass it: it sets the split plan; None means the table's
    capacity). splits > 0 forces at most that many context splits. window > 0
    attends to the last `window` tokens only. float8_e4m3fn caches are read as
    stored value * k_scale / v_scale, and so are 4-bit caches, uint8 [num_blocks, Hkv,
    block_size, int4_row_bytes(D)] as append() writes them. deterministic=True keeps fixed context splits, so
    that repeated calls are bitwise identical (by default the splits of a long context
    share out its tail as they finish, and the last bit may vary from call to call).
    total_tokens, the sum of seq_lens when the caller knows it on the host, helps the
    split plan for batches of mixed lengths. Asynchronous on the current (or given)
    stream. Without `workspace` the call uses the one kept for its device and stream; captured
    calls use one that belongs to their graph (see default_workspace).
    """
    dev, sh, stream = _call_on(q, stream)
    ws = workspace if workspace is not None else _default_workspace(dev, sh)
    rc, out = _native.decode(q, k_cache, v_cache, block_tables, seq_lens, scale, out, max_seq_len,
                             splits, window, k_scale, v_scale, deterministic, total_tokens, ws, sh,
                             stream)
    if rc == PA_ERR_WORKSPACE and workspace is None:  # none yet, or too small: nothing was launched
        ws = workspace_for(make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale,
                                     max_seq_len, splits, window, k_scale, v_scale, deterministic,
                                     total_tokens), q.device, sh, stream)
        rc, out = _native.decode(q, k_cache, v_cache, block_tables, seq_lens, scale, out,
                                 max_seq_len, splits, window, k_scale, v_scale, deterministic,
                                 total_tokens, ws, sh, stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_ex")
    return out


def _only_plain(q, k_cache, v_cache):
    """Refuse what pa_decode and pa_decode_noalloc have no argument for: other caches than of
    q's dtype, and several query rows."""
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError("the caches must have q's dtype here: fp8 and 4-bit caches are for decode()")
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D] here: several query rows are for decode()")


def decode_plain(q, k_cache, v_cache, block_tables, seq_lens, scale, out=None,
                 max_seq_len: Optional[int] = None, workspace=None, stream=None):
    """The same operation through pa_decode, the plain positional entry point: caches of q's
    dtype and one query row per sequence."""
    lib = load()
    _only_plain(q, k_cache, v_cache)
    if out is None:
        out = torch.empty_like(q)
    args = make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, 0)
    sh = _stream_handle(q.device, stream)
    ws = workspace if workspace is not None else workspace_for(args, q.device, sh, stream)
    with _device_of(q):
        rc = lib.pa_decode(args.q, args.k_cache, args.v_cache, args.block_tables, args.seq_lens,
                           args.out, args.B, args.Hq, args.Hkv, args.D, args.block_size,
                           args.num_blocks, args.max_blocks_per_seq, args.max_seq_len,
                           args.scale, args.dtype, ws.data_ptr(), ws.numel(), sh)
    if rc != PA_OK:
        raise PAError(rc, "pa_decode")
    return out


def decode_noalloc(q, k_cache, v_cache, block_tables, seq_lens, scale, out=None,
                   max_seq_len: Optional[int] = None, stream=None):
    """The same operation through pa_decode_noalloc: no workspace, no allocation by
    the library (the split partials live in a fixed device array of the library,
    shared by all such calls on a device; see include/pa.h for the limit). Caches of q's
    dtype and one query row per sequence."""
    lib = load()
    _only_plain(q, k_cache, v_cache)
    if out is None:
        out = torch.empty_like(q)
    args = make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, 0)
    sh = _stream_handle(q.device, stream)
    with _device_of(q):
        rc = lib.pa_decode_noalloc(args.q, args.k_cache, args.v_cache, args.block_tables,
                                   args.seq_lens, args.out, args.B, args.Hq, args.Hkv, args.D,
                                   args.block_size, args.num_blocks, args.max_blocks_per_seq,
                                   args.max_seq_len, args.scale, args.dtype, sh)
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_noalloc")
    return out


class Rope(NamedTuple):
    """Rotary positions: `turns` is int64 [rot_dim / 2] on the device, the angle of each pair
    per token as a fraction of a turn in units of 2^-64 (see include/pa.h)."""
    turns: torch.Tensor
    interleaved: bool = False
    amplitude: float = 1.0


_NO_ROPE = (None, False, 1.0)
_ROPE_KINDS = {"linear": 1, "ntk": 2, "yarn": 3, "banded": 4}


def rope(rot_dim: int, base: float = 10000.0, interleaved: bool = False,
         scaling: Optional[str] = None, factor: float = 1.0, original_max: int = 0,
         slow: float = 1.0, fast: float = 32.0, device="cuda") -> Rope:
    """Rotary positions of the first rot_dim elements of a head, with frequencies
    base^(-2i / rot_dim), scaled for long contexts by "linear", "ntk", "yarn" or "banded"
    (include/pa.h, pa_rope_kind). interleaved: pairs (2i, 2i + 1) instead of
    (i, i + rot_dim / 2). Made once and kept."""
    lib = load()
    if scaling is not None and scaling not in _ROPE_KINDS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_KINDS)}")
    turns = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.int64)
    amp = ctypes.c_float(1.0)
    s = RopeScaling(_ROPE_KINDS.get(scaling, 0), int(original_max), float(factor), float(slow),
                    float(fast))
    rc = lib.pa_rope_turns(int(rot_dim), float(base), ctypes.byref(s), turns.data_ptr() or None,
                           ctypes.byref(amp))
    if rc != PA_OK:
        raise PAError(rc, "pa_rope_turns")
    return Rope(turns.to(device), bool(interleaved), amp.value)


def append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, seq_lens: torch.Tensor,
           q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
           starts: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
           k_scale: float = 1.0, v_scale: float = 1.0,
           workspace: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Write the keys (rotated) and values of new tokens into a paged cache, and rotate the
    queries of the same tokens; returns the rotated queries (None without q).

    k, v [B, Hkv, D], or [B, R, Hkv, D] for R new tokens per sequence, or [rows, Hkv, D] packed
    with starts [B + 1] int32 (rows starts[b] to starts[b + 1] - 1 belong to sequence b; others
    are padding). q likewise with Hq heads. They may be slices of one projection: the heads of
    a row contiguous, the rows evenly spaced. seq_lens [B] counts the new tokens: token i of n
    has position seq_lens[b] - n + i and lies where block_tables puts it. The caches are as in
    decode(): 16-bit, float8_e4m3fn or 4-bit uint8; the last two hold value / k_scale
    (v_scale). q_out must be contiguous and may be q itself when that is contiguous.
    Asynchronous on the current (or given) stream.
    """
    dev, sh, stream = _call_on(k_cache, stream)
    turns, interleaved, amplitude = _NO_ROPE if rope is None else rope
    ws = workspace if workspace is not None else _rows_workspace(k_cache, dev, sh, stream)
    rc, rotated = _native.append(k, v, k_cache, v_cache, block_tables, seq_lens, q, q_out, starts,
                                 turns, interleaved, amplitude, k_scale, v_scale, ws, sh, stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_append")
    return rotated


def gather(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
           seq_lens: torch.Tensor, rows: int, starts: Optional[torch.Tensor] = None,
           dtype: Optional[torch.dtype] = None, k_out: Optional[torch.Tensor] = None,
           v_out: Optional[torch.Tensor] = None, k_scale: float = 1.0, v_scale: float = 1.0,
           workspace: Optional[torch.Tensor] = None,
           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Read the last tokens of each sequence back from a paged cache, contiguous and in 16
    bits: (k, v) [B, rows, Hkv, D], the last `rows` tokens of every sequence, or with starts
    [B + 1] int32 packed [rows, Hkv, D], of which rows starts[b] to starts[b + 1] - 1 are the
    last tokens of sequence b and others are left alone (uninitialised in tensors made here).
    Keys stay rotated. dtype is that of the rows (float16 or bfloat16; needed for fp8 and 4-bit
    caches, whose values are multiplied by k_scale, v_scale). A row without a token is zero.
    """
    dev, sh, stream = _call_on(k_cache, stream)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else k_cache.dtype
    code = _DT.get(dtype)
    if code is None:
        raise TypeError("dtype must be float16 or bfloat16")
    ws = workspace if workspace is not None else _rows_workspace(k_cache, dev, sh, stream)
    rc, k, v = _native.gather(k_cache, v_cache, block_tables, seq_lens, rows, starts, code, k_out,
                              v_out, k_scale, v_scale, ws, sh, stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_gather")
    return k, v


def plan(B: int, Hq: int, Hkv: int, D: int, block_size: int, max_seq_len: int,
         splits: int = 0, sm_count: int = 0, window: int = 0,
         kv_fp8: bool = False, total_tokens: int = 0, kv_int4: bool = False,
         rows: int = 1) -> Tuple[int, int]:
    """(splits, tokens per split) the library would launch with. sm_count <= 0 asks
    the current device; a positive sm_count needs no GPU. kv_fp8, kv_int4: FP8 E4M3 and
    4-bit caches (their warp tile is 32 tokens, so splits are multiples of 32). rows: query rows
    per sequence (4-bit plans depend on them)."""
    lib = load()
    a = DecodeArgs()
    a.B, a.Hq, a.Hkv, a.D = B, Hq, Hkv, D
    a.block_size, a.num_blocks = block_size, 1
    a.max_blocks_per_seq = max(1, -(-max_seq_len // block_size))
    a.max_seq_len = max_seq_len
    a.dtype = PA_BF16
    a.splits = splits
    a.window = window
    a.q_len = rows
    if kv_fp8 or kv_int4:
        a.kv_dtype, a.k_scale, a.v_scale = PA_KV_INT4 if kv_int4 else PA_KV_FP8_E4M3, 1.0, 1.0
    a.total_tokens = int(total_tokens)
    S, P = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib.pa_decode_plan(ctypes.byref(a), int(sm_count), ctypes.byref(S), ctypes.byref(P))
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_plan")
    return S.value, P.value


def kernel_count(q, k_cache, v_cache, block_tables, seq_lens, scale, max_seq_len=None,
                 splits: int = 0, window: int = 0, total_tokens: int = 0) -> int:
    """Kernels one decode call with these tensors launches on their device (1, or 2
    with a merge grid; 0 for an empty batch). Nothing is launched."""
    lib = load()
    out = q  # only its shape and dtype are read
    args = make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len,
                     splits, window, total_tokens=total_tokens)
    n = ctypes.c_int(-1)
    with _device_of(q):
        rc = lib.pa_decode_kernel_count(ctypes.byref(args), ctypes.byref(n))
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_kernel_count")
    return n.value


def read_device_errors(workspace: torch.Tensor, stream=None) -> int:
    """Wait for the stream, return and clear the PA_DEVERR_* bits of a workspace (and, of a
    default one, those of the smaller ones that it took the place of)."""
    lib = load()
    sh = _stream_handle(workspace.device, stream)
    found = 0
    while workspace is not None:
        flags = ctypes.c_uint32(0)
        with _device_of(workspace):
            rc = lib.pa_read_device_errors(workspace.data_ptr(), sh, ctypes.byref(flags))
        if rc != PA_OK:
            raise PAError(rc, "pa_read_device_errors")
        found |= flags.value
        workspace = getattr(workspace, "outgrown", None)
    return found


def default_workspace(device=None, stream=None) -> Optional[torch.Tensor]:
    """The workspace that calls without one use on this device and stream, if they had any. In
    a capture it is the graph's: taken there, it holds the error bits of the graph's last
    replay."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    load()
    return _default_workspace(dev.index, _stream_handle(dev, stream))
