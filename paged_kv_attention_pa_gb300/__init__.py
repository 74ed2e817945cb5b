"""Python binding of libpa.so: single-query paged-attention decode on GB300, and the
rows of its paged cache (append with rotary positions, gather).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/pa.h. PyTorch provides device
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
import struct
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
_lib_lock = threading.Lock()
_tls = threading.local()


def load(path: str = LIB_PATH):
    """Load libpa.so (built in-tree). Raises if it is missing: there is no fallback."""
    global _lib
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
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().pa_status_string(int(code)).decode()


def version() -> str:
    return load().pa_version().decode()


_DT = {torch.float16: PA_F16, torch.bfloat16: PA_BF16}


def _ensure_device(lib, index: int):
    if getattr(_tls, "device", None) != index:
        rc = lib.pa_set_device(index)
        if rc != PA_OK:
            raise PAError(rc, "pa_set_device")
        _tls.device = index


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


# The argument structures are packed in one go: setting their fields one by one costs a
# call several microseconds.
_DECODE = struct.Struct("<6Q8if4i2fiI4xq")
_APPEND = struct.Struct("<10Q3q10i2f2if4x")
_GATHER = struct.Struct("<7Q9i2f4x")
assert _DECODE.size == ctypes.sizeof(DecodeArgs) and _APPEND.size == ctypes.sizeof(AppendArgs) \
    and _GATHER.size == ctypes.sizeof(GatherArgs)


def _pack(layout, *values) -> bytes:
    try:
        return layout.pack(*values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is out of range: {e}") from None


def _where(first, tensors) -> int:
    """The device index all (name, tensor) pairs share with `first`; contiguous tensors only."""
    dev = first.get_device()
    for name, t in tensors:
        d = t.get_device()
        if d != dev or d < 0:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
            raise ValueError(f"{name} is on {t.device}, another tensor of the call on {first.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return dev


def _decode_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, splits,
                 window, k_scale, v_scale, deterministic, total_tokens):
    """Check shapes / dtypes / devices; the packed pa_decode_args and the device index."""
    shape = q.shape
    if len(shape) == 3:
        (B, Hq, D), R = shape, 1
    elif len(shape) == 4:
        B, R, Hq, D = shape
    else:
        raise ValueError("q must be [B, Hq, D] or [B, R, Hq, D]")
    dtype = _DT.get(q.dtype)
    if dtype is None or out.dtype != q.dtype:
        raise TypeError("q and out must be float16 or bfloat16")
    kv, nb, bs, Hkv, Dk = _cache_shape(k_cache, v_cache, q.dtype)
    if Dk != D:
        raise ValueError("k_cache / v_cache / q shapes disagree")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_tables and seq_lens must be int32")
    bts = block_tables.shape
    if len(bts) != 2 or bts[0] != B or seq_lens.shape != (B,):
        raise ValueError("block_tables must be [B, max_blocks] and seq_lens [B]")
    if out.shape != shape:
        raise ValueError("out must have q's shape")
    dev = _where(q, (("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                     ("block_tables", block_tables), ("seq_lens", seq_lens), ("out", out)))
    if kv == PA_KV_AS_DTYPE:
        k_scale = v_scale = 1.0
    return dev, _pack(
        _DECODE, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), out.data_ptr(), B, Hq, Hkv, D, bs, nb, bts[1],
        0 if max_seq_len is None else int(max_seq_len), float(scale), dtype, int(splits),
        int(window), kv, float(k_scale), float(v_scale), R,
        PA_FLAG_DETERMINISTIC if deterministic else 0, int(total_tokens))


def make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale: float,
              max_seq_len: Optional[int] = None, splits: int = 0, window: int = 0,
              k_scale: float = 1.0, v_scale: float = 1.0,
              deterministic: bool = False, total_tokens: int = 0) -> DecodeArgs:
    """Check shapes / dtypes / devices and fill a pa_decode_args. q is [B, Hq, D], or
    [B, R, Hq, D] for R causal query rows per sequence."""
    return DecodeArgs.from_buffer_copy(_decode_args(
        q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, splits, window,
        k_scale, v_scale, deterministic, total_tokens)[1])


# One workspace per (device, stream); grown on demand, zero-filled when made. Workspaces that
# were outgrown stay allocated: a captured graph may still write to them when it is replayed.
# Graphs that may be replayed at the same time need workspaces of their own.
_workspaces = {}
_outgrown = []


def _workspace(need: int, device: torch.device, stream_handle: int) -> torch.Tensor:
    key = (device.index, stream_handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        if ws is not None:
            _outgrown.append(ws)
            need = max(need, 2 * ws.numel())
        ws = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def workspace_for(args: DecodeArgs, device: torch.device, stream_handle: int) -> torch.Tensor:
    need = load().pa_decode_ex_workspace_bytes(ctypes.byref(args))
    if need == 0:
        raise PAError(PA_ERR_INVALID_ARG, "pa_decode_ex_workspace_bytes")
    return _workspace(need, device, stream_handle)


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
    stream.
    """
    lib = _lib or load()
    if out is None:
        out = torch.empty_like(q)
    dev, args = _decode_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len,
                             splits, window, k_scale, v_scale, deterministic, total_tokens)
    _ensure_device(lib, dev)
    sh = _stream_of(dev, stream)
    ws = workspace if workspace is not None else _workspaces.get((dev, sh))
    rc = PA_ERR_WORKSPACE if ws is None else lib.pa_decode_ex(args, ws.data_ptr(), ws.numel(), sh)
    if rc == PA_ERR_WORKSPACE and workspace is None:  # none yet, or too small: nothing was launched
        ws = workspace_for(DecodeArgs.from_buffer_copy(args), q.device, sh)
        rc = lib.pa_decode_ex(args, ws.data_ptr(), ws.numel(), sh)
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_ex")
    return out


def decode_plain(q, k_cache, v_cache, block_tables, seq_lens, scale, out=None,
                 max_seq_len: Optional[int] = None, workspace=None, stream=None):
    """The same operation through pa_decode, the plain positional entry point."""
    lib = load()
    if out is None:
        out = torch.empty_like(q)
    args = make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, 0)
    _ensure_device(lib, q.device.index)
    sh = _stream_handle(q.device, stream)
    ws = workspace if workspace is not None else workspace_for(args, q.device, sh)
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
    shared by all such calls on a device; see include/pa.h for the limit)."""
    lib = load()
    if out is None:
        out = torch.empty_like(q)
    args = make_args(q, k_cache, v_cache, block_tables, seq_lens, out, scale, max_seq_len, 0)
    _ensure_device(lib, q.device.index)
    sh = _stream_handle(q.device, stream)
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


def _row_stride(name, t, shape) -> int:
    """Elements between the rows of a [B, H, D], [B, R, H, D] or packed [rows, H, D] tensor,
    whose heads are dense and whose rows are evenly spaced."""
    st = t.stride()
    H, D = shape[-2:]
    if (st[-1] != 1 or (H > 1 and st[-2] != D)) and t.numel():
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if len(shape) == 3 or shape[1] == 1:
        return st[0] if shape[0] > 1 else H * D
    if shape[0] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError(f"the rows of {name} must be evenly spaced")
    return st[1]


def _tables(block_tables, seq_lens, starts):
    """(B, table width) of a call's index tensors."""
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or \
            (starts is not None and starts.dtype != torch.int32):
        raise TypeError("block_tables, seq_lens and starts must be int32")
    bts, sls = block_tables.shape, seq_lens.shape
    if len(sls) != 1 or len(bts) != 2 or bts[0] != sls[0] or \
            (starts is not None and starts.shape != (sls[0] + 1,)):
        raise ValueError("block_tables must be [B, max_blocks], seq_lens [B] and starts [B + 1]")
    return bts


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
    lib = _lib or load()
    dtype, shape = _DT.get(k.dtype), k.shape
    if dtype is None or v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise TypeError("q, k and v must be float16 or bfloat16, all the same")
    kv, nb, bs, Hkv, D = _cache_shape(k_cache, v_cache, k.dtype)
    B, width = _tables(block_tables, seq_lens, starts)
    packed = starts is not None
    if len(shape) != 3 and (packed or len(shape) != 4) or (not packed and shape[0] != B):
        raise ValueError("k must be [B, Hkv, D] or [B, R, Hkv, D], or [rows, Hkv, D] with starts")
    if v.shape != shape or shape[-2] != Hkv or shape[-1] != D:
        raise ValueError("k and v must have one shape ending in the caches' [Hkv, D]")
    dev = k.get_device()
    dense = [("k_cache", k_cache), ("v_cache", v_cache), ("block_tables", block_tables),
             ("seq_lens", seq_lens)]
    if k.get_device() != v.get_device() or (q is not None and q.get_device() != dev):
        raise ValueError("q, k and v must be CUDA tensors on one device (no CPU path)")
    qp = qop = Hq = q_stride = 0
    if q is not None:
        qs = q.shape
        if len(qs) != len(shape) or qs[:-2] != shape[:-2] or qs[-1] != D:
            raise ValueError("q must have k's rows and head_dim")
        if q_out is None:
            q_out = torch.empty(qs, dtype=q.dtype, device=q.device)
        elif q_out.shape != qs or q_out.dtype != q.dtype:
            raise ValueError("q_out must have q's shape and dtype")
        q_stride, Hq = _row_stride("q", q, qs), qs[-2]
        qp, qop = q.data_ptr(), q_out.data_ptr()
        dense.append(("q_out", q_out))
    elif q_out is not None:
        raise ValueError("q_out needs q")
    tp = rot = interleaved = 0
    amplitude = 1.0
    if rope is not None:
        turns, interleaved, amplitude = rope
        if turns.dtype != torch.int64 or turns.dim() != 1:
            raise TypeError("rope.turns must be int64 [rot_dim / 2]")
        tp, rot = turns.data_ptr(), 2 * turns.shape[0]
        dense.append(("rope.turns", turns))
    if packed:
        dense.append(("starts", starts))
    _where(k, dense)
    args = _pack(
        _APPEND, qp, qop, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), seq_lens.data_ptr(), starts.data_ptr() if packed else 0, tp,
        q_stride, _row_stride("k", k, shape), _row_stride("v", v, shape), B,
        shape[0] if packed else (1 if len(shape) == 3 else shape[1]), Hq, Hkv, D, bs, nb, width,
        dtype, kv, float(k_scale), float(v_scale), rot,
        PA_ROPE_INTERLEAVED if interleaved else PA_ROPE_HALF, float(amplitude))
    _ensure_device(lib, dev)
    sh = _stream_of(dev, stream)
    ws = workspace if workspace is not None else _workspaces.get((dev, sh))
    if ws is None:
        ws = _workspace(PA_WORKSPACE_HEADER_BYTES, k_cache.device, sh)
    rc = lib.pa_append(args, ws.data_ptr(), ws.numel(), sh)
    if rc != PA_OK:
        raise PAError(rc, "pa_append")
    return q_out


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
    lib = _lib or load()
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else k_cache.dtype
    code = _DT.get(dtype)
    if code is None:
        raise TypeError("dtype must be float16 or bfloat16")
    kv, nb, bs, Hkv, D = _cache_shape(k_cache, v_cache, dtype)
    B, width = _tables(block_tables, seq_lens, starts)
    if rows < 0:
        raise ValueError("rows must not be negative")
    shape = (B, rows, Hkv, D) if starts is None else (rows, Hkv, D)
    dense = [("k_cache", k_cache), ("v_cache", v_cache), ("block_tables", block_tables),
             ("seq_lens", seq_lens)]
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=k_cache.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=k_cache.device)
    if k_out.shape != shape or v_out.shape != shape or k_out.dtype != dtype or v_out.dtype != dtype:
        raise ValueError(f"k_out and v_out must be {dtype} {list(shape)}")
    dense += [("k_out", k_out), ("v_out", v_out)]
    if starts is not None:
        dense.append(("starts", starts))
    dev = _where(k_cache, dense)
    args = _pack(
        _GATHER, k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), starts.data_ptr() if starts is not None else 0, k_out.data_ptr(),
        v_out.data_ptr(), B, rows, Hkv, D, bs, nb, width, code, kv, float(k_scale), float(v_scale))
    _ensure_device(lib, dev)
    sh = _stream_of(dev, stream)
    ws = workspace if workspace is not None else _workspaces.get((dev, sh))
    if ws is None:
        ws = _workspace(PA_WORKSPACE_HEADER_BYTES, k_cache.device, sh)
    rc = lib.pa_gather(args, ws.data_ptr(), ws.numel(), sh)
    if rc != PA_OK:
        raise PAError(rc, "pa_gather")
    return k_out, v_out


def plan(B: int, Hq: int, Hkv: int, D: int, block_size: int, max_seq_len: int,
         splits: int = 0, sm_count: int = 0, window: int = 0,
         kv_fp8: bool = False, total_tokens: int = 0, kv_int4: bool = False) -> Tuple[int, int]:
    """(splits, tokens per split) the library would launch with. sm_count <= 0 asks
    the current device; a positive sm_count needs no GPU. kv_fp8: FP8 E4M3 caches
    (their warp tile is 32 tokens, so splits are multiples of 32). kv_int4: 4-bit caches."""
    lib = load()
    a = DecodeArgs()
    a.B, a.Hq, a.Hkv, a.D = B, Hq, Hkv, D
    a.block_size, a.num_blocks = block_size, 1
    a.max_blocks_per_seq = max(1, -(-max_seq_len // block_size))
    a.max_seq_len = max_seq_len
    a.dtype = PA_BF16
    a.splits = splits
    a.window = window
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
    _ensure_device(lib, q.device.index)
    n = ctypes.c_int(-1)
    rc = lib.pa_decode_kernel_count(ctypes.byref(args), ctypes.byref(n))
    if rc != PA_OK:
        raise PAError(rc, "pa_decode_kernel_count")
    return n.value


def read_device_errors(workspace: torch.Tensor, stream=None) -> int:
    """Wait for the stream, return and clear the PA_DEVERR_* bits of a workspace."""
    lib = load()
    _ensure_device(lib, workspace.device.index)
    flags = ctypes.c_uint32(0)
    rc = lib.pa_read_device_errors(workspace.data_ptr(),
                                   _stream_handle(workspace.device, stream), ctypes.byref(flags))
    if rc != PA_OK:
        raise PAError(rc, "pa_read_device_errors")
    return flags.value


def default_workspace(device=None, stream=None) -> Optional[torch.Tensor]:
    """The workspace decode() used last on this device and stream, if any."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return _workspaces.get((dev.index, _stream_handle(dev, stream)))
