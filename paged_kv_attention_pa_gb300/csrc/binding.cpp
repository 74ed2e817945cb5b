// CPython module with the hot calls of the Python binding: it checks tensors and fills the
// argument structures of pa.h from them. The Python functions around it (see __init__.py)
// document the calls and find the stream and the workspace. Checked and filled in Python a
// call costs 13 to 29 us of host time, longer than a small call's kernels run.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>
#include <optional>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"
#include "pa_internal.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A refused argument: the Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw Refused{};
}
[[noreturn]] void refuse_value(const char* what) { refuse(PyExc_ValueError, what); }
[[noreturn]] void refuse_type(const char* what) { refuse(PyExc_TypeError, what); }

const Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) refuse_type("a torch.Tensor is needed");
  return THPVariable_Unpack(o);
}
const Tensor* optional_tensor(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

int64_t integer(PyObject* o) {  // int(o)
  PyObject* n = PyLong_Check(o) ? Py_NewRef(o) : PyNumber_Long(o);
  if (!n) throw Refused{};
  const long long v = PyLong_AsLongLong(n);
  Py_DECREF(n);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse_value("an argument is out of range");
  return (int32_t)v;
}
int32_t to32(int64_t v) {
  if (v > INT32_MAX) refuse_value("a tensor is too large");
  return (int32_t)v;
}
float number(PyObject* o) {  // float(o)
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

int dtype_of(ScalarType t) {
  return t == ScalarType::Half ? PA_F16 : t == ScalarType::BFloat16 ? PA_BF16 : -1;
}

struct Cache {
  int32_t kv, num_blocks, block_size, Hkv, D;
};

// Caches are [num_blocks, block_size, Hkv, D] in the call's type or float8_e4m3fn, or 4 bits
// as uint8 [num_blocks, Hkv, block_size, row bytes].
Cache cache_of(const Tensor& k, const Tensor& v, ScalarType type) {
  if (k.dim() != 4 || k.sizes() != v.sizes())
    refuse_value("k_cache and v_cache must be four-dimensional and of one shape");
  const ScalarType t = k.scalar_type();
  if (v.scalar_type() != t) refuse_type("k_cache and v_cache must have one dtype");
  Cache c{PA_KV_AS_DTYPE, to32(k.size(0)), to32(k.size(1)), to32(k.size(2)), to32(k.size(3))};
  if (t == type) return c;
  if (t == ScalarType::Float8_e4m3fn) {
    c.kv = PA_KV_FP8_E4M3;
    return c;
  }
  if (t != ScalarType::Byte)
    refuse_type("the caches must both have the 16-bit dtype of the call, or both be float8_e4m3fn, or "
                "both uint8 (4-bit rows)");
  if (k.size(3) % 5 != 0) refuse_value("a 4-bit cache row has int4_row_bytes(D) bytes (80 or 160)");
  c.kv = PA_KV_INT4;
  c.Hkv = to32(k.size(1));
  c.block_size = to32(k.size(2));
  c.D = to32(k.size(3) / 5 * 8);
  return c;
}

// Every tensor on one CUDA device, and dense.
void on_device(const Tensor& t, int64_t device, bool dense, const char* name) {
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor (no CPU path)", name);
    throw Refused{};
  }
  if (t.get_device() != device) {
    PyErr_Format(PyExc_ValueError, "%s is on another device than the rest of the call", name);
    throw Refused{};
  }
  if (dense && !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    throw Refused{};
  }
}

// block_tables [B, width], seq_lens [B], starts [B + 1] or null; returns B.
int32_t tables_of(const Tensor& bt, const Tensor& sl, const Tensor* starts) {
  if (bt.scalar_type() != ScalarType::Int || sl.scalar_type() != ScalarType::Int ||
      (starts && starts->scalar_type() != ScalarType::Int))
    refuse_type("block_tables, seq_lens and starts must be int32");
  if (sl.dim() != 1 || bt.dim() != 2 || bt.size(0) != sl.size(0) ||
      (starts && (starts->dim() != 1 || starts->size(0) != sl.size(0) + 1)))
    refuse_value("block_tables must be [B, max_blocks], seq_lens [B] and starts [B + 1]");
  return to32(sl.size(0));
}

// Elements between the rows of a [B, H, D], [B, R, H, D] or packed [rows, H, D] tensor, whose
// heads are dense and whose rows are evenly spaced.
int64_t row_stride(const Tensor& t, const char* name) {
  const auto s = t.sizes(), st = t.strides();
  const int d = (int)s.size();
  if (t.numel() == 0) return 0;  // no rows: their spacing says nothing
  if (st[d - 1] != 1 || (s[d - 2] > 1 && st[d - 2] != s[d - 1])) {
    PyErr_Format(PyExc_ValueError, "the heads of a row of %s must be contiguous", name);
    throw Refused{};
  }
  if (d == 3 || s[1] == 1) return s[0] > 1 ? st[0] : s[d - 2] * s[d - 1];
  if (s[0] > 1 && st[0] != s[1] * st[1]) {
    PyErr_Format(PyExc_ValueError, "the rows of %s must be evenly spaced", name);
    throw Refused{};
  }
  return st[1];
}

template <typename T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

struct Workspace {
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, int64_t device) {
    if (const Tensor* t = optional_tensor(o)) {
      on_device(*t, device, true, "workspace");
      at = t->data_ptr();
      bytes = t->nbytes();
    }
  }
};

// The library's own call, made on the tensors' device and without the interpreter's lock.
template <typename Args, typename Fn>
pa_status launch(Fn fn, const Args& a, int64_t device, const Workspace& ws, PyObject* stream) {
  const pa_stream_t s = reinterpret_cast<pa_stream_t>(static_cast<uintptr_t>(integer(stream)));
  const c10::DeviceGuard guard(c10::Device(at::kCUDA, (c10::DeviceIndex)device));
  pa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fn(&a, ws.at, ws.bytes, s);
  Py_END_ALLOW_THREADS;
  return rc;
}

// Outputs that a call makes. With a stream given (a torch.Stream, else None) they are allocated
// in its order, and not reused before the current stream, where they are used next, is done
// with them.
class Outputs {
 public:
  Outputs(PyObject* given, int64_t device) : device_(at::kCUDA, (c10::DeviceIndex)device) {
    if (given == Py_None) return;
    if (number_of(given, "device_index") != device) refuse_value("stream is of another device than the call's tensors");
    stream_.emplace(c10::Stream::UNSAFE, device_, number_of(given, "stream_id"));
  }
  Tensor make(at::IntArrayRef shape, const at::TensorOptions& options) const {
    if (!stream_) return at::empty(shape, options);
    const c10::Stream current = c10::impl::VirtualGuardImpl(at::kCUDA).getStream(device_);
    Tensor t;
    {
      const c10::StreamGuard guard(*stream_);
      t = at::empty(shape, options);
    }
    if (current != *stream_ && t.numel()) t.record_stream(current);
    return t;
  }
  Tensor like(const Tensor& t) const { return make(t.sizes(), t.options().requires_grad(false)); }

 private:
  static int64_t number_of(PyObject* o, const char* name) {
    PyObject* n = PyObject_GetAttrString(o, name);
    if (!n) throw Refused{};
    const long long v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
  }
  c10::Device device_;
  std::optional<c10::Stream> stream_;
};

// decode(q, k_cache, v_cache, block_tables, seq_lens, scale, out, max_seq_len, splits, window,
//        k_scale, v_scale, deterministic, total_tokens, workspace, stream handle, stream or None) -> (status, out)
PyObject* do_decode(PyObject* const* v) {
  const Tensor &q = tensor(v[0]), &kc = tensor(v[1]), &vc = tensor(v[2]), &bt = tensor(v[3]), &sl = tensor(v[4]);
  const int64_t d = q.dim();
  if (d != 3 && d != 4) refuse_value("q must be [B, Hq, D] or [B, R, Hq, D]");
  const Tensor* given = optional_tensor(v[6]);
  pa_decode_args a{};
  const int dt = dtype_of(q.scalar_type());
  if (dt < 0 || (given && given->scalar_type() != q.scalar_type()))
    refuse_type("q and out must be float16 or bfloat16");
  const Cache c = cache_of(kc, vc, q.scalar_type());
  if (c.D != q.size(d - 1)) refuse_value("k_cache / v_cache / q shapes disagree");
  if (bt.scalar_type() != ScalarType::Int || sl.scalar_type() != ScalarType::Int)
    refuse_type("block_tables and seq_lens must be int32");
  if (bt.dim() != 2 || bt.size(0) != q.size(0) || sl.dim() != 1 || sl.size(0) != q.size(0))
    refuse_value("block_tables must be [B, max_blocks] and seq_lens [B]");
  if (given && given->sizes() != q.sizes()) refuse_value("out must have q's shape");
  a.max_seq_len = v[7] == Py_None ? 0 : integer32(v[7]);
  a.scale = number(v[5]);
  a.splits = integer32(v[8]);
  a.window = integer32(v[9]);
  a.k_scale = c.kv == PA_KV_AS_DTYPE ? 1.f : number(v[10]);
  a.v_scale = c.kv == PA_KV_AS_DTYPE ? 1.f : number(v[11]);
  a.flags = truth(v[12]) ? PA_FLAG_DETERMINISTIC : 0u;
  a.total_tokens = integer(v[13]);
  const int64_t dev = q.get_device();
  on_device(q, dev, true, "q");
  on_device(kc, dev, true, "k_cache");
  on_device(vc, dev, true, "v_cache");
  on_device(bt, dev, true, "block_tables");
  on_device(sl, dev, true, "seq_lens");
  if (given) on_device(*given, dev, true, "out");
  a.B = to32(q.size(0));
  a.q_len = d == 4 ? to32(q.size(1)) : 1;
  a.Hq = to32(q.size(d - 2));
  a.D = c.D;
  a.Hkv = c.Hkv;
  a.block_size = c.block_size;
  a.num_blocks = c.num_blocks;
  a.max_blocks_per_seq = to32(bt.size(1));
  a.dtype = dt;
  a.kv_dtype = c.kv;
  const Workspace ws(v[14], dev);
  const Outputs outputs(v[16], dev);
  const Tensor out = given ? *given : outputs.like(q);
  a.q = data<void>(q);
  a.k_cache = data<void>(kc);
  a.v_cache = data<void>(vc);
  a.block_tables = data<int32_t>(bt);
  a.seq_lens = data<int32_t>(sl);
  a.out = data<void>(out);
  const pa_status rc = launch(pa_decode_ex, a, dev, ws, v[15]);
  return Py_BuildValue("(iN)", (int)rc, given ? Py_NewRef(v[6]) : THPVariable_Wrap(out));
}

// append(k, v, k_cache, v_cache, block_tables, seq_lens, q, q_out, starts, turns, interleaved,
//        amplitude, k_scale, v_scale, workspace, stream handle, stream or None) -> (status, q_out or None)
PyObject* do_append(PyObject* const* v) {
  const Tensor &k = tensor(v[0]), &val = tensor(v[1]), &kc = tensor(v[2]), &vc = tensor(v[3]), &bt = tensor(v[4]),
               &sl = tensor(v[5]);
  const Tensor *q = optional_tensor(v[6]), *given = optional_tensor(v[7]), *starts = optional_tensor(v[8]),
               *turns = optional_tensor(v[9]);
  const ScalarType type = k.scalar_type();
  pa_append_args a{};
  a.dtype = dtype_of(type);
  if (a.dtype < 0 || val.scalar_type() != type || (q && q->scalar_type() != type))
    refuse_type("q, k and v must be float16 or bfloat16, all the same");
  const Cache c = cache_of(kc, vc, type);
  a.B = tables_of(bt, sl, starts);
  const int64_t d = k.dim();
  if ((d != 3 && (starts || d != 4)) || (!starts && k.size(0) != a.B))
    refuse_value("k must be [B, Hkv, D] or [B, R, Hkv, D], or [rows, Hkv, D] with starts");
  if (val.sizes() != k.sizes() || k.size(d - 2) != c.Hkv || k.size(d - 1) != c.D)
    refuse_value("k and v must have one shape ending in the caches' [Hkv, D]");
  if (q && (q->dim() != d || q->size(0) != k.size(0) || (d == 4 && q->size(1) != k.size(1)) ||
            q->size(d - 1) != c.D))
    refuse_value("q must have k's rows and head_dim");
  if (given && !q) refuse_value("q_out needs q");
  if (given && (given->sizes() != q->sizes() || given->scalar_type() != type))
    refuse_value("q_out must have q's shape and dtype");
  if (turns && (turns->scalar_type() != ScalarType::Long || turns->dim() != 1))
    refuse_type("rope.turns must be int64 [rot_dim / 2]");
  a.k_stride = row_stride(k, "k");
  a.v_stride = row_stride(val, "v");
  if (q) a.q_stride = row_stride(*q, "q");
  const int64_t dev = kc.get_device();
  on_device(kc, dev, true, "k_cache");
  on_device(vc, dev, true, "v_cache");
  on_device(k, dev, false, "k");
  on_device(val, dev, false, "v");
  on_device(bt, dev, true, "block_tables");
  on_device(sl, dev, true, "seq_lens");
  if (q) on_device(*q, dev, false, "q");
  if (given) on_device(*given, dev, true, "q_out");
  if (starts) on_device(*starts, dev, true, "starts");
  if (turns) on_device(*turns, dev, true, "rope.turns");
  a.rows = starts || d == 4 ? to32(k.size(starts ? 0 : 1)) : 1;
  a.Hkv = c.Hkv;
  a.D = c.D;
  a.block_size = c.block_size;
  a.num_blocks = c.num_blocks;
  a.max_blocks_per_seq = to32(bt.size(1));
  a.kv_dtype = c.kv;
  a.k_scale = number(v[12]);
  a.v_scale = number(v[13]);
  a.rope_layout = truth(v[10]) ? PA_ROPE_INTERLEAVED : PA_ROPE_HALF;
  a.rope_amplitude = number(v[11]);
  const Outputs outputs(v[16], dev);
  Tensor out;
  if (q) {
    a.Hq = to32(q->size(d - 2));
    out = given ? *given : outputs.like(*q);
    a.q = data<void>(*q);
    a.q_out = data<void>(out);
  }
  const Workspace ws(v[14], dev);
  a.k = data<void>(k);
  a.v = data<void>(val);
  a.k_cache = data<void>(kc);
  a.v_cache = data<void>(vc);
  a.block_tables = data<int32_t>(bt);
  a.seq_lens = data<int32_t>(sl);
  a.starts = starts ? data<int32_t>(*starts) : nullptr;
  if (turns) {
    a.rope_turns = reinterpret_cast<const uint64_t*>(data<int64_t>(*turns));
    a.rot_dim = to32(2 * turns->size(0));
  }
  const pa_status rc = launch(pa_append, a, dev, ws, v[15]);
  return Py_BuildValue("(iN)", (int)rc,
                       given ? Py_NewRef(v[7]) : q ? THPVariable_Wrap(out) : Py_NewRef(Py_None));
}

// gather(k_cache, v_cache, block_tables, seq_lens, rows, starts, like, k_out, v_out, k_scale,
//        v_scale, workspace, stream handle, stream or None) -> (status, k_out, v_out); like: 0 float16, 1 bfloat16
PyObject* do_gather(PyObject* const* v) {
  const Tensor &kc = tensor(v[0]), &vc = tensor(v[1]), &bt = tensor(v[2]), &sl = tensor(v[3]);
  const Tensor *starts = optional_tensor(v[5]), *kg = optional_tensor(v[7]), *vg = optional_tensor(v[8]);
  pa_gather_args a{};
  a.dtype = integer32(v[6]);
  const ScalarType type = a.dtype == PA_F16 ? ScalarType::Half : ScalarType::BFloat16;
  const Cache c = cache_of(kc, vc, type);
  a.B = tables_of(bt, sl, starts);
  a.rows = integer32(v[4]);
  if (a.rows < 0) refuse_value("rows must not be negative");
  const int64_t dims[4] = {a.B, a.rows, c.Hkv, c.D};
  const at::IntArrayRef shape(dims + (starts ? 1 : 0), starts ? 3 : 4);
  for (const Tensor* t : {kg, vg})
    if (t && (t->sizes() != shape || t->scalar_type() != type))
      refuse_value("k_out and v_out must have the call's dtype and [B, rows, Hkv, D], or [rows, Hkv, D] with starts");
  const int64_t dev = kc.get_device();
  on_device(kc, dev, true, "k_cache");
  on_device(vc, dev, true, "v_cache");
  on_device(bt, dev, true, "block_tables");
  on_device(sl, dev, true, "seq_lens");
  if (starts) on_device(*starts, dev, true, "starts");
  if (kg) on_device(*kg, dev, true, "k_out");
  if (vg) on_device(*vg, dev, true, "v_out");
  a.Hkv = c.Hkv;
  a.D = c.D;
  a.block_size = c.block_size;
  a.num_blocks = c.num_blocks;
  a.max_blocks_per_seq = to32(bt.size(1));
  a.kv_dtype = c.kv;
  a.k_scale = number(v[9]);
  a.v_scale = number(v[10]);
  const Workspace ws(v[11], dev);
  const Outputs outputs(v[13], dev);
  const auto options = kc.options().dtype(type).requires_grad(false);
  const Tensor ko = kg ? *kg : outputs.make(shape, options), vo = vg ? *vg : outputs.make(shape, options);
  a.k_cache = data<void>(kc);
  a.v_cache = data<void>(vc);
  a.block_tables = data<int32_t>(bt);
  a.seq_lens = data<int32_t>(sl);
  a.starts = starts ? data<int32_t>(*starts) : nullptr;
  a.k_out = data<void>(ko);
  a.v_out = data<void>(vo);
  const pa_status rc = launch(pa_gather, a, dev, ws, v[12]);
  return Py_BuildValue("(iNN)", (int)rc, kg ? Py_NewRef(v[7]) : THPVariable_Wrap(ko),
                       vg ? Py_NewRef(v[8]) : THPVariable_Wrap(vo));
}

// capture_id(stream) -> id of the capture that the stream takes part in, 0 outside one
PyObject* do_capture_id(PyObject* const* v) {
  return PyLong_FromUnsignedLongLong(
      pa_stream_capture_id(reinterpret_cast<pa_stream_t>(static_cast<uintptr_t>(integer(v[0])))));
}

// A call with its exceptions turned into Python's.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (...) {  // torch's own (a failed allocation is torch.OutOfMemoryError)
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<do_decode, 17>("decode"), method<do_append, 17>("append"),
                          method<do_gather, 14>("gather"),
                          method<do_capture_id, 1>("capture_id"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
