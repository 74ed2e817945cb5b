// Host side of pa_cross and pa_decode_shared: checks, the workspace, tensor maps and the launch.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "pa.h"
#include "pa_attend.h"
#include "pa_launch.h"
#include "pa_params.h"

namespace pa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// What both calls share.
struct Call {
  const void *q, *k_cache, *v_cache;
  const int32_t *block_tables, *seq_lens;
  void* out;
  int64_t q_stride;
  int32_t B, Hq, Hkv, D, block_size, num_blocks, max_blocks, max_seq_len;
  float scale;
  int32_t dtype, kv_dtype;
  float k_scale, v_scale;
  int64_t T, item_rows;  // query rows in all, of the largest segment
};

pa_status check_sizes(const Call& c, int* cap) {
  if (c.B < 0 || c.T < 0 || c.Hq <= 0 || c.Hkv <= 0 || c.D <= 0) return PA_ERR_INVALID_ARG;
  if (c.Hq % c.Hkv != 0 || c.Hq / c.Hkv > PA_MAX_GQA_GROUP) return PA_ERR_INVALID_ARG;
  if (c.D != 128 && c.D != 256) return PA_ERR_UNSUPPORTED;
  if (c.block_size <= 0 || c.num_blocks <= 0 || c.max_blocks <= 0) return PA_ERR_INVALID_ARG;
  if (c.dtype != PA_F16 && c.dtype != PA_BF16) return PA_ERR_INVALID_ARG;
  if (c.kv_dtype == PA_KV_INT4) return PA_ERR_UNSUPPORTED;
  if (c.kv_dtype != PA_KV_AS_DTYPE && c.kv_dtype != PA_KV_FP8_E4M3) return PA_ERR_INVALID_ARG;
  if (c.kv_dtype == PA_KV_FP8_E4M3 &&
      !(c.k_scale > 0.f && c.v_scale > 0.f && c.k_scale < INFINITY && c.v_scale < INFINITY))
    return PA_ERR_INVALID_ARG;
  if (rows_beyond_32_bits(c.num_blocks, c.block_size, c.Hkv)) return PA_ERR_UNSUPPORTED;
  if (c.T > INT_MAX / c.Hq) return PA_ERR_UNSUPPORTED;  // rows of the output
  // a tensor copy's strides are below 2^40 bytes, and all queries lie below 2^62
  if (c.T > 1 && (c.q_stride >= 1ll << 39 || c.q_stride > (INT64_MAX >> 2) / (c.T - 1))) return PA_ERR_UNSUPPORTED;
  const int64_t all = (int64_t)c.max_blocks * c.block_size;
  const int64_t len = c.max_seq_len <= 0 ? all : c.max_seq_len;
  if (len > all || len > INT_MAX - 1024) return PA_ERR_OUT_OF_RANGE;  // 1024: tiles past the end
  *cap = (int)len;
  return PA_OK;
}

struct Layout {
  size_t plan, segments, split, slot_ml, slot_acc, row_ml, row_acc, total;
  int slot_rows;
};
// both: rows may have two contexts
Layout layout_of(const Call& c, int ctas, int segments, bool both) {
  Layout w{};
  const int G = c.Hq / c.Hkv;
  w.slot_rows = (int)std::min<int64_t>(attend_row_tiles(c.D) * (128 / G), std::max<int64_t>(c.item_rows, 1)) * G;
  const size_t slots = (size_t)ctas * 2 * w.slot_rows, rows = both ? (size_t)(2 * c.T * c.Hq) : 0;
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  w.plan = take(2 * 8);
  w.segments = take(both ? (size_t)segments * sizeof(SegmentRecord) : 0);
  w.split = take((size_t)ctas * sizeof(SplitItem));
  w.slot_ml = take(slots * 8);
  w.slot_acc = take(slots * c.D * 4);
  w.row_ml = take(rows * 8);
  w.row_acc = take(rows * c.D * 4);
  w.total = off;
  return w;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static EncodeTiled found = nullptr;
  EncodeTiled f = __atomic_load_n(&found, __ATOMIC_ACQUIRE);
  if (f) return f;
  void* at = nullptr;
  cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &got) != cudaSuccess ||
      got != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeTiled>(at);
  __atomic_store_n(&found, f, __ATOMIC_RELEASE);
  return f;
}

// [rows, heads, D] with `stride` elements between rows; a copy takes `box` rows of `box_heads` heads,
// 64 elements wide (128 bytes, the swizzle's row).
bool make_map(CUtensorMap* map, const Call& c, const void* at, int64_t rows, int64_t stride, int heads, int box,
              int box_heads) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)c.D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t tile[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box}, step[3] = {1, 1, 1};
  return encode(map, c.dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                const_cast<void*>(at), dims, strides, tile, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

pa_status run(const Call& c, AttendParams& p, int cap, void* workspace, size_t bytes, pa_stream_t stream) {
  if (!c.q || !c.k_cache || !c.v_cache || !c.block_tables || !c.seq_lens || !c.out) return PA_ERR_INVALID_ARG;
  if (!aligned16(c.q) || !aligned16(c.k_cache) || !aligned16(c.v_cache) || !aligned16(c.out)) return PA_ERR_INVALID_ARG;
  // rows of out are written while other rows' queries are still read
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(c.q), o0 = reinterpret_cast<uintptr_t>(c.out);
  const uintptr_t row = (uintptr_t)c.Hq * c.D * 2, q1 = q0 + (uintptr_t)(c.T - 1) * c.q_stride * 2 + row;
  if (q0 < o0 + (uintptr_t)c.T * row && o0 < q1) return PA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PA_ERR_WORKSPACE;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const Layout w = layout_of(c, sms, p.B + p.N, p.shared != 0);
  if (bytes < w.total) return PA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = c.q;
  p.out = c.out;
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.block_tables = c.block_tables;
  p.seq_lens = c.seq_lens;
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.plan = reinterpret_cast<long long*>(ws + w.plan);
  p.segments = reinterpret_cast<SegmentRecord*>(ws + w.segments);
  p.split = reinterpret_cast<SplitItem*>(ws + w.split);
  p.slot_ml = reinterpret_cast<float2*>(ws + w.slot_ml);
  p.slot_acc = reinterpret_cast<float*>(ws + w.slot_acc);
  p.row_ml = reinterpret_cast<float2*>(ws + w.row_ml);
  p.row_acc = reinterpret_cast<float*>(ws + w.row_acc);
  p.slot_rows = w.slot_rows;
  p.T = (int)c.T;
  p.Hq = c.Hq;
  p.Hkv = c.Hkv;
  p.G = c.Hq / c.Hkv;
  // r (m G - 2^32) < 2^16 * 16 < 2^32 with m = ceil(2^32 / G): floor(r m / 2^32) = floor(r / G)
  p.g_magic = p.G == 1 ? 0u : (uint32_t)(((1ull << 32) + p.G - 1) / p.G);
  p.tile_tokens = 128 / p.G;
  p.spread_tokens = 32 / p.G;
  p.out_wide = (reinterpret_cast<uintptr_t>(c.out) & 31u) == 0;
  p.block_size = c.block_size;
  p.num_blocks = c.num_blocks;
  p.max_blocks = c.max_blocks;
  p.cap = cap;
  set_block_division(c.block_size, &p.bs_magic, &p.bs_shift);
  p.ctas = sms;
  const bool fp8 = c.kv_dtype == PA_KV_FP8_E4M3;
  p.v_scale = fp8 ? c.v_scale : 1.f;
  // The kernel masks scores before it scales them, so its scale is positive: a negative one negates
  // the queries in the product, and with one that is (or rounds to) zero the smallest normal number
  // gives the same equal weights.
  const double scale = (double)c.scale * 1.4426950408889634 * (fp8 ? (double)c.k_scale : 1.0);
  p.scale_log2 = std::max((float)std::fabs(scale), FLT_MIN);
  p.negate = scale < 0.0;
  // The largest power of two that divides the block size, up to a tile; the swizzle's pattern
  // repeats every eight rows, so smaller ones are staged.
  p.box = std::min(c.block_size & -c.block_size, attend_tile(c.D));
  const AttendLoad load =
      fp8 ? kLoadFp8 : p.box >= 8 && (int64_t)c.num_blocks * c.block_size <= INT_MAX ? kLoadTensor : kLoad16;
  AttendMaps maps{};
  const int64_t q_stride = c.T > 1 ? c.q_stride : (int64_t)c.Hq * c.D;
  if (!make_map(&maps.q, c, c.q, c.T, q_stride, c.Hq, p.tile_tokens, p.G) ||
      !make_map(&maps.q_spread, c, c.q, c.T, q_stride, c.Hq, p.spread_tokens, p.G))
    return PA_ERR_CUDA;
  if (load == kLoadTensor) {
    const int64_t tokens = (int64_t)c.num_blocks * c.block_size, stride = (int64_t)c.Hkv * c.D;
    if (!make_map(&maps.k, c, c.k_cache, tokens, stride, c.Hkv, p.box, 1) ||
        !make_map(&maps.v, c, c.v_cache, tokens, stride, c.Hkv, p.box, 1))
      return PA_ERR_CUDA;
  } else {
    p.box = 1;
  }
  const bool bf16 = c.dtype == PA_BF16;
  cudaStream_t st = (cudaStream_t)stream;
  std::lock_guard<std::mutex> lock(launch_mutex(workspace));
  const cudaError_t e = c.D == 128 ? (bf16 ? launch_attend_bf16_d128(p, maps, load, st) : launch_attend_f16_d128(p, maps, load, st))
                                   : (bf16 ? launch_attend_bf16_d256(p, maps, load, st) : launch_attend_f16_d256(p, maps, load, st));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return PA_OK;
}

pa_status cross_call(const pa_cross_args* a, Call* c, int* cap) {
  if (!a) return PA_ERR_INVALID_ARG;
  if (a->rows < 0 || a->B < 0) return PA_ERR_INVALID_ARG;
  const int64_t T = a->B == 0 ? 0 : a->starts ? (int64_t)a->rows : (int64_t)a->B * a->rows;
  *c = Call{a->q, a->k_cache, a->v_cache, a->block_tables, a->seq_lens, a->out, a->q_stride, a->B, a->Hq, a->Hkv, a->D,
            a->block_size, a->num_blocks, a->max_blocks_per_seq, a->max_seq_len, a->scale, a->dtype, a->kv_dtype,
            a->k_scale, a->v_scale, T, (int64_t)a->rows};
  if (a->q_stride % 8 != 0 || (T > 1 && a->q_stride < (int64_t)a->Hq * a->D)) return PA_ERR_INVALID_ARG;
  return check_sizes(*c, cap);
}

pa_status shared_call(const pa_decode_args* a, int num_groups, Call* c, int* cap) {
  if (!a || num_groups < 0) return PA_ERR_INVALID_ARG;
  if (a->q_len < 0 || a->splits < 0 || a->window < 0 || a->total_tokens < 0 || (a->flags & ~PA_FLAG_DETERMINISTIC))
    return PA_ERR_INVALID_ARG;
  if (a->splits > 0 || a->window > 0) return PA_ERR_UNSUPPORTED;
  const int64_t R = std::max(a->q_len, 1), T = (int64_t)a->B * R;
  *c = Call{a->q, a->k_cache, a->v_cache, a->block_tables, a->seq_lens, a->out, (int64_t)a->Hq * a->D, a->B, a->Hq,
            a->Hkv, a->D, a->block_size, a->num_blocks, a->max_blocks_per_seq, a->max_seq_len, a->scale, a->dtype,
            a->kv_dtype, a->k_scale, a->v_scale, T, num_groups > 0 ? T : R};
  if ((int64_t)num_groups + a->B > INT_MAX / 2) return PA_ERR_UNSUPPORTED;
  return check_sizes(*c, cap);
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_cross_workspace_bytes(const pa_cross_args* a) {
  pa::Call c;
  int cap = 0;
  if (pa::cross_call(a, &c, &cap) != PA_OK) return 0;
  const int sms = pa::current_sm_count();
  return sms > 0 ? pa::layout_of(c, sms, a->B, false).total : 0;
}

pa_status pa_cross(const pa_cross_args* a, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  pa::Call c;
  int cap = 0;
  const pa_status st = pa::cross_call(a, &c, &cap);
  if (st != PA_OK) return st;
  if (c.T == 0) return PA_OK;
  pa::AttendParams p{};
  p.B = a->B;
  p.R = a->starts ? 1 : a->rows;
  p.starts = a->starts;
  return pa::run(c, p, cap, workspace, workspace_bytes, stream);
}

size_t pa_decode_shared_workspace_bytes(const pa_decode_args* a, int num_groups) {
  pa::Call c;
  int cap = 0;
  if (pa::shared_call(a, num_groups, &c, &cap) != PA_OK) return 0;
  const int sms = pa::current_sm_count();
  return sms > 0 ? pa::layout_of(c, sms, a->B + num_groups, true).total : 0;
}

pa_status pa_decode_shared(const pa_decode_args* a, const int32_t* groups, const int32_t* prefix_lens, int num_groups,
                           void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  pa::Call c;
  int cap = 0;
  const pa_status st = pa::shared_call(a, num_groups, &c, &cap);
  if (st != PA_OK) return st;
  if (num_groups > 0 && (!groups || !prefix_lens)) return PA_ERR_INVALID_ARG;
  if (c.T == 0) return PA_OK;
  pa::AttendParams p{};
  p.B = a->B;
  p.R = std::max(a->q_len, 1);
  p.shared = 1;
  p.groups = groups;
  p.prefix = prefix_lens;
  p.N = num_groups;
  return pa::run(c, p, cap, workspace, workspace_bytes, stream);
}

}  // extern "C"
