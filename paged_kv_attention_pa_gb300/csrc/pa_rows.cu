// Rows of a paged cache: pa_append writes new tokens' keys (rotated) and values into the
// pages and rotates their queries on the way; pa_gather reads rows back, contiguous.
//
// Row r of a call is new token i of sequence b, at position t = L - n + i of its context
// (L = seq_lens[b] with the new tokens counted, n new tokens), the token that row i of
// pa_decode's query rows stands for. Packed rows find b by a 32-way search of `starts`.
//
// Rotation. Pair j of a head at position t turns by the angle t * f_j. The angle is kept
// as a 64-bit fraction of a turn, turns[j] = f_j / 2 pi * 2^64, so that t * turns[j] modulo
// 2^64 is the fraction at any position, with an error of t * 2^-64 turns; fp32 enters only
// at the sine of the eighth of a turn that is left beside the nearest quarter.
//
// Both kernels move bytes: a lane handles 16 elements of a row (two 16-byte words of 16-bit
// elements), D / 16 lanes a row, all loads of a warp's rows in flight together. What bounds
// them is HBM for prompts and the chain length -> table entry -> store for single tokens.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_params.h"

namespace pa {

struct RowsParams {
  const void* q;  // append: queries in; q_out rotated
  void* q_out;
  const void* k;  // append: new rows in; gather: unused
  const void* v;
  void* k_out;  // gather: rows out
  void* v_out;
  void* k_cache;
  void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* starts;   // [B + 1], or null: `rows` rows per sequence
  const uint64_t* turns;   // [rot / 2]
  uint32_t* err;
  long long q_stride, k_stride, v_stride;  // elements between rows
  int B, rows, T;          // T rows in all
  int Hq, Hkv;
  int block_size, num_blocks, max_blocks, cap;
  uint32_t bs_magic;       // t / block_size as in DecodeParams
  int bs_shift;
  int rot, interleaved;    // rotated elements of a head
  float amplitude;
  float k_scale, v_scale;  // append: 1 / scale, gather: scale
  float k_div, v_div;      // append: scale
};

constexpr int kRowThreads = 128, kRowWarps = kRowThreads / 32;

// Where row r lives: sequence b, position pos (negative: a context shorter than its rows).
struct Place {
  bool row;  // a row of some sequence (padding rows are left alone)
  bool len;  // whose length is valid
  int b, pos;
  __device__ bool live() const { return row && len && pos >= 0; }
};

// All lanes of the warp together; r is the same in all of them.
__device__ __forceinline__ Place find_row(const RowsParams& p, int r, bool report) {
  Place at{false, false, 0, 0};
  long long n, i;
  int L;
  if (p.starts == nullptr) {
    at.b = r / p.rows;
    n = p.rows;
    i = r - at.b * p.rows;
    L = __ldg(p.seq_lens + at.b);
  } else {
    const int lane = threadIdx.x & 31;
    int s0, s1;
    if (p.B < 32) {  // every start and length in one round trip
      const int start = lane <= p.B ? __ldg(p.starts + lane) : INT_MAX;
      const int len = lane < p.B ? __ldg(p.seq_lens + lane) : 0;
      const int k = __popc(__ballot_sync(0xffffffffu, lane <= p.B && start <= r));
      at.b = k - 1;
      s0 = __shfl_sync(0xffffffffu, start, k - 1);
      s1 = __shfl_sync(0xffffffffu, start, k);
      L = __shfl_sync(0xffffffffu, len, k - 1);
      if (k == 0 || k > p.B) return at;  // before the first row, or behind the last sequence
    } else {
      // the last of starts[0 .. B] at or below r: 32 probes a round
      int lo = 0, len = p.B + 1;
      for (;;) {
        const int step = (len + 31) / 32;
        const int idx = lane * step;
        const bool le = idx < len && __ldg(p.starts + lo + idx) <= r;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        if (k == 0) return at;
        lo += (k - 1) * step;
        len = min(step, len - (k - 1) * step);
        if (step == 1) break;
      }
      if (lo >= p.B) return at;
      at.b = lo;
      s0 = __ldg(p.starts + lo);
      s1 = __ldg(p.starts + lo + 1);
      L = __ldg(p.seq_lens + lo);
    }
    n = (long long)s1 - s0;
    i = (long long)r - s0;
    if (i >= n) return at;  // starts that do not ascend
  }
  at.row = true;
  at.len = L >= 0 && L <= p.cap;
  if (!at.len && report) atomicOr(p.err, PA_DEVERR_SEQ_LEN);
  at.pos = (int)max((long long)L - n + i, -(1ll << 30));
  return at;
}

// Block of the pool that holds token pos of sequence b, and its slot; -1 for a bad table entry.
__device__ __forceinline__ int block_index(const RowsParams& p, int pos) {
  return p.bs_magic == 0 ? pos >> p.bs_shift : (int)(__umulhi((uint32_t)pos, p.bs_magic) >> p.bs_shift);
}
__device__ __forceinline__ int checked_block(const RowsParams& p, int phys, bool report) {
  if ((unsigned)phys < (unsigned)p.num_blocks) return phys;
  if (report) atomicOr(p.err, PA_DEVERR_BLOCK_INDEX);
  return -1;
}

template <KvKind KIND>
__device__ __forceinline__ size_t cache_row(const RowsParams& p, int phys, int slot, int head) {
  return KIND == kKvInt4 ? ((size_t)phys * p.Hkv + head) * p.block_size + slot
                         : ((size_t)phys * p.block_size + slot) * p.Hkv + head;
}

template <typename T>
__device__ __forceinline__ void unpack8(float* x, const uint4& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<T>(word_of(w, i));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                    pack2<T>(x[6], x[7]));
}

// Cosine and sine of the angle turn / 2^32 turns. The nearest quarter turn comes off in integers,
// so that fp32 rounds only the at most eighth of a turn that is left: taken whole, angles near a
// half turn were off by 9e-8, however small their sine.
__device__ __forceinline__ float2 cos_sin(uint32_t turn) {
  const uint32_t quarters = (turn + 0x20000000u) >> 30;
  float s, c;
  sincospif((float)(int32_t)(turn - (quarters << 30)) * 4.656612873077393e-10f, &s, &c);  // half turns: * 2^-31
  const float x = quarters & 1 ? -s : c, y = quarters & 1 ? c : s;
  return quarters & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// (a, b) turned by the angle with cosine cs.x and sine cs.y; of each sum one product is rounded.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float2 cs) {
  const float x = __fmaf_rn(a, cs.x, -__fmul_rn(b, cs.y));
  b = __fmaf_rn(b, cs.x, __fmul_rn(a, cs.y));
  a = x;
}

// x / s, correctly rounded, where y is 1 / s so rounded: as in int4_octet. Quotients from 2^100 on,
// which saturate in every cache, are left as x y (their residual overflows).
__device__ __forceinline__ float quotient(float x, float s, float y) {
  const float q = __fmul_rn(x, y);
  return fabsf(q) < 1.267650600228229e30f ? fmaf(fmaf(-q, s, x), y, q) : q;
}

// Four fp32 values to four E4M3 codes: nearest even, saturating at +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x4(const float* x) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if either is
  float c;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// A quarter of a group (8 consecutive elements; the others in the lanes that differ in the low
// two bits) to its word of codes, and the group's step and minimum. The minimum is rounded
// down and the step up, so every element lies between the first and the sixteenth value.
// Elements saturate at +-65280: with the step's rounding (less than 8) the sixteenth value is
// then below 65280 + 15 * 8 and rounds to a finite fp16 (gather's outputs), and the step is at
// most 130560 / 15 = 8704, whose products with weights are finite in fp16 (decode).
//
// The code is the nearest integer to (x - minimum) / step, exact ties (frequent for 16-bit
// inputs) to even, so the quotient has to be the correctly rounded one. With y the correctly
// rounded 1 / step, which a group shares, q = d y, r = d - q step and q + r y give it
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990). Adding 1.5 * 2^23 rounds it to an integer in the low bits, and eight of them become
// a word by multiplications with 16, less what the constant's bits add up to. Six
// instructions an element: with an IEEE division each, appending 4095 rows of 24/4 heads of
// 256 took 6.6 us more (of 35.7; 27.0 now).
__device__ __forceinline__ uint32_t int4_octet(float (&x)[8], uint16_t* step16, uint16_t* min16) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
  }
  const bool bad = !(lo > -INFINITY && hi < INFINITY);  // a NaN or an infinity in the group
  constexpr float kMost = 65280.f;
  if (lo < -kMost || hi > kMost) {
    lo = fminf(fmaxf(lo, -kMost), kMost);
    hi = fminf(fmaxf(hi, -kMost), kMost);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kMost), kMost);
  }
  const __half mn = __float2half_rd(lo);
  const float low = __half2float(mn);
  const __half st = __float2half_ru(__fdiv_rn(__fsub_rn(hi, low), 15.f));
  const float step = __half2float(st);
  const float y = step > 0.f ? __frcp_rn(step) : 0.f;
  constexpr uint32_t kMagic = 0x4b400000u;         // 1.5 * 2^23
  constexpr uint32_t kSum = kMagic * 0x11111111u;  // its bits over eight nibbles, modulo 2^32
  uint32_t word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float d = __fsub_rn(x[i], low);
    const float q = __fmul_rn(d, y);
    const float n = __fadd_rn(fmaf(fmaf(-q, step, d), y, q), 12582912.f);
    word = word * 16u + __float_as_uint(n);
  }
  *step16 = bad ? (uint16_t)0x7fffu : __half_as_ushort(st);
  *min16 = bad ? (uint16_t)0x7fffu : __half_as_ushort(mn);
  return bad ? 0u : word - kSum;
}

// One row per CTA column blockIdx.x; its warps (and the parts blockIdx.y) share the row's
// warp tasks: IPW query heads, then IPW key heads, then IPW value heads at a time. DIV: a scale is
// no power of two, so that values are divided by it (4096 rows of 24/4 heads of 256 into 4 bits
// 27.4 us, with products 26.8).
template <typename T, KvKind KIND, int D, bool DIV>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const RowsParams p) {
  constexpr int LPI = D / 16, IPW = 32 / LPI;  // lanes per row item, items per warp
  constexpr int ROWB = kv_row_bytes(D, KIND);
  __shared__ __align__(16) float2 turn[D / 2];
  __shared__ __align__(16) float stage[KIND == kKvInt4 ? kRowWarps : 1][KIND == kKvInt4 ? IPW * D : 4];
  __shared__ __align__(16) uint8_t line[KIND == kKvInt4 ? kRowWarps : 1]
                                       [KIND == kKvInt4 ? IPW * PA_INT4_ROW_BYTES(D) : 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = lane / LPI, li = lane % LPI;
  const int r = blockIdx.x;
  const int ntq = (p.Hq + IPW - 1) / IPW, ntk = (p.Hkv + IPW - 1) / IPW;
  const int tasks = ntq + 2 * ntk, stride = kRowWarps * gridDim.y;
  const bool half = !p.interleaved && p.rot > 0;
  const int h = p.rot / 16;  // chunks of eight elements in half of the rotated part

  // A lane holds two chunks of eight elements of a head, one 16-byte load each, so that the
  // lanes' words lie side by side; where pairs lie apart the second chunk of a query or key
  // holds the other halves of the first's pairs.
  const bool on0 = half ? li < h : li < 2 * h, on1 = half ? li < h : li + LPI < 2 * h;  // they turn
  const int q0 = half && li >= h ? li + h : li, q1 = half && li < h ? li + h : li + LPI;
  const T* const qrow = static_cast<const T*>(p.q) + (long long)r * p.q_stride;
  const T* const krow = static_cast<const T*>(p.k) + (long long)r * p.k_stride;
  const T* const vrow = static_cast<const T*>(p.v) + (long long)r * p.v_stride;

  struct Task {
    int which, head;  // which = 0 query, 1 key, 2 value
    bool live;
  };
  auto task_of = [&](int t) -> Task {
    Task k;
    k.which = t < ntq ? 0 : t < ntq + ntk ? 1 : 2;
    k.head = (t - (k.which == 0 ? 0 : k.which == 1 ? ntq : ntq + ntk)) * IPW + item;
    k.live = t < tasks && k.head < (k.which == 0 ? p.Hq : p.Hkv);
    return k;
  };
  auto load = [&](const Task& k, uint4* a, uint4* b) {
    *a = *b = make_uint4(0u, 0u, 0u, 0u);
    if (!k.live) return;
    const uint4* row = reinterpret_cast<const uint4*>((k.which == 0 ? qrow : k.which == 1 ? krow : vrow) + k.head * D);
    *a = __ldcs(row + (k.which == 2 ? li : q0));  // read once (and q may be written in place)
    *b = __ldcs(row + (k.which == 2 ? li + LPI : q1));
  };

  pdl_wait();
  int t = warp + kRowWarps * blockIdx.y;
  Task cur = task_of(t);
  uint4 a, b;
  load(cur, &a, &b);  // independent of where the row goes
  pdl_launch_dependents();

  const bool report = threadIdx.x == 0 && blockIdx.y == 0;
  const Place at = find_row(p, r, report);
  if (!at.row) return;
  int phys = -1;
  size_t row0 = 0;  // the cache row of head 0
  if (at.live()) {
    const int blk = block_index(p, at.pos);
    phys = checked_block(p, __ldg(p.block_tables + (size_t)at.b * p.max_blocks + blk), report);
    row0 = cache_row<KIND>(p, phys, at.pos - blk * p.block_size, 0);
  }
  const int head_rows = KIND == kKvInt4 ? p.block_size : 1;  // cache rows between heads
  for (int j = threadIdx.x; j < p.rot / 2; j += kRowThreads) {
    const float2 cs = cos_sin((uint32_t)(__ldg(p.turns + j) * (uint64_t)(uint32_t)at.pos >> 32));
    const float c = cs.x, s = cs.y;
    const int chunk = half ? j / 8 : j / 4, e = half ? j % 8 : j % 4;
    turn[2 * chunk + e / 2 * (half ? 2 : 4) * LPI + e % 2] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
  // Turns 2 i and 2 i + 1 of a chunk lie side by side, those of the lanes' chunks behind one
  // another: no bank conflicts (a chunk's turns in a row: 4-bit rows as below 29.1 us, not 27.0).
  // Kept in registers over the heads they cost more in resident warps than the loads: 32.9 us
  // against 25.9 for 16-bit rows.
  const float4* const turns = reinterpret_cast<const float4*>(turn);

  while (t < tasks) {
    const int tn = t + stride;
    const Task next = task_of(tn);
    uint4 an, bn;
    load(next, &an, &bn);
    float x0[8], x1[8];  // the first and the second chunk
    unpack8<T>(x0, a);
    unpack8<T>(x1, b);
    // (16-bit chunks that do not turn pass through as they are)
    const bool turn0 = cur.which < 2 && on0, turn1 = cur.which < 2 && on1;
    const int c0 = cur.which == 2 ? li : q0, c1 = cur.which == 2 ? li + LPI : q1;
    if (half) {
      if (turn0) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 w = turns[li + e / 2 * LPI];
          rotate_pair(x0[e], x1[e], make_float2(w.x, w.y));
          rotate_pair(x0[e + 1], x1[e + 1], make_float2(w.z, w.w));
        }
      }
    } else {
      if (turn0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 w = turns[li + e * 2 * LPI];
          rotate_pair(x0[4 * e], x0[4 * e + 1], make_float2(w.x, w.y));
          rotate_pair(x0[4 * e + 2], x0[4 * e + 3], make_float2(w.z, w.w));
        }
      }
      if (turn1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 w = turns[li + LPI + e * 2 * LPI];
          rotate_pair(x1[4 * e], x1[4 * e + 1], make_float2(w.x, w.y));
          rotate_pair(x1[4 * e + 2], x1[4 * e + 3], make_float2(w.z, w.w));
        }
      }
    }
    if (cur.which == 0) {
      if (cur.live) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + ((size_t)r * p.Hq + cur.head) * D);
        const bool zero = !at.live();
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        dst[c0] = zero ? z : turn0 ? pack8<T>(x0) : a;
        dst[c1] = zero ? z : turn1 ? pack8<T>(x1) : b;
      }
    } else if (phys >= 0) {
      uint8_t* cache = static_cast<uint8_t*>(cur.which == 1 ? p.k_cache : p.v_cache);
      const float inv = cur.which == 1 ? p.k_scale : p.v_scale;
      uint8_t* dst = cache + (row0 + (size_t)cur.head * head_rows) * ROWB;
      if constexpr (KIND == kKv16) {
        if (cur.live) {
          reinterpret_cast<uint4*>(dst)[c0] = turn0 ? pack8<T>(x0) : a;
          reinterpret_cast<uint4*>(dst)[c1] = turn1 ? pack8<T>(x1) : b;
        }
      } else {
        const float div = cur.which == 1 ? p.k_div : p.v_div;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x0[e] = DIV ? quotient(x0[e], div, inv) : x0[e] * inv;
          x1[e] = DIV ? quotient(x1[e], div, inv) : x1[e] * inv;
        }
        if constexpr (KIND == kKvFp8) {
          if (cur.live) {
            reinterpret_cast<uint2*>(dst)[c0] = make_uint2(e4m3x4(x0), e4m3x4(x0 + 4));
            reinterpret_cast<uint2*>(dst)[c1] = make_uint2(e4m3x4(x1), e4m3x4(x1 + 4));
          }
        } else {
          using R = Int4Row<D>;
          int g0 = c0, g1 = c1;  // the chunks that x0 and x1 hold
          if (half && cur.which == 1 && h % 4 != 0) {
            // a group's four chunks are not in the four lanes of a quad: exchange them
            // through shared memory
            float4* st = reinterpret_cast<float4*>(stage[warp] + item * D);
            st[2 * c0] = make_float4(x0[0], x0[1], x0[2], x0[3]);
            st[2 * c0 + 1] = make_float4(x0[4], x0[5], x0[6], x0[7]);
            st[2 * c1] = make_float4(x1[0], x1[1], x1[2], x1[3]);
            st[2 * c1 + 1] = make_float4(x1[4], x1[5], x1[6], x1[7]);
            __syncwarp();
            g0 = li;
            g1 = li + LPI;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 u = st[2 * g0 + i], w = st[2 * g1 + i];
              x0[4 * i] = u.x;
              x0[4 * i + 1] = u.y;
              x0[4 * i + 2] = u.z;
              x0[4 * i + 3] = u.w;
              x1[4 * i] = w.x;
              x1[4 * i + 1] = w.y;
              x1[4 * i + 2] = w.z;
              x1[4 * i + 3] = w.w;
            }
          }
          // the row in shared memory, then whole 16-byte words to the page
          uint8_t* l = line[warp] + item * R::BYTES;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = i ? g1 : g0, g = c >> 2;
            uint16_t step16, min16;
            reinterpret_cast<uint32_t*>(l)[(c & 3) * R::G + g] = int4_octet(i ? x1 : x0, &step16, &min16);
            if ((c & 3) == 0) {
              reinterpret_cast<uint16_t*>(l + R::CODES)[g] = step16;
              reinterpret_cast<uint16_t*>(l + R::MINS)[g] = min16;
            }
          }
          __syncwarp();
          const uint4* lv = reinterpret_cast<const uint4*>(l);
          if (cur.live)
            for (int i = li; i < R::BYTES / 16; i += LPI) reinterpret_cast<uint4*>(dst)[i] = lv[i];
          __syncwarp();
        }
      }
    }
    t = tn;
    cur = next;
    a = an;
    b = bn;
  }
}

// One warp per row and IPW KV heads: of each head's K and V, the lane's chunks li and li + LPI of
// eight elements, so that the lanes' words of one load or store lie side by side (16 elements
// in a row per lane left half-written sectors: 36.1 against 30.8 us for 32768 rows of 4 4-bit
// heads of 256, 5.7 TB/s). Two, four or eight rows a warp, their loads in flight together,
// took 41, 48 and 55 us: many short-lived warps keep more in flight.
template <typename T, KvKind KIND, int D>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const RowsParams p) {
  constexpr int LPI = D / 16, IPW = 32 / LPI, ROWB = kv_row_bytes(D, KIND);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = lane / LPI, li = lane % LPI;
  const int nk = (p.Hkv + IPW - 1) / IPW;
  const unsigned id = blockIdx.x * kRowWarps + warp;
  pdl_wait();
  pdl_launch_dependents();
  if (id >= (unsigned)p.T * (unsigned)nk) return;
  const int r = (int)(id / (unsigned)nk), hk = (int)(id - (unsigned)r * nk);
  const int head = hk * IPW + item;
  const bool report = lane == 0 && hk == 0;
  const Place at = find_row(p, r, report);
  if (!at.row) return;
  int slot = 0, phys = -1;
  if (at.live()) {
    const int blk = block_index(p, at.pos);
    slot = at.pos - blk * p.block_size;
    phys = checked_block(p, __ldg(p.block_tables + (size_t)at.b * p.max_blocks + blk), report);
  }
  if (head >= p.Hkv) return;
  uint4 y[2][2];  // K and V, chunks li and li + LPI
#pragma unroll
  for (int s = 0; s < 2; ++s) y[s][0] = y[s][1] = make_uint4(0u, 0u, 0u, 0u);
  if (phys >= 0) {
    const size_t row = cache_row<KIND>(p, phys, slot, head) * ROWB;
    const uint8_t* src[2] = {static_cast<const uint8_t*>(p.k_cache) + row, static_cast<const uint8_t*>(p.v_cache) + row};
    if constexpr (KIND == kKv16) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) y[s][i] = __ldcs(reinterpret_cast<const uint4*>(src[s]) + li + i * LPI);
    } else if constexpr (KIND == kKvFp8) {
      uint2 w[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[s][i] = __ldcs(reinterpret_cast<const uint2*>(src[s]) + li + i * LPI);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t c = e < 2 ? w[s][i].x : w[s][i].y;
            const float2 v = unpack2<__half>(e4m3x2_to_half2((uint16_t)(c >> (16 * (e & 1)))));
            x[2 * e] = v.x * (s ? p.v_scale : p.k_scale);
            x[2 * e + 1] = v.y * (s ? p.v_scale : p.k_scale);
          }
          y[s][i] = pack8<T>(x);
        }
    } else {
      using R = Int4Row<D>;
      uint32_t w[2][2], st[2][2], mn[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = li + i * LPI, g = c >> 2;
          w[s][i] = __ldg(reinterpret_cast<const uint32_t*>(src[s]) + (c & 3) * R::G + g);
          st[s][i] = __ldg(reinterpret_cast<const uint16_t*>(src[s] + R::CODES) + g);
          mn[s][i] = __ldg(reinterpret_cast<const uint16_t*>(src[s] + R::MINS) + g);
        }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 m = unpack2<__half>(st[s][i] | (mn[s][i] << 16));
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = fmaf((float)((w[s][i] >> (4 * e)) & 15u), m.x, m.y) * (s ? p.v_scale : p.k_scale);
          y[s][i] = pack8<T>(x);
        }
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(s ? p.v_out : p.k_out) + ((size_t)r * p.Hkv + head) * D);
    dst[li] = y[s][0];
    dst[li + LPI] = y[s][1];
  }
}

namespace {

template <typename Kern>
cudaError_t launch_rows(Kern kern, dim3 grid, cudaStream_t st, const RowsParams& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

bool power_of_two(float s) {
  int e;
  return std::frexp(s, &e) == 0.5f;
}

template <bool APPEND, typename T, KvKind KIND, int D>
cudaError_t launch_kind(const RowsParams& p, int sms, cudaStream_t st) {
  constexpr int IPW = 32 / (D / 16);
  const int nk = (p.Hkv + IPW - 1) / IPW;
  if constexpr (APPEND) {
    // few rows: their heads over more CTAs (a warp per task at most); many: a CTA per row
    const int tasks = (p.Hq + IPW - 1) / IPW + 2 * nk;
    const int most = (tasks + kRowWarps - 1) / kRowWarps;
    const int parts = (int)std::min<long long>(most, std::max<long long>(1, 4ll * sms / p.T));
    const dim3 grid(p.T, std::min(parts, 65535));
    if constexpr (KIND != kKv16)
      if (!power_of_two(p.k_div) || !power_of_two(p.v_div))
        return launch_rows(append_kernel<T, KIND, D, true>, grid, st, p);
    return launch_rows(append_kernel<T, KIND, D, false>, grid, st, p);
  } else {
    const unsigned ctas = ((unsigned)p.T * (unsigned)nk + kRowWarps - 1) / kRowWarps;
    return launch_rows(gather_kernel<T, KIND, D>, dim3(ctas), st, p);
  }
}

template <bool APPEND>
cudaError_t launch(const RowsParams& p, int D, bool bf16, KvKind kind, int sms, cudaStream_t st) {
#define PA_ROWS_KIND(T, DD)                                                           \
  (kind == kKv16 ? launch_kind<APPEND, T, kKv16, DD>(p, sms, st)                       \
   : kind == kKvFp8 ? launch_kind<APPEND, T, kKvFp8, DD>(p, sms, st)                   \
                    : launch_kind<APPEND, T, kKvInt4, DD>(p, sms, st))
  if (D == 128) return bf16 ? PA_ROWS_KIND(__nv_bfloat16, 128) : PA_ROWS_KIND(__half, 128);
  return bf16 ? PA_ROWS_KIND(__nv_bfloat16, 256) : PA_ROWS_KIND(__half, 256);
#undef PA_ROWS_KIND
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good_scale(float s) { return s > 0.f && s < INFINITY && 1.f / s < INFINITY; }

// The checks that pa_append and pa_gather share. *T: rows in all.
pa_status check_rows(int B, int rows, const int32_t* starts, int Hkv, int D, int block_size,
                     int num_blocks, int max_blocks, int dtype, int kv_dtype, float k_scale,
                     float v_scale, int64_t* T, int* cap) {
  if (B < 0 || rows < 0 || Hkv <= 0 || Hkv > 65535 || D <= 0) return PA_ERR_INVALID_ARG;
  if (D != 128 && D != 256) return PA_ERR_UNSUPPORTED;
  if (block_size <= 0 || num_blocks <= 0 || max_blocks <= 0) return PA_ERR_INVALID_ARG;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_AS_DTYPE && kv_dtype != PA_KV_FP8_E4M3 && kv_dtype != PA_KV_INT4)
    return PA_ERR_INVALID_ARG;
  if (kv_dtype != PA_KV_AS_DTYPE && !(good_scale(k_scale) && good_scale(v_scale)))
    return PA_ERR_INVALID_ARG;
  if (rows_beyond_32_bits(num_blocks, block_size, Hkv)) return PA_ERR_UNSUPPORTED;
  const int64_t c = (int64_t)max_blocks * block_size;
  if (c > INT_MAX) return PA_ERR_OUT_OF_RANGE;
  *cap = (int)c;
  *T = B == 0 ? 0 : starts ? (int64_t)rows : (int64_t)B * rows;
  if (*T > INT_MAX) return PA_ERR_INVALID_ARG;
  // gather's grid: one warp per row and 32 / (D / 16) heads
  const int64_t nk = (Hkv + 512 / D - 1) / (512 / D);
  if (*T * nk > INT_MAX) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_workspace(const void* ws, size_t bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || bytes < PA_WORKSPACE_HEADER_BYTES)
    return PA_ERR_WORKSPACE;
  return PA_OK;
}

KvKind kind_of(int kv_dtype) {
  return kv_dtype == PA_KV_INT4 ? kKvInt4 : kv_dtype == PA_KV_FP8_E4M3 ? kKvFp8 : kKv16;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_append(const pa_append_args* a, void* workspace, size_t workspace_bytes,
                    pa_stream_t stream) {
  using namespace pa;
  if (!a) return PA_ERR_INVALID_ARG;
  int64_t T = 0;
  RowsParams p{};
  pa_status st = check_rows(a->B, a->rows, a->starts, a->Hkv, a->D, a->block_size, a->num_blocks,
                            a->max_blocks_per_seq, a->dtype, a->kv_dtype, a->k_scale, a->v_scale,
                            &T, &p.cap);
  if (st != PA_OK) return st;
  if ((a->q == nullptr) != (a->q_out == nullptr)) return PA_ERR_INVALID_ARG;
  const int Hq = a->q ? a->Hq : 0;
  if (a->q && (a->Hq <= 0 || a->Hq > 65535)) return PA_ERR_INVALID_ARG;
  if (a->rot_dim < 0 || a->rot_dim > a->D || a->rot_dim % 16 != 0) return PA_ERR_INVALID_ARG;
  if (a->rope_layout != PA_ROPE_HALF && a->rope_layout != PA_ROPE_INTERLEAVED) return PA_ERR_INVALID_ARG;
  if (a->rot_dim > 0 && !(std::fabs(a->rope_amplitude) < INFINITY)) return PA_ERR_INVALID_ARG;
  for (int64_t s : {a->k_stride, a->v_stride, a->q ? a->q_stride : 0})
    if (s < 0 || s % 8 != 0) return PA_ERR_INVALID_ARG;
  if (T == 0) return PA_OK;
  if (a->q && a->q_out == a->q && T > 1 && a->q_stride != (int64_t)a->Hq * a->D) return PA_ERR_INVALID_ARG;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->block_tables || !a->seq_lens ||
      (a->rot_dim > 0 && !a->rope_turns))
    return PA_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->q_out) || !aligned16(a->k) || !aligned16(a->v) ||
      !aligned16(a->k_cache) || !aligned16(a->v_cache))
    return PA_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes);
  if (st != PA_OK) return st;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;

  p.q = a->q;
  p.q_out = a->q_out;
  p.k = a->k;
  p.v = a->v;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.block_tables = a->block_tables;
  p.seq_lens = a->seq_lens;
  p.starts = a->starts;
  p.turns = a->rope_turns;
  p.err = static_cast<uint32_t*>(workspace);
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.B = a->B;
  p.rows = a->rows;
  p.T = (int)T;
  p.Hq = Hq;
  p.Hkv = a->Hkv;
  p.block_size = a->block_size;
  p.num_blocks = a->num_blocks;
  p.max_blocks = a->max_blocks_per_seq;
  set_block_division(a->block_size, &p.bs_magic, &p.bs_shift);
  p.rot = a->rot_dim;
  p.interleaved = a->rope_layout == PA_ROPE_INTERLEAVED;
  p.amplitude = a->rope_amplitude;
  const bool scaled = a->kv_dtype != PA_KV_AS_DTYPE;
  p.k_scale = scaled ? 1.f / a->k_scale : 1.f;
  p.v_scale = scaled ? 1.f / a->v_scale : 1.f;
  p.k_div = a->k_scale;
  p.v_div = a->v_scale;
  if (launch<true>(p, a->D, a->dtype == PA_BF16, kind_of(a->kv_dtype), sms, (cudaStream_t)stream) !=
      cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return PA_OK;
}

pa_status pa_gather(const pa_gather_args* a, void* workspace, size_t workspace_bytes,
                    pa_stream_t stream) {
  using namespace pa;
  if (!a) return PA_ERR_INVALID_ARG;
  int64_t T = 0;
  RowsParams p{};
  pa_status st = check_rows(a->B, a->rows, a->starts, a->Hkv, a->D, a->block_size, a->num_blocks,
                            a->max_blocks_per_seq, a->dtype, a->kv_dtype, a->k_scale, a->v_scale,
                            &T, &p.cap);
  if (st != PA_OK) return st;
  if (T == 0) return PA_OK;
  if (!a->k_out || !a->v_out || !a->k_cache || !a->v_cache || !a->block_tables || !a->seq_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(a->k_out) || !aligned16(a->v_out) || !aligned16(a->k_cache) || !aligned16(a->v_cache))
    return PA_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes);
  if (st != PA_OK) return st;
  const int sms = current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;

  p.k_out = a->k_out;
  p.v_out = a->v_out;
  p.k_cache = const_cast<void*>(a->k_cache);
  p.v_cache = const_cast<void*>(a->v_cache);
  p.block_tables = a->block_tables;
  p.seq_lens = a->seq_lens;
  p.starts = a->starts;
  p.err = static_cast<uint32_t*>(workspace);
  p.B = a->B;
  p.rows = a->rows;
  p.T = (int)T;
  p.Hkv = a->Hkv;
  p.block_size = a->block_size;
  p.num_blocks = a->num_blocks;
  p.max_blocks = a->max_blocks_per_seq;
  set_block_division(a->block_size, &p.bs_magic, &p.bs_shift);
  const bool scaled = a->kv_dtype != PA_KV_AS_DTYPE;
  p.k_scale = scaled ? a->k_scale : 1.f;
  p.v_scale = scaled ? a->v_scale : 1.f;
  if (launch<false>(p, a->D, a->dtype == PA_BF16, kind_of(a->kv_dtype), sms, (cudaStream_t)stream) !=
      cudaSuccess) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  return PA_OK;
}

pa_status pa_rope_turns(int rot_dim, double base, const pa_rope_scaling* s, uint64_t* turns,
                        float* amplitude) {
  if (!turns || !amplitude) return PA_ERR_INVALID_ARG;
  if (rot_dim <= 0 || rot_dim > 256 || rot_dim % 16 != 0) return PA_ERR_INVALID_ARG;
  if (!(base > 1.0 && base < INFINITY)) return PA_ERR_INVALID_ARG;
  const int kind = s ? s->kind : PA_ROPE_PLAIN;
  const double factor = kind == PA_ROPE_PLAIN ? 1.0 : s->factor;
  if (kind < PA_ROPE_PLAIN || kind > PA_ROPE_BANDED) return PA_ERR_INVALID_ARG;
  if (!(factor >= 1.0 && factor < INFINITY)) return PA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  const int n = rot_dim / 2;
  double low = 0.0, high = 0.0;
  *amplitude = 1.f;
  if (kind == PA_ROPE_NTK) {
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  } else if (kind == PA_ROPE_YARN) {
    if (s->original_max <= 0 || !(s->slow > 0.0 && s->fast > s->slow && s->fast < INFINITY))
      return PA_ERR_INVALID_ARG;
    // the pair that makes `turns` turns over the original context
    auto pair_of = [&](double t) { return n * std::log(s->original_max / (t * two_pi)) / std::log(base); };
    low = std::max(std::floor(pair_of(s->fast)), 0.0);
    high = std::min(std::ceil(pair_of(s->slow)), (double)(rot_dim - 1));
    *amplitude = (float)(0.1 * std::log(factor) + 1.0);
  } else if (kind == PA_ROPE_BANDED) {
    if (s->original_max <= 0 || !(s->slow > 0.0 && s->fast > s->slow && s->fast < INFINITY))
      return PA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -(double)i / n);
    double g = f;
    if (kind == PA_ROPE_LINEAR) {
      g = f / factor;
    } else if (kind == PA_ROPE_YARN) {
      const double ramp = std::min(std::max((i - low) / std::max(high - low, 1e-3), 0.0), 1.0);
      g = f / factor * ramp + f * (1.0 - ramp);
    } else if (kind == PA_ROPE_BANDED) {
      const double t = s->original_max * f / two_pi;  // turns over the original context
      const double keep = std::min(std::max((t - s->slow) / (s->fast - s->slow), 0.0), 1.0);
      g = f / factor * (1.0 - keep) + f * keep;
    }
    const double turn = g / two_pi;
    turns[i] = (uint64_t)std::ldexp(turn - std::floor(turn), 64);
  }
  return PA_OK;
}

}  // extern "C"
