// Launch parameters shared by the host launcher and the decode kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

// Split counts are bounded, so that the partials stay a small fraction of the KV
// bytes at any context length.
constexpr int kMaxSplits = 1024;
constexpr int kPartitionMin = 64;   // tokens: below this a split's fixed cost dominates
// Tokens per warp tile (a multiple of the score MMA's 16 rows); split partitions
// and static shares are whole tiles.
#ifndef PA_TILE_TOKENS_D128
#define PA_TILE_TOKENS_D128 32
#endif
#ifndef PA_TILE_TOKENS_D256
#define PA_TILE_TOKENS_D256 16
#endif
#ifndef PA_TILE_TOKENS_F8_D128
#define PA_TILE_TOKENS_F8_D128 32
#endif
#ifndef PA_TILE_TOKENS_F8_D256
#define PA_TILE_TOKENS_F8_D256 32
#endif
// What the caches hold: elements of the q/out type, FP8 E4M3, or 4-bit groups.
enum KvKind { kKv16 = 0, kKvFp8 = 1, kKvInt4 = 2 };
// Bytes of one cache row (one token of one KV head) of K or V.
__host__ __device__ constexpr int kv_row_bytes(int D, KvKind kind) {
  return kind == kKv16 ? 2 * D : kind == kKvFp8 ? D : PA_INT4_ROW_BYTES(D);
}
// Per head_dim and cache type: a 256-wide 16-bit row pair is already 1 KB a token;
// fp8 rows carry half the bytes of a 16-bit row for the same arithmetic.
__host__ __device__ constexpr int tile_tokens(int D, KvKind kind) {
  return kind == kKvInt4  ? 32
         : kind == kKvFp8 ? (D == 128 ? PA_TILE_TOKENS_F8_D128 : PA_TILE_TOKENS_F8_D256)
                          : (D == 128 ? PA_TILE_TOKENS_D128 : PA_TILE_TOKENS_D256);
}
// Warps per decode CTA, per head_dim and cache type: fp8 tiles cost more math per
// byte, so the fp8 kernel at head_dim 128 runs more warps.
#ifndef PA_WARPS_D128
#define PA_WARPS_D128 4
#endif
#ifndef PA_WARPS_D256
#define PA_WARPS_D256 4
#endif
#ifndef PA_WARPS_F8_D128
#define PA_WARPS_F8_D128 8
#endif
#ifndef PA_WARPS_F8_D256
#define PA_WARPS_F8_D256 4
#endif
#ifndef PA_WARPS_I4_D128
#define PA_WARPS_I4_D128 12
#endif
#ifndef PA_WARPS_I4_WIDE  // more than 8 columns
#define PA_WARPS_I4_WIDE 8
#endif
#ifndef PA_WARPS_I4_D256
#define PA_WARPS_I4_D256 8
#endif
__host__ __device__ constexpr int warps_per_cta(int D, KvKind kind, int column_tiles = 1) {
  return kind == kKvInt4  ? (column_tiles > 1 ? PA_WARPS_I4_WIDE : D == 128 ? PA_WARPS_I4_D128 : PA_WARPS_I4_D256)
         : kind == kKvFp8 ? (D == 128 ? PA_WARPS_F8_D128 : PA_WARPS_F8_D256)
                          : (D == 128 ? PA_WARPS_D128 : PA_WARPS_D256);
}
// 4-bit caches: from this many query fragments a warp on (column tiles times head_dim / 16)
// they live in shared memory, and with one tile at head_dim 128, whose twelve warps have fewer
// registers each (GB300, us per call in registers / shared: 32/8 heads of 128, 8 query rows of
// 8 sequences of 16K tokens, 32 fragments, 191 / 132; 4 rows, 16 fragments, 55.3 / 56.0; 32
// sequences of 16K, one tile, 126.9 / 125.0; 24/4 heads of 256, 2 rows of 8 sequences of 8K,
// 32 fragments, 36.1 / 35.7; hybrid layer, 32K, one tile, 16 fragments, 13.9 / 14.1).
#ifndef PA_I4_QSHARED
#define PA_I4_QSHARED 32
#endif
// 4-bit caches: bulk copies (one per block and tile) or 16-byte cp.async.
#ifndef PA_I4_BULK_D128
#define PA_I4_BULK_D128 0
#endif
#ifndef PA_I4_BULK_D256
#define PA_I4_BULK_D256 1
#endif
// Work sharing among the splits of a sequence: each split keeps about
// (1 - 1/kStealDiv) of its P tokens as a static share, and the rest of the context
// is claimed tile by tile through one counter per (sequence, KV head) held in the
// workspace header, for up to kStealUnits such pairs (beyond that, static splits)
// and for splits that stream at least kStealMinBytes.
#ifndef PA_STEAL_DIV
#define PA_STEAL_DIV 8
#endif
constexpr int kStealDiv = PA_STEAL_DIV;
// Shorter splits stay static: their imbalance costs less than a claim's round trip.
#ifndef PA_STEAL_MIN_KIB
#define PA_STEAL_MIN_KIB 512
#endif
constexpr long long kStealMinBytes = (long long)PA_STEAL_MIN_KIB * 1024;  // K + V bytes per split
constexpr int kStealUnits = 2048;
// Largest split count whose splits merge inside their thread-block cluster (the
// portable cluster size).
constexpr int kMaxClusterMerge = 8;
constexpr int kHeaderBytes = 256 + kStealUnits * 4;  // error word, then the counters
static_assert(kHeaderBytes % 256 == 0, "header keeps 256-byte alignment");
static_assert(kHeaderBytes == PA_WORKSPACE_HEADER_BYTES, "header size is part of the ABI");

// How a 4-bit decode call runs (see make_plan): as the others do, unsplit with the longest
// sequences' CTAs first (batches of up to kOrderedBatch), or unsplit with short CTAs.
enum Int4Mode { kPlain, kOrdered, kShort };
constexpr int kOrderedBatch = 256;

struct DecodeParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  void* out;
  float* ws_m;        // [B*Hkv*S][G]   running max of each split (log2 domain)
  float* ws_l;        // [B*Hkv*S][G]   softmax denominator of each split
  float* ws_acc;      // [B*Hkv*S][G][D] unnormalised output of each split
  uint32_t* err;      // device error word
  int* steal;         // [B*Hkv] claimed shared tiles per (sequence, KV head); zero between calls
  int B, Hq, Hkv, G;
  int block_size, num_blocks, max_blocks, max_seq_len;
  // t / block_size for 0 <= t < 2^31 without a division: (t >> bs_shift) for a
  // power of two (bs_magic == 0), else umulhi(t, bs_magic) >> bs_shift
  uint32_t bs_magic;
  int bs_shift;
  int S, P;           // splits and tokens per split
  int Ps;             // static tokens per split (== P: no shared tiles)
  int window;         // > 0: attend to the last `window` tokens only
  int q_len;          // query rows per sequence (causal among themselves)
  Int4Mode mode;      // 4-bit caches
  KvKind kv;          // what the caches hold (fp8, 4-bit: k_scale is folded into scale_log2)
  int cmerge;         // 0, or C = S: the S splits of each (sequence, KV head) run as one
                      // thread-block cluster and merge in distributed shared memory (set
                      // by the launcher; no merge grid)
  float v_scale;      // cache V value = stored value * v_scale
  float scale_log2;   // scale * log2(e): scores live in the exp2 domain
};

// Host helpers shared by the entry points (pa_api.cu).
int current_sm_count();
void set_block_division(int d, uint32_t* magic, int* shift);

// One launcher per (dtype, head_dim); each dispatches on the GQA group size. With
// kernels != nullptr nothing is launched: *kernels is set to the number of kernels
// the launch would make (1, or 2 with a merge grid).
cudaError_t launch_decode_bf16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_bf16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_f16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_f16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
// FP8 E4M3 caches with bf16 / fp16 queries and outputs.
cudaError_t launch_decode_fp8_bf16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_fp8_bf16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_fp8_f16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_fp8_f16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
// 4-bit caches with bf16 / fp16 queries and outputs.
cudaError_t launch_decode_int4_bf16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_int4_bf16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_int4_f16_d128(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);
cudaError_t launch_decode_int4_f16_d256(const DecodeParams& p, cudaStream_t st, int* kernels = nullptr);

}  // namespace pa
