// Launch parameters of the kernels behind pa_cross and pa_decode_shared.
#pragma once

#include <cuda.h>  // CUtensorMap (a type only: the library does not link the driver)

#include "pa_params.h"

namespace pa {

// How K and V reach shared memory: 16-bit caches whose blocks are whole groups of eight tokens by
// tensor copies, other 16-bit caches row by row, fp8 ones likewise and through a ring of raw tiles.
enum AttendLoad { kLoadTensor = 0, kLoad16 = 1, kLoadFp8 = 2 };

// What the merge of rows with two contexts needs of a segment (see pa_attend.cuh).
struct SegmentRecord {
  long long first;     // its first unit
  int tiles, tok0, n;  // of its context; its query tokens
  int group;           // own segments: the group whose prefix the sequence shares, -1 for none
  int pad[2];
};
// An item whose pieces several CTAs hold.
struct SplitItem {
  int tok, rows, kvh;  // first query token, rows (token and head of the group)
  int pieces;          // 0: none
};

struct AttendParams {
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* starts;     // cross: [B + 1], or null
  const int32_t* groups;     // shared prefixes: [N + 1]
  const int32_t* prefix;     // [N]
  uint32_t* err;             // device error word
  // workspace (see layout_of in pa_attend.cu)
  long long* plan;           // units per CTA, units in all
  SegmentRecord* segments;
  SplitItem* split;          // [CTAs] the item that begins in a CTA and ends in a later one
  float2* slot_ml;           // [CTAs][2][slot_rows] reference and sum of the pieces of items that
                             // CTAs share: 0 the end of one, 1 the start of the next
  float* slot_acc;           // [CTAs][2][slot_rows][D] their unnormalised outputs
  float2* row_ml;            // [2][T * Hq] the same of whole items whose rows have two contexts
  float* row_acc;            // [2][T * Hq][D]
  int B, N, T, R;            // sequences, groups (cross: 0), query rows, rows per sequence
  int shared;                // pa_decode_shared
  int Hq, Hkv, G;
  uint32_t g_magic;          // r / G = umulhi(r, g_magic) for r < 2^16, G > 1
  int tile_tokens;           // query tokens of a row tile of the tensor cores, 128 / G
  int spread_tokens;         // of an item whose rows fit in a warp, 32 / G
  int out_wide;              // out is 32-byte aligned
  int block_size, num_blocks, max_blocks, cap;
  uint32_t bs_magic;         // t / block_size as in DecodeParams
  int bs_shift;
  int box;                   // tokens of a tensor copy, a power of two that divides the block size
  int ctas;                  // CTAs that share out the work
  int slot_rows;             // bound on an item's rows
  float scale_log2, v_scale; // |scale| log2(e) (and the scale of K), not zero
  int negate;                // the scale is negative
};

// Row tiles of an item; tokens of the context in a tile.
__host__ __device__ constexpr int attend_row_tiles(int D) { return D == 128 ? 2 : 1; }
__host__ __device__ constexpr int attend_tile(int D) { return D == 128 ? 128 : 64; }

struct AttendMaps {
  CUtensorMap k, v, q, q_spread;
};

// One launcher per type and head_dim: the attention grid and the grid that merges its pieces.
cudaError_t launch_attend_bf16_d128(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st);
cudaError_t launch_attend_bf16_d256(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st);
cudaError_t launch_attend_f16_d128(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st);
cudaError_t launch_attend_f16_d256(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st);

}  // namespace pa
