// The split-KV decode kernel for 4-bit caches. Splits, work sharing among them, the merge
// of a CTA's warps and of its cluster, and the merge grid are those of pa_decode_kernel.cuh;
// the copies and the arithmetic (pa_int4.cuh) differ.
//
// Loads. As in decode_kernel, every warp streams its own tiles through its own ring, DEPTH - 1
// tiles in flight while it computes one. At head_dim 128 with 16-byte cp.async; at 256 with
// bulk copies, one per block that a tile touches (a KV head's tokens of a block are
// contiguous in a 4-bit page), which complete on the mbarrier of the tile's slot. Measured
// both ways on GB300: head_dim 256, one sequence of 4K / 32K tokens 7.65 / 14.1 us against
// 8.06 / 14.4 us with cp.async; head_dim 128, 32 sequences of 16K 134 us against 125 us (a
// warp's bulk copies issue lane after lane in the path of its arithmetic, and 16-token
// blocks make four a tile). A warp whose copy does not arrive within two seconds reports
// PA_DEVERR_COPY, issues nothing more, waits as long again for each copy in flight and ends.
//
// Math. 160 bytes per token and KV head at head_dim 128 pass through an SM in 3.6 ns at the
// memory's rate, and the arithmetic of its tiles takes as long. Twelve warps at head_dim 128
// with up to 8 columns: 5.5 TB/s with every SM busy (152 pairs of 8K tokens, 36.0 us), against
// 6.2 TB/s for the copies alone. (An earlier build, 34.9 us: eight warps 40.3; two CTAs of six
// warps an SM 37.6; tiles of 64 tokens whose length is known at run time only, with the refill
// behind the arithmetic, 38.3-40.1 with fewer instructions.) More than 16 columns at head_dim 128
// and more than 8 at 256 spill registers (320 and 178 bytes a thread) and run at 0.18 and 0.34
// of the copy rate, where 8 and 16 reach 0.78 and 0.46.
#pragma once

#include "pa_decode_kernel.cuh"
#include "pa_int4.cuh"

namespace pa {

template <int D, int NT, Int4Mode MODE>
struct Int4Cfg {
  static constexpr bool SHORT = MODE == kShort;
  static constexpr int NW = SHORT ? 4 : warps_per_cta(D, kKvInt4, NT);
  static constexpr int CTAS = SHORT ? (D == 128 ? 3 : 2) : 1;  // resident per SM
  static constexpr int THREADS = NW * 32;
  static constexpr int TW = tile_tokens(D, kKvInt4);  // tokens per tile, at most one per lane
  static constexpr int GT = 8 * NT;
  static constexpr int KS = D / 16;
  static constexpr int ROWB = kv_row_bytes(D, kKvInt4);
  static constexpr int CPR = ROWB / 16;  // 16-byte chunks per row
  static constexpr int TILE_BYTES = TW * ROWB;
  static constexpr int SLOT_BYTES = 2 * TILE_BYTES;  // K, then V
  static constexpr bool BULK = D == 256 ? PA_I4_BULK_D256 : PA_I4_BULK_D128;
  static constexpr bool QSHARED = NT * KS >= PA_I4_QSHARED || (NT == 1 && D == 128);  // query fragments
                                                                                 // in shared memory
  static constexpr int QBYTES = QSHARED ? NT * KS * 256 : 0;
  static constexpr int FIXED = 1024 + QBYTES;  // the slots' mbarriers, by_length's answer; the query
  static constexpr int DEPTH_FIT = (kSmemBudget / CTAS - FIXED) / (NW * SLOT_BYTES);
  static constexpr int DEPTH = DEPTH_FIT > 5 ? 5 : DEPTH_FIT;  // slots per warp
  static constexpr int WARP_RING = DEPTH * SLOT_BYTES;
  static constexpr int RING = NW * WARP_RING;
  static constexpr int SMEM = RING + FIXED;
  static_assert(TW == 32 && (TW * CPR) % 32 == 0, "tile shape");
  static_assert(DEPTH >= 2 && NW * DEPTH * 8 <= 1020, "two slots at least, an mbarrier each");
};

// All lanes wait for the bulk copies of the warp's k-th tile; its slots' mbarriers lie at `bars`.
// Where they are late (two seconds) the error is reported and false returned, once the copies
// in flight behind them have landed or are late themselves: this memory is used again.
static __device__ __noinline__ bool wait_for_tile(uint32_t bars, int k, int depth, uint32_t* err) {
  if (__all_sync(0xffffffffu, mbar_wait_long(bars + 8 * (k % depth), (k / depth) & 1))) return true;
  atomicOr(err, PA_DEVERR_COPY);
  for (int i = k; i < k + depth; ++i) mbar_wait_long(bars + 8 * (i % depth), (i / depth) & 1);
  return false;
}

// The sequence whose CTAs run r-th when the longest come first (see make_plan), up to a sixteenth of
// max_seq_len (W words of 32 sequences). All lanes together; every CTA finds the same order.
template <int W>
__device__ __forceinline__ int by_length(const DecodeParams& p, int r) {
  const int lane = threadIdx.x & 31;
  const float per = 16.f / (p.max_seq_len + 1.f);
  int bucket[W];  // 0: the longest
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const int b = 32 * j + lane;
    bucket[j] = b < p.B ? 15 - min(15, max(0, (int)(__ldg(p.seq_lens + b) * per))) : 16;
  }
  // the last bucket with at most r sequences before it, by halves
  int k = 0, before = 0;
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) n += __popc(__ballot_sync(0xffffffffu, bucket[j] < k + half));
    if (n <= r) {
      k += half;
      before = n;
    }
  }
  r -= before;
  int b = 0;
#pragma unroll
  for (int j = 0; j < W; ++j) {  // the sequences of bucket k in their order
    const uint32_t in = __ballot_sync(0xffffffffu, bucket[j] == k);
    const uint32_t at = __ballot_sync(0xffffffffu, bucket[j] == k && __popc(in & ((1u << lane) - 1u)) == r);
    if (at) b = 32 * j + __ffs(at) - 1;
    r -= __popc(in);
  }
  return b;
}

template <typename T, int D, int NT, bool WIN, Int4Mode MODE>
__global__ void __launch_bounds__(Int4Cfg<D, NT, MODE>::THREADS, Int4Cfg<D, NT, MODE>::CTAS)
    decode_int4_kernel(const DecodeParams p) {
  using C = Int4Cfg<D, NT, MODE>;
  constexpr bool ORDERED = MODE == kOrdered;
  using Row = Int4Row<D>;
  constexpr int kWarps = C::NW, kThreads = C::THREADS;
  constexpr int MT = C::TW / 16;  // MMA row blocks of a tile
  extern __shared__ __align__(128) uint8_t smem[];

  const int split = blockIdx.x;
  const int kvh = blockIdx.y;
  int b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int gid = lane >> 2;
  const int tig = lane & 3;
  const int G = p.G;
  const int R = p.q_len;
  const int cols = G * R;  // MMA columns: column c is (row c / G, head kvh*G + c % G)
  T* out = reinterpret_cast<T*>(p.out);
  auto qrow = [&](int c) -> size_t {
    return ((size_t)b * R + c / G) * p.Hq + (size_t)kvh * G + c % G;
  };
  const uint32_t ring = smem_addr(smem) + warp * C::WARP_RING;
  const uint32_t bars = smem_addr(smem) + C::RING + warp * C::DEPTH * 8;  // bulk: a barrier per slot
  if constexpr (C::BULK) {
    if (lane < C::DEPTH) mbar_init(bars + 8 * lane);
    mbar_init_fence();
    __syncwarp();
  }

  // as in decode_kernel: wait for the previous kernel's writes; a split grid lets its merge
  // grid get scheduled at once
  pdl_wait();
  if (p.S > 1 && !p.cmerge) pdl_launch_dependents();
  const uint32_t sequence = smem_addr(smem) + C::RING + 1020;  // b, kept for the epilogue
  if constexpr (ORDERED) {
    b = p.B <= 32 ? by_length<1>(p, b) : p.B <= 64 ? by_length<2>(p, b) : by_length<kOrderedBatch / 32>(p, b);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sequence), "r"(b) : "memory");
    __syncwarp();
  }

  // ---- prologue: length, table entries of the first static tiles and query fragments
  // requested at once
  const int32_t* bt_row = p.block_tables + (size_t)b * p.max_blocks;
  const int cap = (int)min((long long)p.max_seq_len, (long long)p.max_blocks * p.block_size);
  int L = __ldg(p.seq_lens + b);
  auto validate_len = [&]() {
    if (L < 0 || L > cap) {
      if (split == 0 && kvh == 0 && threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_SEQ_LEN);
      L = L < 0 ? 0 : cap;
    }
  };
  int t_lo = 0;
  if constexpr (WIN) {
    validate_len();
    t_lo = max(0, L - p.window);
  }
  const int s_lo = t_lo + split * p.Ps;
  auto static_t0 = [&](int k) { return s_lo + (warp + k * kWarps) * C::TW; };
  // What lane needs of the table for the tile at t0 (0 where there is none): the entry of
  // token t0 + lane, or for bulk copies of the lane-th block that the tile touches.
  const int bst = min(p.block_size, C::TW);
  auto locate = [&](int t0) -> int {
    if (t0 < 0 || t0 >= cap) return 0;
    if constexpr (C::BULK) {
      const int blk = div_block(p, t0);
      return lane * bst < C::TW + bst && lane < p.max_blocks - blk ? __ldg(bt_row + blk + lane) : 0;
    } else {
      return lane < cap - t0 ? __ldg(bt_row + div_block(p, t0 + lane)) : 0;
    }
  };
  int pe[C::DEPTH];  // of tiles 0 .. DEPTH - 1
#pragma unroll
  for (int k = 0; k < C::DEPTH; ++k) pe[k] = locate(static_t0(k));
  uint32_t qf[NT][C::KS][2];
  {
    const uint32_t* q32 = reinterpret_cast<const uint32_t*>(p.q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int c = nt * 8 + gid;
      const bool ok = c < cols;
      const uint4* q4 = reinterpret_cast<const uint4*>(q32 + (qrow(ok ? c : 0) * D) / 2);
#pragma unroll
      for (int g = 0; g < C::KS / 2; ++g) {  // eight consecutive elements of each group
        const uint4 v = ok ? __ldg(q4 + 4 * g + tig) : make_uint4(0u, 0u, 0u, 0u);
        qf[nt][2 * g][0] = v.x;
        qf[nt][2 * g][1] = v.y;
        qf[nt][2 * g + 1][0] = v.z;
        qf[nt][2 * g + 1][1] = v.w;
      }
    }
  }
  if constexpr (!WIN) validate_len();
  if (L == 0 && !p.cmerge) {  // empty context: zero rows, written once
    if (split == 0)
      for (int i = threadIdx.x; i < cols * D; i += kThreads)
        out[qrow(i / D) * D + i % D] = from_f32<T>(0.f);
    return;
  }
  const bool past = t_lo + split * p.P >= L;
  if (past && !p.cmerge) return;
  const int n_splits = (L - t_lo + p.P - 1) / p.P;
  const bool steal = p.Ps < p.P && n_splits > 1;
  const int s_hi = steal ? min(L, s_lo + p.Ps) : min(L, t_lo + (split + 1) * p.P);
  const int n_stat = past ? 0 : (s_hi - s_lo + C::TW - 1) / C::TW;
  const int ns = warp < n_stat ? (n_stat - warp + kWarps - 1) / kWarps : 0;  // this warp's
  const int dyn_lo = steal ? min(L, t_lo + n_splits * p.Ps) : L;
  const int n_dyn = (L - dyn_lo + C::TW - 1) / C::TW;  // shared tiles of the sequence
  int* const ctr = steal ? p.steal + (size_t)b * p.Hkv + kvh : nullptr;
  // ---- copies of one tile into a slot
  const uint64_t pol = l2_evict_first_policy();
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(p.k_cache);
  const ptrdiff_t v_minus_k =
      reinterpret_cast<const uint8_t*>(p.v_cache) - reinterpret_cast<const uint8_t*>(p.k_cache);
  auto issue = [&](int k, int entry, int t0) {  // the warp's k-th tile (none for t0 < 0)
    if (t0 >= 0) {
      const int n = min(C::TW, L - t0);
      const uint32_t dst = ring + (k % C::DEPTH) * C::SLOT_BYTES;
      const bool bad = (unsigned)entry >= (unsigned)p.num_blocks;
      const uint32_t block = ((uint32_t)(bad ? 0 : entry) * (uint32_t)p.Hkv + (uint32_t)kvh) * (uint32_t)p.block_size;
      if constexpr (C::BULK) {
        const int off = t0 - div_block(p, t0) * p.block_size;
        const int first = min(n, p.block_size - off);  // tokens in the first block
        const int start = lane == 0 ? 0 : first + (lane - 1) * bst;
        const uint32_t bar = bars + 8 * (k % C::DEPTH);
        if (lane == 0) mbar_expect(bar, n * 2 * C::ROWB);
        __syncwarp();
        if (start < n) {
          if (bad) atomicOr(p.err, PA_DEVERR_BLOCK_INDEX);
          const uint8_t* src = kbase + (size_t)(block + (lane == 0 ? off : 0)) * C::ROWB;
          const uint32_t bytes = (lane == 0 ? first : min(bst, n - start)) * C::ROWB;
          bulk_copy(dst + start * C::ROWB, src, bytes, bar, pol);
          bulk_copy(dst + C::TILE_BYTES + start * C::ROWB, src + v_minus_k, bytes, bar, pol);
        }
      } else {
        if (lane < n && bad) atomicOr(p.err, PA_DEVERR_BLOCK_INDEX);
        const int t = t0 + lane;  // lanes resolve a row each
        const uint32_t row = block + (uint32_t)(t - div_block(p, t) * p.block_size);
#pragma unroll
        for (int i = 0; i < C::CPR; ++i) {
          const int r = (i * 32 + lane) / C::CPR, c = (i * 32 + lane) % C::CPR;
          const uint32_t rr = __shfl_sync(0xffffffffu, row, r);
          if (r < n) {
            const uint8_t* src = kbase + (size_t)rr * C::ROWB + c * 16;
            cp_async16(dst + 16 * (i * 32 + lane), src, pol);
            cp_async16(dst + 16 * (i * 32 + lane) + C::TILE_BYTES, src + v_minus_k, pol);
          }
        }
      }
    }
    if constexpr (!C::BULK) cp_async_commit();
  };

  // This warp's tiles: its static ones, then shared ones, each claimed one step before its
  // table entries are requested.
  int st_next = 0;        // t0 of the next static tile (none from s_hi on)
  int claim = 0;          // lane 0: result of the claim in flight
  bool claiming = false;  // a claim is in flight
  bool more = n_dyn > 0;  // shared tiles may remain
  auto next_t0 = [&]() -> int {  // t0 of the next tile of the stream, -1 past its end
    int t0 = -1;
    if (st_next < s_hi) {
      t0 = st_next;
      st_next += kWarps * C::TW;
    } else if (more) {
      if (!claiming && lane == 0) claim = atomicAdd(ctr, 1);
      const int g = __shfl_sync(0xffffffffu, claim, 0);
      claiming = false;
      if (g < n_dyn)
        t0 = dyn_lo + g * C::TW;
      else
        more = false;
    }
    if (more && !claiming && st_next >= s_hi) {  // claim the tile after this one now
      if (lane == 0) claim = atomicAdd(ctr, 1);
      claiming = true;
    }
    return t0;
  };
  // The first DEPTH tiles: the static ones among the first DEPTH - 1 go out at once, the
  // shared ones when one claim for all of them and their entries have arrived.
#pragma unroll
  for (int k = 0; k < C::DEPTH - 1; ++k)
    if (k < ns) issue(k, pe[k], static_t0(k));
  int tq[C::DEPTH];  // t0 of tiles k .. k + DEPTH - 1
  {
    const int m0 = ns < C::DEPTH ? C::DEPTH - ns : 0;
    int g0 = 0;
    if (m0 > 0 && more) {
      if (lane == 0) g0 = atomicAdd(ctr, m0);
      g0 = __shfl_sync(0xffffffffu, g0, 0);
    }
#pragma unroll
    for (int k = 0; k < C::DEPTH; ++k) {
      if (k < ns) {
        tq[k] = static_t0(k);
      } else {
        const int g = g0 + (k - ns);
        if (more && g >= n_dyn) more = false;
        tq[k] = more ? dyn_lo + g * C::TW : -1;
        pe[k] = locate(tq[k]);
      }
    }
    st_next = past ? s_hi : static_t0(C::DEPTH);
    if (more && st_next >= s_hi) {
      if (lane == 0) claim = atomicAdd(ctr, 1);
      claiming = true;
    }
  }
#pragma unroll
  for (int k = 0; k < C::DEPTH - 1; ++k)
    if (k >= ns) issue(k, pe[k], tq[k]);
  int next_entry = pe[C::DEPTH - 1];  // for the tile issued in the first loop iteration

  // query fragments in the codes' order, the group sums for the minima, and the factors
  // that turn the two parts of a column's scores into log2 units
  uint32_t qs[NT][2];
  float cs[NT][2], cm[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float f = int4_query<T, D>(qf[nt], qs[nt], tig) * p.scale_log2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cm[nt][h] = __shfl_sync(0xffffffffu, f, 4 * (2 * tig + h));
      cs[nt][h] = cm[nt][h] * 16777216.f;
    }
  }
  // causal limit of each of this thread's columns: row i sees tokens t < L - R + i + 1
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) lim[nt][h] = L - R + (nt * 8 + 2 * tig + h) / G + 1;

  Int4Query<D, NT, C::QSHARED> query;
  if constexpr (C::QSHARED) {  // every warp holds the same fragments: the first one's are kept
    query.at = smem_addr(smem) + C::RING + 1024 + 8 * lane;
    if (warp == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int kk = 0; kk < C::KS; ++kk)
          sts64(query.at + (nt * C::KS + kk) * 256, qf[nt][kk][0], qf[nt][kk][1]);
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int kk = 0; kk < C::KS; ++kk) {
        query.r[nt][kk][0] = qf[nt][kk][0];
        query.r[nt][kk][1] = qf[nt][kk][1];
      }
  }

  // running state: this thread's columns are nt*8 + 2*tig + {0, 1}
  float m[NT][2], l[NT][2];
  float ref[NT][2];  // m, or 0 before the first token
  float o[NT][C::KS][4];
  float om[NT][4];  // the weighted minima
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    om[nt][0] = om[nt][1] = om[nt][2] = om[nt][3] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    ref[nt][0] = ref[nt][1] = 0.f;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int dd = 0; dd < C::KS; ++dd) o[nt][dd][0] = o[nt][dd][1] = o[nt][dd][2] = o[nt][dd][3] = 0.f;
  }
  const int trow = int4_row_of(gid);  // token of this lane's score rows (+ 8)
  // The running max is a reference point, as for fp8 caches: weights are 2^(s - m) against
  // the m in use, raised only when a score exceeds it by more than kSlack, so almost every
  // step skips the rescaling. The weights are also multiplied by the values' steps in fp16:
  // at most 2^2 * 8734, the largest step of a finite fp16 range.
  constexpr float kSlack = 2.f;  // log2 units

  for (int k = 0; tq[0] >= 0; ++k) {  // tile k of the stream: tokens tq[0] ..
    const int entry = next_entry;
    const int t_new = next_t0();   // tile k + DEPTH
    next_entry = locate(t_new);    // one iteration ahead of its use
    issue(k + C::DEPTH - 1, entry, tq[C::DEPTH - 1]);
    const int t0 = tq[0];
#pragma unroll
    for (int i = 0; i + 1 < C::DEPTH; ++i) tq[i] = tq[i + 1];
    tq[C::DEPTH - 1] = t_new;
    const int n = min(C::TW, L - t0);
    const uint32_t kt = ring + (k % C::DEPTH) * C::SLOT_BYTES, vt = kt + C::TILE_BYTES;
    if constexpr (C::BULK) {  // tile k has landed
      const uint32_t bar = bars + 8 * (k % C::DEPTH), parity = (k / C::DEPTH) & 1;
      if (!__all_sync(0xffffffffu, mbar_try(bar, parity)) && !wait_for_tile(bars, k, C::DEPTH, p.err))
        break;  // the outputs mean nothing
    } else {
      cp_async_wait<C::DEPTH - 1>();
    }
    if (n < C::TW) {
      // V rows past the context were never copied: zero their steps and minima (the codes
      // are finite whatever they are), so that p = 0 meets 0
      for (int i = lane; i < (C::TW - n) * Row::W; i += 32)
        sts128_zero(vt + (n + i / Row::W) * C::ROWB + Row::CODES + 16 * (i % Row::W));
      if constexpr (C::BULK) {
        async_proxy_fence();
        __syncwarp();
      }
    }
    if constexpr (!C::BULK) __syncwarp();  // every lane's copies (and the zeros) are visible

    // ---- scores S^T[token][column], in two parts
    float s[MT][NT][4], sm[MT][NT][4];
    int4_scores<D, NT, MT, C::QSHARED>(s, sm, kt, query, qs, gid, tig);
    // ---- online softmax over the tile; -inf by select past each column's limit
    float x[NT][MT][4];
    float mx[NT][2];
    bool grow = false;  // some column of this lane sees a score above its running max + slack
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[nt][mt][i] = fmaf(s[mt][nt][i], cs[nt][i & 1], sm[mt][nt][i] * cm[nt][i & 1]);
    if (t0 + C::TW > L - R + 1) {  // some token is at or past some column's limit
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * mt + trow + 8 * (i >> 1) >= lim[nt][i & 1]) x[nt][mt][i] = -INFINITY;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mx[nt][0] = fmaxf(mx[nt][0], fmaxf(x[nt][mt][0], x[nt][mt][2]));
        mx[nt][1] = fmaxf(mx[nt][1], fmaxf(x[nt][mt][1], x[nt][mt][3]));
      }
      grow = grow || mx[nt][0] > m[nt][0] + kSlack || mx[nt][1] > m[nt][1] + kSlack;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx0 = mx[nt][0], mx1 = mx[nt][1];
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o2));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o2));
        }
        const float mn0 = fmaxf(m[nt][0], mx0), mn1 = fmaxf(m[nt][1], mx1);
        ref[nt][0] = mn0 == -INFINITY ? 0.f : mn0;
        ref[nt][1] = mn1 == -INFINITY ? 0.f : mn1;
        const float al0 = exp2_approx(m[nt][0] - ref[nt][0]);
        const float al1 = exp2_approx(m[nt][1] - ref[nt][1]);
        m[nt][0] = mn0;
        m[nt][1] = mn1;
        l[nt][0] *= al0;
        l[nt][1] *= al1;
        om[nt][0] *= al0;
        om[nt][1] *= al1;
#pragma unroll
        for (int dd = 0; dd < C::KS; ++dd) {
          o[nt][dd][0] *= al0;
          o[nt][dd][1] *= al1;
          o[nt][dd][2] *= al0;
          o[nt][dd][3] *= al1;
        }
      }
    }
    uint32_t pb[MT][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float r0 = ref[nt][0], r1 = ref[nt][1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float p0 = exp2_approx(x[nt][mt][0] - r0), p1 = exp2_approx(x[nt][mt][1] - r1);
        const float p2 = exp2_approx(x[nt][mt][2] - r0), p3 = exp2_approx(x[nt][mt][3] - r1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        pb[mt][nt][0] = movmatrix_trans(pack2<__half>(p0, p1));
        pb[mt][nt][1] = movmatrix_trans(pack2<__half>(p2, p3));
      }
    }
    // ---- O^T[d][column] += V_step^T . P^T
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint32_t rows16 = vt + 16 * mt * C::ROWB;
      if (mt & 1)
        int4_pv<D, NT, true>(o, om, rows16, pb[mt], lane);
      else
        int4_pv<D, NT, false>(o, om, rows16, pb[mt], lane);
    }
    __syncwarp();  // every lane is done with this slot before it is refilled
  }
  if constexpr (!C::BULK) cp_async_wait<0>();

  if (p.S == 1 || p.cmerge) pdl_launch_dependents();
  int4_finish<D, NT>(o, om, tig);
  if constexpr (ORDERED) b = lds32(sequence);
  // Where registers are scarce the epilogue's indexes are made anew there rather than kept
  // through the main loop (GB300, us per call, kept / anew: 32/8 heads of 128, 32 sequences of
  // 16K 126.4 / 125.0, 8 query rows of 8 of 16K 141.9 / 132.5, 4 rows 54.2 / 55.3 (by length,
  // 32 of 1K-16K, 101.4 / 97.2); 24/4 heads
  // of 256, 2 rows of 8 of 8K 35.0 / 35.6).
  if constexpr (D == 128 && (NT != 2 || ORDERED)) {
    const int warp2 = threadIdx.x >> 5, gid2 = (threadIdx.x & 31) >> 2, tig2 = threadIdx.x & 3;
    const int G2 = p.G, R2 = p.q_len, kvh2 = blockIdx.y;
    auto qrow2 = [&](int c) -> size_t {
      return ((size_t)b * R2 + c / G2) * p.Hq + (size_t)kvh2 * G2 + c % G2;
    };
    finish_cta<T, kKvInt4, D, NT, C>(p, smem, blockIdx.x, kvh2, b, warp2, gid2, tig2, G2 * R2,
                                     reinterpret_cast<T*>(p.out), qrow2, n_splits, m, l, o);
  } else {
    finish_cta<T, kKvInt4, D, NT, C>(p, smem, split, kvh, b, warp, gid, tig, cols, out, qrow,
                                     n_splits, m, l, o);
  }
}

template <typename T, int D, int NT, bool WIN, Int4Mode MODE>
struct DecodeKernel<T, int4g32, D, NT, WIN, MODE> {
  using C = Int4Cfg<D, NT, MODE>;
  static constexpr auto kernel = decode_int4_kernel<T, D, NT, WIN, MODE>;
};

}  // namespace pa
