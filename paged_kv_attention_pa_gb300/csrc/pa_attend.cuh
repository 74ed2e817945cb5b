// Attention of many query rows over paged contexts: pa_cross and pa_decode_shared.
//
// Segments. A call is a list of segments, each a run of query tokens that attend to the same
// tokens [lo, hi) of one table row: for cross attention a sequence's queries over its states;
// for shared prefixes first every group's queries over the group's prefix, then every sequence's
// over the rest of its own context. The rows of a segment and KV head are its (query token, head
// of the group) pairs, whole tokens to a row tile of at most 128, cut into items of two row tiles at
// head_dim 128 and of one at 256.
//
// Division of the work. An item's time is taken as a number of units: 5, and for every token tile 2,
// or 3 with two row tiles (GB300: a tile of two takes about 1.6 times one of one; 3 or 4 units an item are
// 0.9% and 0.3% slower over 36 calls). Every CTA, one per SM, takes an equal run of
// the units of all items in order, found from the lengths on the device: runs begin and end inside
// items, and the pieces of an item that several CTAs hold, as well as the two contexts of a row with
// a shared prefix, leave (reference, sum, unnormalised output) in the workspace, which a second grid
// joins. The division depends on the sizes alone, so repeated calls give the same bits.
//
// Roles of the warps of a CTA:
//   softmax   one or two groups of four warps, a thread per row
//   products  one warp, whose lane 0 issues the tensor core products
//   plan      one warp that writes the items into a ring
//   queries   one warp that copies the items' queries
//   load      four warps that issue tensor copies of K and V, or eight that copy their rows and widen fp8
// S = Q K^T goes to tensor memory, a thread reads its row's scores, writes the weights over them
// as the A operand of O += P V, and O stays in tensor memory. Step i of an item uses score buffer
// i % 2, so that the tensor cores work on one while the softmax of the other runs (barriers are kept
// by score buffer: a group never falls two phases of one behind, which parities could not tell): with two groups
// of softmax warps (head_dim 128) each has its own buffer and accumulator, and takes either one of
// the item's two row tiles over the same K and V, or, when all rows fit in one tile, every other
// token tile (the two states then merge in the epilogue).
//
// The reference of a row's weights is its running maximum, raised only when a score exceeds it by
// more than kSlack: the accumulator in tensor memory is rescaled only then, by its softmax warp.
// Weights are 2^(s - ref) in fp32, summed in fp32, and rounded once to the type of the products.
// fp16 weights are kept 2^kLift larger (up to 2^14), so that only those under 2^-20 of the
// row's largest become subnormal.
//
// What bounds it: for few rows HBM (K and V are read once for all rows of an item); for many rows
// the tensor cores and, per row, the exponentials.
#pragma once

#include <cstdint>
#include <type_traits>

#include "pa.h"
#include "pa_attend.h"
#include "pa_device.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

template <typename T, int D, AttendLoad LOAD>
struct AttendCfg {
  using TM = std::conditional_t<LOAD == kLoadFp8, __half, T>;  // type of the products
  static constexpr int NWG = attend_row_tiles(D);              // groups of softmax warps
  static constexpr int TN = attend_tile(D);
  static constexpr int PANELS = D / 64;
  static constexpr int QTILE = 128 * D * 2, NQ = D == 128 ? 2 : 1;
  static constexpr int STAGE = TN * D * 2;
  static constexpr int NS = LOAD == kLoadFp8 ? 3 : 5;
  static constexpr int KVB = LOAD == kLoadFp8 ? 1 : 2;
  static constexpr int RAW = LOAD == kLoadFp8 ? TN * D : 0;  // a staged tile
  static constexpr int NR = 2;                               // of K and of V
  static constexpr int NSW = 4 * NWG;
  static constexpr int W_MMA = NSW, W_PLAN = NSW + 1, W_Q = NSW + 2, W_LOAD = NSW + 3;
  static constexpr int NLOAD = LOAD == kLoadTensor ? 4 : 8;
  static constexpr int READERS = NSW + 2 + NLOAD;  // warps that read the ring of items
  static constexpr int WARPS = NSW + 3 + NLOAD, THREADS = WARPS * 32;
  // Scores that a softmax thread reads at a time: a CTA of 480 threads has 128 registers for each, one of
  // 608 has 96.
  static constexpr int CHUNK = NWG == 2 && NLOAD == 8 ? 16 : 32;
  static constexpr int ITEMS = 4;            // slots of that ring
  static constexpr int OFF_STAGE = NQ * QTILE;
  static constexpr int OFF_RAW = OFF_STAGE + NS * STAGE;
  static constexpr int OFF_SYNC = OFF_RAW + 2 * NR * RAW;
  static constexpr int SYNC_BYTES = 3 * 1024;
  static constexpr int SMEM = OFF_SYNC + SYNC_BYTES;
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
  // tensor memory: score buffers, then accumulators
  static constexpr int S_COL = 0, O_COL = 256;
  static_assert(2 * TN <= 256 && O_COL + NWG * D <= (int)kTmemColumns, "tensor memory");
  // At head_dim 256 Q lies beside the score buffers, and the products take it from there: with 64 tokens
  // a tile, a product of 128 x 64 x 16 from shared memory reads 6 KB in the time of 4, and took 55 cycles
  // instead of 32 (500 rows of 24 heads over 3000 to 6500 tokens, two sequences: 106 us, from tensor memory 96).
  static constexpr bool kQInTmem = D == 256;
  static constexpr int Q_COL = 2 * TN;
  static_assert(!kQInTmem || Q_COL + D / 2 <= O_COL, "Q in tensor memory");
  static constexpr bool kSpread = LOAD == kLoadFp8;        // items of few rows, see spread_rows
  static constexpr int kSpreadTiles = D == 128 ? 6 : 1;
  static constexpr float kSlack = 8.f;  // log2 units
  static constexpr float kLift = std::is_same_v<TM, __half> ? 6.f : 0.f;
};

// ------------------------------------------------------------------ segments
struct Segment {
  int tok0, n;    // its query tokens
  int lo, hi;     // its context
  int table;      // row of the block tables
  int partial;    // 0: the rows' only context; 1, 2: the shared, the own part of two
  int group;      // partial == 2: whose prefix
};
// Sequences [first, end) share their first `tokens` tokens: none in a group of one.
struct Group {
  int first, end, tokens;
};

__device__ __forceinline__ int clamp_len(const AttendParams& p, int b) {
  const int L = __ldg(p.seq_lens + b);
  return L < 0 ? 0 : min(L, p.cap);
}
__device__ __forceinline__ Group read_group(const AttendParams& p, int n) {
  Group g;
  const int a = __ldg(p.groups + n), b = __ldg(p.groups + n + 1), x = __ldg(p.prefix + n);
  g.first = min(max(a, 0), p.B);
  g.end = min(max(b, g.first), p.B);
  g.tokens = g.end - g.first < 2 ? 0 : max(0, min(x, clamp_len(p, g.first)));
  return g;
}
// The group that sequence b is in: the last n of [0, N) that begins at or before it, -1 for none.
template <typename Begin>
__device__ __forceinline__ int group_of(const AttendParams& p, int b, const Begin& begin) {
  int lo = 0, hi = p.N;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (begin(mid) <= b)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}
__device__ __forceinline__ int segment_count(const AttendParams& p) { return p.N + p.B; }
__device__ __forceinline__ Segment prefix_segment(const AttendParams& p, const Group& g) {
  Segment s{};
  s.hi = g.tokens;
  s.tok0 = g.first * p.R;
  s.n = g.tokens > 0 ? (g.end - g.first) * p.R : 0;
  s.table = g.first;
  s.partial = 1;
  return s;
}
// n, g: the group that begins at or before sequence b (n = -1: none)
__device__ __forceinline__ Segment own_segment(const AttendParams& p, int b, int n, const Group& g) {
  Segment s{};
  s.table = b;
  s.hi = clamp_len(p, b);
  if (p.starts) {
    s.tok0 = min(max(__ldg(p.starts + b), 0), p.T);
    s.n = min(max(__ldg(p.starts + b + 1), s.tok0), p.T) - s.tok0;
  } else {
    s.tok0 = b * p.R;
    s.n = p.R;
  }
  if (n >= 0 && b >= g.first && b < g.end && g.tokens > 0) {
    s.lo = g.tokens;
    s.partial = 2;
    s.group = n;
  }
  return s;
}

// A segment's items and units. Its tiles start at a multiple of a tensor copy's box; an empty
// context has one tile without a token. A KV head's items are equal but for the last.
constexpr int kItemUnits = 5;
// A CTA's run is at least two tiles, one for each softmax group. (With less than a tile's units a
// CTA amid an item's pieces could hold none of it.)
constexpr int kLeastUnits = 4;
__host__ __device__ constexpr int tile_units(int row_tiles) { return row_tiles == 2 ? 3 : 2; }
struct Shape {
  int tiles, items;   // of an item, of a KV head
  int full, last;     // units of a tile
  long long head;     // units of a KV head
};
__device__ __forceinline__ int first_token(const AttendParams& p, const Segment& g) { return g.lo & -p.box; }
template <int D>
__device__ __forceinline__ int tiles_of(const AttendParams& p, const Segment& g) {
  return max(1, (g.hi - first_token(p, g) + attend_tile(D) - 1) / attend_tile(D));
}
template <int D>
__device__ __forceinline__ Shape shape_of(const AttendParams& p, int tiles, int n) {
  Shape z;
  const unsigned tokens = p.tile_tokens * attend_row_tiles(D);
  z.tiles = tiles;
  z.items = (int)(((unsigned)n + tokens - 1) / tokens);
  z.full = tile_units(attend_row_tiles(D));
  z.last = n - (z.items - 1) * (int)tokens > p.tile_tokens ? z.full : tile_units(1);
  z.head = z.items == 0 ? 0 : (long long)z.items * kItemUnits + ((long long)(z.items - 1) * z.full + z.last) * tiles;
  return z;
}
// First unit of an item's first tile, in its segment.
__device__ __forceinline__ long long units_before(const Shape& z, int kvh, int item) {
  return kvh * z.head + (long long)item * (kItemUnits + z.full * z.tiles) + kItemUnits;
}
__device__ __forceinline__ int div_group(const AttendParams& p, int r) {
  return p.G == 1 ? r : (int)__umulhi((uint32_t)r, p.g_magic);
}
__device__ __forceinline__ int div_block(const AttendParams& p, int t) {
  return p.bs_magic == 0 ? t >> p.bs_shift : (int)(__umulhi((uint32_t)t, p.bs_magic) >> p.bs_shift);
}
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A piece of an item: the tiles of it that a CTA computes.
enum Dest { kDirect = 0, kSlotFirst = 1, kSlotNext = 2, kRowShared = 3, kRowOwn = 4 };
struct Item {
  int tiles;      // 0: the end of the CTA's work
  int t0;         // first token of the first tile
  int lo, hi;     // the segment's context
  int table, kvh;
  int tok, rows;  // its first query token, its rows
  int of_prefix;  // rows of several sequences
  int dest;
};

// ------------------------------------------------------------------ waits
// Waits end after two seconds, and 5 us for each unit of the CTA's run: warps may wait for a whole item, and
// one of 10^8 tokens takes seconds.
struct GiveUp {
  volatile int now;
  volatile unsigned long long after;  // ns
};
constexpr unsigned long long kGiveUpAfter = 2000000000ull, kGiveUpUnit = 5000ull;
// Wait for a phase of a barrier; false when it took too long or another warp gave up. The
// whole warp together. (The slow part is a function of its own: inlined everywhere it cost 2%, 4096 rows
// over 8192 tokens 352 us instead of 345.)
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, GiveUp* give_up) {
  const uint64_t t0 = global_ns(), after = give_up->after;
  for (;;) {
    const bool over = global_ns() - t0 >= after || give_up->now != 0;
    const bool done = mbar_try(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if (__any_sync(0xffffffffu, over)) {
      give_up->now = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, GiveUp* give_up) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  return wait_long(bar, parity, give_up);
}

// ------------------------------------------------------------------ shared memory
template <typename C>
struct AttendShared {
  uint64_t kv_full[C::NS], kv_empty[C::NS];
  uint64_t q_raw[C::NQ], q_full[C::NQ], q_empty[C::NQ], q_tmem;
  uint64_t s_full[2], p_full[2];
  uint64_t pv_done[2];  // by the step's score buffer
  uint64_t item_full[C::ITEMS], item_empty[C::ITEMS];
  uint64_t pair, drain;
  uint32_t tmem;
  GiveUp give_up;
  int first_segment;
  long long first_unit, per, total;
  Item items[C::ITEMS];
  float2 state[2][128];    // (reference, sum) of the two softmax groups
  long long scan[32];
};

#define PA_WAIT(bar, parity)                                          \
  do {                                                                \
    if (!wait_for(smem_addr(&(bar)), (parity), &sh.give_up)) return;  \
  } while (0)

// ------------------------------------------------------------------ plan
// Every CTA finds the first unit of its run: a sum over the segments' units. CTA 0 writes what the
// merge reads and reports lengths, groups and starts that are out of range. `groups`: room for
// kGroupTable groups in shared memory; with more they are read from global memory as needed.
constexpr int kGroupTable = 8192;
template <typename C, int D>
__device__ __forceinline__ void plan_work(const AttendParams& p, AttendShared<C>& sh, Group* groups) {
  static_assert(kGroupTable * sizeof(Group) <= C::NS * C::STAGE, "groups in the ring's memory");
  const int n = segment_count(p), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool report = blockIdx.x == 0, table = p.N <= kGroupTable;
  if (table && p.N > 0) {
    for (int i = tid; i < p.N; i += C::THREADS) groups[i] = read_group(p, i);
    __syncthreads();
  }
  auto group_at = [&](int i) { return table ? groups[i] : read_group(p, i); };
  auto segment_of = [&](int s) -> Segment {
    if (s < p.N) return prefix_segment(p, group_at(s));
    const int b = s - p.N;
    int g = -1;
    if (p.N > 0)
      g = table ? group_of(p, b, [&](int i) { return groups[i].first; })
                : group_of(p, b, [&](int i) { return __ldg(p.groups + i); });
    return own_segment(p, b, g, g >= 0 ? group_at(g) : Group{});
  };
  auto shape = [&](const Segment& g) { return shape_of<D>(p, tiles_of<D>(p, g), g.n); };
  const int each = (n + C::THREADS - 1) / C::THREADS;
  const int s0 = min(n, tid * each), s1 = min(n, s0 + each);
  long long mine = 0;
  Segment only{};  // with one segment a thread, it
  long long only_units = 0;
  for (int s = s0; s < s1; ++s) {
    only = segment_of(s);
    only_units = shape(only).head * p.Hkv;
    mine += only_units;
    if (report) {
      uint32_t bad = 0;
      if (s < p.N) {
        const int a = __ldg(p.groups + s), b = __ldg(p.groups + s + 1), x = __ldg(p.prefix + s);
        if (a < 0 || b < a || b > p.B) bad |= PA_DEVERR_ROWS;
        if (x < 0 || x > p.cap) bad |= PA_DEVERR_SEQ_LEN;
      } else {
        const int b = s - p.N, L = __ldg(p.seq_lens + b);
        if (L < 0 || L > p.cap) bad |= PA_DEVERR_SEQ_LEN;
        if (p.starts) {
          const int x = __ldg(p.starts + b), y = __ldg(p.starts + b + 1);
          if (x < 0 || y < x || y > p.T) bad |= PA_DEVERR_ROWS;
        }
      }
      if (bad) atomicOr(p.err, bad);
    }
  }
  long long upto = mine;  // inclusive sum over the threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  long long total = lane < C::WARPS ? sh.scan[lane] : 0;  // then the inclusive sum over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, total, o);
    if (lane >= o) total += x;
  }
  const long long warps_before = __shfl_sync(0xffffffffu, total, warp - 1 & 31);
  if (warp > 0) upto += warps_before;
  total = __shfl_sync(0xffffffffu, total, 31);
  const long long per = max((long long)kLeastUnits, quotient(total + p.ctas - 1, p.ctas));
  const long long from = per * blockIdx.x;
  if (tid == 0) {
    p.split[blockIdx.x].pieces = 0;  // until the plan warp finds one
    sh.per = per;
    sh.give_up.after = kGiveUpAfter + kGiveUpUnit * per;
    sh.total = total;
    if (from >= total) sh.first_segment = n;
    if (report) {
      p.plan[0] = per;
      p.plan[1] = total;
    }
  }
  long long at = upto - mine;
  const bool here = from >= at && from < upto, write = report && p.shared;
  if (here || write) {
    for (int s = s0; s < s1; ++s) {
      const Segment g = each == 1 ? only : segment_of(s);
      const long long u = each == 1 ? only_units : shape(g).head * p.Hkv;
      if (from >= at && from < at + u) {
        sh.first_segment = s;
        sh.first_unit = at;
      }
      if (write) {
        SegmentRecord r{};
        r.first = at;
        r.tiles = tiles_of<D>(p, g);
        r.tok0 = g.tok0;
        r.n = g.n;
        r.group = g.partial == 2 ? g.group : -1;
        p.segments[s] = r;
      }
      at += u;
    }
  }
  // Tensor copies will write where the groups lay: a fence of every thread orders its accesses, which
  // are ordinary ones, before them (with the barrier of the CTA that follows).
  if (table && p.N > 0) async_proxy_fence();
}

// The plan warp: the pieces of this CTA's run, in order.
template <typename C, int D>
__device__ __forceinline__ void plan_role(const AttendParams& p, AttendShared<C>& sh) {
  const int lane = threadIdx.x & 31;
  const long long lo = sh.per * blockIdx.x, hi = min(lo + sh.per, sh.total);
  uint32_t count = 0;
  const int n = segment_count(p);
  long long at = sh.first_unit;
  bool first = true;
  int held = -2;  // the group read last
  Group group{};
  for (int s = sh.first_segment; s < n && at < hi; ++s) {
    Segment g;
    if (s < p.N) {
      g = prefix_segment(p, read_group(p, s));
    } else {
      const int b = s - p.N;
      if (held == -2 || b >= group.end) {  // sequences ascend
        held = p.N > 0 ? group_of(p, b, [&](int i) { return __ldg(p.groups + i); }) : -1;
        group = held >= 0 ? read_group(p, held) : Group{};
      }
      g = own_segment(p, b, held, group);
    }
    const Shape z = shape_of<D>(p, tiles_of<D>(p, g), g.n);
    int kvh = 0, r = 0;
    if (first && z.items > 0) {  // the item that holds unit lo
      kvh = (int)quotient(lo - at, z.head);
      r = (int)min((long long)z.items - 1, quotient(lo - at - kvh * z.head, kItemUnits + z.full * z.tiles));
    }
    first = false;
    for (; kvh < p.Hkv && z.items > 0; ++kvh, r = 0) {
      for (; r < z.items; ++r) {
        const long long u = at + units_before(z, kvh, r);
        if (u - kItemUnits >= hi) break;
        // tile t, from unit u + w t on, is the CTA's whose run holds that unit
        const int w = r == z.items - 1 ? z.last : z.full;
        const int ta = u >= lo ? 0 : (int)quotient(lo - u + w - 1, w);
        const int tb = hi <= u ? 0 : (int)min((long long)z.tiles, quotient(hi - u + w - 1, w));
        if (ta >= tb) continue;
        const int slot = count % C::ITEMS;
        PA_WAIT(sh.item_empty[slot], ((count / C::ITEMS) & 1) ^ 1);
        if (lane == 0) {
          Item& it = sh.items[slot];
          it.tiles = tb - ta;
          it.t0 = first_token(p, g) + ta * C::TN;
          it.lo = g.lo;
          it.hi = g.hi;
          it.table = g.table;
          it.kvh = kvh;
          const int t0 = r * C::NWG * p.tile_tokens;
          it.tok = g.tok0 + t0;
          it.rows = min(C::NWG * p.tile_tokens, g.n - t0) * p.G;
          it.of_prefix = g.partial == 1;
          it.dest = ta > 0 ? kSlotNext
                    : tb < z.tiles ? kSlotFirst
                    : g.partial == 1 ? kRowShared : g.partial == 2 ? kRowOwn : kDirect;
          mbar_arrive(smem_addr(&sh.item_full[slot]));
          if (it.dest == kSlotFirst) {
            const long long last = min((long long)p.ctas - 1, quotient(u + (long long)w * (z.tiles - 1), sh.per));
            p.split[blockIdx.x] = SplitItem{it.tok, it.rows, kvh, (int)last - (int)blockIdx.x + 1};
          }
        }
        __syncwarp();
        ++count;
      }
      if (at + (kvh + 1) * z.head >= hi) break;
    }
    at += z.head * p.Hkv;
  }
  const int slot = count % C::ITEMS;
  PA_WAIT(sh.item_empty[slot], ((count / C::ITEMS) & 1) ^ 1);
  if (lane == 0) {
    sh.items[slot].tiles = 0;
    mbar_arrive(smem_addr(&sh.item_full[slot]));
  }
}

// The next item, read by a whole warp.
template <typename C>
__device__ __forceinline__ bool next_item(AttendShared<C>& sh, uint32_t& count, Item& it) {
  const int slot = count % C::ITEMS;
  if (!wait_for(smem_addr(&sh.item_full[slot]), (count / C::ITEMS) & 1, &sh.give_up)) return false;
  it = sh.items[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&sh.item_empty[slot]));
  ++count;
  return it.tiles > 0;
}

// Both softmax groups work on the item's two row tiles, or share the tiles of one.
template <typename C>
__device__ __forceinline__ bool two_row_tiles(const AttendParams& p, const Item& it) {
  return C::NWG == 2 && it.rows > p.tile_tokens * p.G;
}

// An fp8 item whose rows fit in a warp is spread: the row tile holds them four times, and each of a
// group's four warps, which reach 32 rows each, sees a quarter of a tile's tokens: the weights of the others
// are zero in its rows. One warp for all tokens, while three have nothing to do, is slower than fp8 tiles come
// in: 24 sequences of 14 rows a KV head over 1000 to 6000 tokens took 102 us, 93 spread, 16 of 6 rows of 256
// behind two prefixes 63 and 47. 16-bit tiles take twice as long to come: 64 sequences 67.3 us, 69.1 spread, and
// at head_dim 256 57.3 and 58.0.
// The states of the warps are joined behind an item's last tile, which costs more than it saves in short ones:
// 128 contexts of 16 to 700 tokens behind a document took 118.0 us with all of them spread, 116.6 with those of
// 6 tiles and more.
template <typename C>
__device__ __forceinline__ bool spread_rows(const AttendParams& p, const Item& it) {
  return C::kSpread && it.rows <= p.spread_tokens * p.G && it.tiles >= C::kSpreadTiles;
}

// ------------------------------------------------------------------ load
// The order in which the products need K and V: K runs `lead` tiles ahead.
//   K(0) .. K(lead - 1), V(0), K(lead), V(1), ...
// Tiles are staged in this order; place_k and place_v are a tile's place among an item's
// 2 * tiles.
template <typename C>
__device__ __forceinline__ int lead_of(const AttendParams& p, const Item& it) {
  return two_row_tiles<C>(p, it) ? 1 : 2;
}
__device__ __forceinline__ int place_k(int t, int lead) { return t < lead ? t : 2 * t - lead + 1; }
__device__ __forceinline__ int place_v(int t, int lead, int tiles) { return min(t + lead, tiles) + t; }

// Tensor copies, two warps for K and two for V, which take half of the panels each: a warp is held
// for about 75 cycles and 4.4 for every 128-byte row of a copy, so that of blocks of 16 tokens one
// warp brings 15 bytes a cycle and four bring 59 (with an L2 policy fewer once they are many: 66
// bytes a cycle at most, without one 84). The tensor cores need 32 at head_dim 128, HBM gives 24.
// Lane l copies box l of a tile; boxes without a token are left out.
template <typename C, int D>
__device__ __forceinline__ void tensor_load_role(const AttendParams& p, const CUtensorMap* map, bool is_k, int half,
                                                 AttendShared<C>& sh, uint8_t* stages) {
  constexpr int P0 = C::PANELS / 2;  // panels of a warp
  const int lane = threadIdx.x & 31;
  const int boxes = C::TN / p.box;
  const uint32_t base = smem_addr(stages) + half * P0 * C::TN * 128, box_bytes = p.box * 128;
  uint32_t before = 0, count = 0;  // tiles of K and V of the items before
  Item it;
  while (next_item(sh, count, it)) {
    const int32_t* row = p.block_tables + (size_t)it.table * p.max_blocks;
    const int lead = lead_of<C>(p, it);
    int tok = it.t0 + lane * p.box;  // the box's first token
    // (a sequence that ends within its group's prefix, in the box where that ends, has none of its own)
    auto holds = [&](int tk) { return lane < boxes && max(tk, it.lo) < min(tk + p.box, it.hi); };
    auto entry = [&](int t, int tk) -> int { return t < it.tiles && holds(tk) ? __ldg(row + div_block(p, tk)) : 0; };
    int phys = entry(0, tok);
    for (int t = 0; t < it.tiles; ++t, tok += C::TN) {
      const uint32_t n = before + (is_k ? place_k(t, lead) : place_v(t, lead, it.tiles));
      const int stage = n % C::NS;
      const int ahead = entry(t + 1, tok + C::TN);
      const bool here = holds(tok);
      if ((unsigned)phys >= (unsigned)p.num_blocks) {
        atomicOr(p.err, PA_DEVERR_BLOCK_INDEX);
        phys = 0;
      }
      const int at = phys * p.block_size + (tok - div_block(p, tok) * p.block_size);
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, here)) * box_bytes * P0;
      const uint32_t bar = smem_addr(&sh.kv_full[stage]);
      PA_WAIT(sh.kv_empty[stage], ((n / C::NS) & 1) ^ 1);
      if (lane == 0) mbar_expect(bar, bytes);
      __syncwarp();
      if (here) {
        const uint32_t dst = base + stage * C::STAGE + lane * box_bytes;
#pragma unroll
        for (int c = 0; c < P0; ++c)
          tensor_load3(dst + c * C::TN * 128, map, bar, (half * P0 + c) * 64, it.kvh, at);
      }
      __syncwarp();
      phys = ahead;
    }
    before += 2 * it.tiles;
  }
}

// Where cp.async brings a tile: four warps for K and four for V, a warp for a quarter of the rows. Lane
// l resolves the warp's row l and the lanes copy 16-byte chunks. 16-bit chunks go to their place in the
// tile, with zeros for rows without a token; fp8 chunks to a ring of raw tiles, from which each lane
// later widens those it copied. A warp takes some 1400 cycles for an fp8 tile, most of them latencies
// between its few instructions, so that K and V side by side take half the time of one after the other.
template <typename C, int D, bool FP8>
struct RowLoader {
  static constexpr int CPR = D * C::KVB / 16;  // chunks of a row
  static constexpr int RW = C::TN / 4;         // rows of a warp
  static constexpr int CH = RW * CPR / 32;     // chunks of a lane
  static constexpr int RPI = 32 / CPR;         // rows of a warp's i-th chunks
  const AttendParams& p;
  AttendShared<C>& sh;
  const bool is_k;
  const int warp, lane;
  const uint8_t* const src;
  uint32_t at;                           // this lane's first chunk in a tile
  uint32_t count = 0, before = 0;        // items; tiles of the items before
  Item it{};
  int t = 0, phys = 0;                   // the tile to issue, lane l's block of its row l
  bool more;

  __device__ __forceinline__ RowLoader(const AttendParams& p, AttendShared<C>& sh, bool is_k, int warp)
      : p(p), sh(sh), is_k(is_k), warp(warp), lane(threadIdx.x & 31),
        src(static_cast<const uint8_t*>(is_k ? p.k_cache : p.v_cache) + (threadIdx.x & 31) % CPR * 16) {
    // Chunk h (8 elements) of row r goes to chunk (h % 8) ^ (r % 8) of its panel's row. Rows i RPI + j
    // of the warp, j < RPI: r % 8 is (i RPI % 8) | j, so that the address is xored with a constant.
    const int j = lane / CPR, h = lane % CPR * (FP8 ? 2 : 1);
    at = (h >> 3) * (C::TN * 128) + (warp * RW + j) * 128 + (((h & 7) ^ j) << 4);
    more = next_item(sh, count, it);
    if (more) phys = entry(0);
  }
  __device__ __forceinline__ uint32_t place_in(uint32_t tile, int i) const {
    return ((tile + at) ^ ((i * RPI & 7) << 4)) + i * RPI * 128;
  }
  __device__ __forceinline__ int entry(int tile) const {
    const int tok = it.t0 + tile * C::TN + warp * RW + lane;
    return tile < it.tiles && lane < RW && tok >= it.lo && tok < it.hi
               ? __ldg(p.block_tables + (size_t)it.table * p.max_blocks + div_block(p, tok))
               : 0;
  }
  __device__ __forceinline__ uint32_t place() const {  // of the tile to issue in the ring
    return before + (is_k ? place_k(t, lead_of<C>(p, it)) : place_v(t, lead_of<C>(p, it), it.tiles));
  }
  __device__ __forceinline__ int2 rows() const {  // of that tile that hold tokens
    const int t0 = it.t0 + t * C::TN;
    return make_int2(max(0, min(C::TN, it.lo - t0)), max(0, min(C::TN, it.hi - t0)));
  }
  // Chunk i goes to to(i). Then the next tile is the one to issue.
  template <typename To>
  __device__ __forceinline__ void issue(const int2& r01, const To& to) {
    const int tok = it.t0 + t * C::TN + warp * RW + lane;
    if ((unsigned)phys >= (unsigned)p.num_blocks) {
      atomicOr(p.err, PA_DEVERR_BLOCK_INDEX);
      phys = 0;
    }
    const int off = tok - div_block(p, tok) * p.block_size;
    const uint32_t row =
        ((uint32_t)phys * (uint32_t)p.block_size + (uint32_t)off) * (uint32_t)p.Hkv + (uint32_t)it.kvh;
    phys = entry(t + 1);
    const bool all = r01.x == 0 && r01.y == C::TN;
    if (all) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const uint32_t rr = __shfl_sync(0xffffffffu, row, i * RPI + lane / CPR);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to(i)), "l"(src + (size_t)rr * (D * C::KVB))
                     : "memory");
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < CH; ++i) {
        const uint32_t rr = __shfl_sync(0xffffffffu, row, i * RPI + lane / CPR);
        const int r = warp * RW + i * RPI + lane / CPR;
        const bool here = r >= r01.x && r < r01.y;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to(i)),
                     "l"(here ? src + (size_t)rr * (D * C::KVB) : src), "r"(here ? 16 : 0)
                     : "memory");
      }
    }
    if (++t == it.tiles) {
      before += 2 * it.tiles;
      more = next_item(sh, count, it);
      t = 0;
      if (more) phys = entry(0);
    }
  }
  __device__ __forceinline__ void landed(uint32_t place) {  // this lane's part of a tile is in its place
    async_proxy_fence();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.kv_full[place % C::NS]));
  }
  __device__ __forceinline__ bool room(uint32_t place) {
    return wait_for(smem_addr(&sh.kv_empty[place % C::NS]), ((place / C::NS) & 1) ^ 1, &sh.give_up);
  }
};

template <typename C, int D>
__device__ __forceinline__ void row_load_role(const AttendParams& p, bool is_k, int warp, AttendShared<C>& sh,
                                              uint8_t* stages) {
  RowLoader<C, D, false> L(p, sh, is_k, warp);
  const uint32_t base = smem_addr(stages);
  uint32_t last = 0;
  bool pending = false;  // a tile is on its way
  while (L.more) {
    const uint32_t n = L.place();
    if (!L.room(n)) break;
    const uint32_t tile = base + n % C::NS * C::STAGE;
    L.issue(L.rows(), [&](int i) { return L.place_in(tile, i); });
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (pending) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      L.landed(last);
    }
    last = n;
    pending = true;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (pending) L.landed(last);
}

template <typename C, int D>
__device__ __forceinline__ void fp8_load_role(const AttendParams& p, bool is_k, int warp, AttendShared<C>& sh,
                                              uint8_t* stages, uint8_t* raw) {
  using Loader = RowLoader<C, D, true>;
  Loader L(p, sh, is_k, warp);
  const int lane = threadIdx.x & 31;
  const uint32_t raw_lane = smem_addr(raw) + (is_k ? 0 : C::NR * C::RAW) + warp * (C::RAW / 4) + lane * 16;
  static_assert(C::NR == 2, "one tile on its way while another is widened");
  uint32_t issued = 0, done = 0, place[2];
  auto issue = [&](int k) {  // the next tile, if there is one
    if (L.more) {
      place[k] = L.place();
      const uint32_t dst = raw_lane + issued % 2 * C::RAW;
      ++issued;
      L.issue(L.rows(), [&](int i) { return dst + i * 512; });
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  issue(0);
  for (;;) {
    issue(1);
    if (done == issued) break;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint32_t n = place[0];
    place[0] = place[1];
    if (!L.room(n)) break;
    const uint32_t from = raw_lane + done % 2 * C::RAW, tile = smem_addr(stages) + n % C::NS * C::STAGE;
    static_assert(Loader::CH == 8, "a tile's chunks of a lane");
    uint4 chunk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) chunk[i] = lds128(from + i * 512);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = chunk[i];
      const uint32_t a = L.place_in(tile, i);
      uint4 lo, hi;
      lo.x = e4m3x2_to_half2(x.x & 0xffff);
      lo.y = e4m3x2_to_half2(x.x >> 16);
      lo.z = e4m3x2_to_half2(x.y & 0xffff);
      lo.w = e4m3x2_to_half2(x.y >> 16);
      hi.x = e4m3x2_to_half2(x.z & 0xffff);
      hi.y = e4m3x2_to_half2(x.z >> 16);
      hi.z = e4m3x2_to_half2(x.w & 0xffff);
      hi.w = e4m3x2_to_half2(x.w >> 16);
      // lanes of odd panels write their upper half first: eight lanes of a row then fill a row
      const bool odd = lane % Loader::CPR * 2 >> 3 & 1;
      sts128(a ^ (odd ? 16 : 0), odd ? hi : lo);
      sts128(a ^ (odd ? 0 : 16), odd ? lo : hi);
    }
    L.landed(n);
    ++done;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ queries
// A tensor copy per panel brings 128 / G tokens with the G heads of the KV head, token after token
// (those past the item's rows are other sequences', or zeros behind the last one: rows nobody reads).
// bf16 queries of an fp8 cache are then rounded to fp16 in place. Spread items have smaller copies, four
// of them where the products read the tile (at head_dim 256 its rows go to tensor memory first).
template <typename C, typename T, int D>
__device__ __forceinline__ void query_role(const AttendParams& p, const AttendMaps& maps, AttendShared<C>& sh,
                                           uint8_t* tiles) {
  constexpr bool kConvert = !std::is_same_v<T, typename C::TM>;
  constexpr int kTimes = C::kQInTmem ? 1 : 4;  // a spread item's rows in the tile
  const int lane = threadIdx.x & 31;
  uint32_t count = 0, used = 0;
  Item it;
  while (next_item(sh, count, it)) {
    const int n = two_row_tiles<C>(p, it) ? 2 : 1;
    const bool spread = spread_rows<C>(p, it);
    const int times = spread && !kConvert ? kTimes : 1;
    const uint32_t bytes = (spread ? p.spread_tokens : p.tile_tokens) * p.G * D * 2 * times;
    for (int i = 0; i < n; ++i, ++used) {
      const int slot = used % C::NQ;
      const uint32_t lap = (used / C::NQ) & 1;
      PA_WAIT(sh.q_empty[slot], lap ^ 1);
      uint64_t* const bar = kConvert ? &sh.q_raw[slot] : &sh.q_full[slot];
      const uint32_t tile = smem_addr(tiles) + slot * C::QTILE;
      if (lane == 0) mbar_expect(smem_addr(bar), bytes);
      __syncwarp();
      if (lane < C::PANELS * times) {
        const int c = lane % C::PANELS;
        tensor_load3(tile + c * (128 * 128) + lane / C::PANELS * (32 * 128), spread ? &maps.q_spread : &maps.q,
                     smem_addr(bar), c * 64, it.kvh * p.G, it.tok + i * p.tile_tokens);
      }
      if constexpr (kConvert) {
        PA_WAIT(*bar, lap);
        const int tile_rows = p.tile_tokens * p.G, rows = min(tile_rows, it.rows - i * tile_rows);
        // loads of a lane on their way together (one by one, six packed prompts took 119 us instead of 113)
        constexpr int BATCH = 8;
        auto place = [&](int f) -> uint32_t {
          const int c = f % (D / 8);
          return tile + (c / 8) * (128 * 128) + f / (D / 8) * 128 + c % 8 * 16;
        };
        for (int f0 = lane; f0 < rows * (D / 8); f0 += 32 * BATCH) {
          uint4 x[BATCH];
#pragma unroll
          for (int j = 0; j < BATCH; ++j)
            if (f0 + 32 * j < rows * (D / 8)) x[j] = lds128(place(f0 + 32 * j));
#pragma unroll
          for (int j = 0; j < BATCH; ++j) {
            if (f0 + 32 * j >= rows * (D / 8)) break;
            uint32_t* w = reinterpret_cast<uint32_t*>(&x[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 y = unpack2<T>(w[i]);
              w[i] = pack2<typename C::TM>(y.x, y.y);
            }
            for (int k = 0; k < (spread ? kTimes : 1); ++k) sts128(place(f0 + 32 * j) + k * (32 * 128), x[j]);
          }
        }
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[slot]));
      }
    }
  }
}

// ------------------------------------------------------------------ products
// Steps of an item: one per token tile, or one per token tile and row tile. Products issued by one
// lane run in order, so that a score buffer is overwritten only after the weights in it are used.
template <typename C, int D>
__device__ __forceinline__ void product_role(const AttendParams& p, AttendShared<C>& sh, uint8_t* q_tiles,
                                             uint8_t* stages, uint32_t tmem_lane) {
  using TM = typename C::TM;
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, tmem_lane);  // uniform, as the compiler sees it
  const uint64_t by_k = operand_desc(16), by_n = operand_desc(C::TN * 128);
  const uint32_t q_lo = (uint32_t)by_k + (smem_addr(q_tiles) >> 4), k_lo = (uint32_t)by_k + (smem_addr(stages) >> 4),
                 v_lo = (uint32_t)by_n + (smem_addr(stages) >> 4);
  const uint32_t k_hi = (uint32_t)(by_k >> 32), v_hi = (uint32_t)(by_n >> 32);
  // a negative scale: the scores of -Q
  const uint32_t for_scores = mma_desc<TM>(C::TN, false) | (p.negate && !C::kQInTmem ? kNegateA : 0u);
  constexpr uint32_t kForValues = mma_desc<TM>(D, true);
  const uint32_t on = elected();
  uint32_t count = 0, used = 0;  // items, query tiles
  uint32_t stage = 0, lap = 0;   // of the next K or V tile
  uint32_t weights[2] = {0, 0};  // steps that used each score buffer
  Item it;
  auto next_tile = [&](uint32_t& which) -> bool {
    which = stage;
    if (!wait_for(smem_addr(&sh.kv_full[stage]), lap, &sh.give_up)) return false;
    if (++stage == C::NS) {
      stage = 0;
      lap ^= 1;
    }
    return true;
  };
  while (next_item(sh, count, it)) {
    const int tiles = __reduce_max_sync(0xffffffffu, it.tiles);
    const int dup = __any_sync(0xffffffffu, two_row_tiles<C>(p, it)) ? 1 : 0;
    const int steps = tiles << dup;
    const int spread = __any_sync(0xffffffffu, spread_rows<C>(p, it));
    const uint32_t q0 = used % C::NQ, q1 = (used + dup) % C::NQ;
    if constexpr (C::kQInTmem) {
      PA_WAIT(sh.q_tmem, used & 1);
    } else {
      for (int i = 0; i <= dup; ++i) PA_WAIT(sh.q_full[(used + i) % C::NQ], ((used + i) / C::NQ) & 1);
    }
    used += 1 + dup;
    uint32_t k_stage = 0, v_stage = 0;
    auto scores = [&](int i) -> bool {  // step i: S = Q K^T
      if (!(i & dup) && !next_tile(k_stage)) return false;
      tc_fence_after();
      const uint32_t q_tile = i & dup ? q1 : q0;
      const uint32_t a = q_lo + q_tile * (C::QTILE >> 4), b = k_lo + k_stage * (C::STAGE >> 4);
      const uint32_t d = tmem + C::S_COL + (i & 1) * C::TN;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t bk = b + (((kk / 4) * (C::TN * 128) + (kk % 4) * 32) >> 4);
        if constexpr (C::kQInTmem)
          mma_ts(on, d, tmem + C::Q_COL + kk * 8, bk, k_hi, for_scores, kk > 0);
        else
          mma_ss(on, d, a + (((kk / 4) * (128 * 128) + (kk % 4) * 32) >> 4), k_hi, bk, k_hi, for_scores, kk > 0);
      }
      mma_commit(on, smem_addr(&sh.s_full[i & 1]));
      if (dup == 0 || (i & 1)) mma_commit(on, smem_addr(&sh.kv_empty[k_stage]));
      if (!C::kQInTmem && i >= steps - 1 - dup && !spread)  // its row tile's last
        mma_commit(on, smem_addr(&sh.q_empty[q_tile]));
      return true;
    };
    for (int i = 0; i < 2 && i < steps; ++i)
      if (!scores(i)) return;
    for (int i = 0; i < steps; ++i) {
      const int buf = i & 1, group = C::NWG == 2 ? buf : 0;
      if (!(i & dup) && !next_tile(v_stage)) return;
      PA_WAIT(sh.p_full[buf], (buf ? weights[1] : weights[0]) & 1);
      if (buf)
        ++weights[1];
      else
        ++weights[0];
      tc_fence_after();
      // O += P V
      const uint32_t a = tmem + C::S_COL + buf * C::TN, b = v_lo + v_stage * (C::STAGE >> 4);
      const uint32_t d = tmem + C::O_COL + group * D;
      mma_ts(on, d, a, b, v_hi, kForValues, i >= C::NWG);
#pragma unroll
      for (int kk = 1; kk < C::TN / 16; ++kk) mma_ts(on, d, a + kk * 8, b + kk * (2048 >> 4), v_hi, kForValues, true);
      mma_commit(on, smem_addr(&sh.pv_done[buf]));
      if (dup == 0 || (i & 1)) mma_commit(on, smem_addr(&sh.kv_empty[v_stage]));
      if (i + 2 < steps && !scores(i + 2)) return;
    }
  }
}

// ------------------------------------------------------------------ softmax
__host__ __device__ constexpr int ilog2(int x) { return x <= 1 ? 0 : 1 + ilog2(x / 2); }

// All softmax warps of the CTA meet. Bit 2 of parities is the barrier's.
template <typename C>
__device__ __forceinline__ bool meet(AttendShared<C>& sh, uint32_t& parities) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&sh.pair));
  if (!wait_for(smem_addr(&sh.pair), parities >> 2 & 1, &sh.give_up)) return false;
  parities ^= 4;
  tc_fence_after();
  return true;
}

// The end of the context that query row r of an item sees, of a live row: causal among the new rows.
__device__ __forceinline__ int seen_to(const AttendParams& p, const Item& it, int r) {
  if (!p.shared) return it.hi;
  const int tok = it.tok + div_group(p, r), b = p.R == 1 ? tok : tok / p.R;
  const int L = it.of_prefix ? clamp_len(p, b) : it.hi;  // the end of its own segment
  return min(it.hi, L - p.R + 1 + (tok - b * p.R));
}

// A spread item: a thread has a row's scores over a quarter of each tile of its group.
template <typename C, typename T, int D, typename Next>
__device__ __forceinline__ bool spread_item(const AttendParams& p, AttendShared<C>& sh, const Item& it, uint8_t* q_tiles,
                                          uint32_t tmem, uint32_t& parities, const Next& place_next) {
  using TM = typename C::TM;
  static_assert(!C::kSpread || C::KVB == 1, "V rows outside the context are zeros already");
  constexpr int N = C::TN / 4;      // the warp's columns of a tile
  constexpr int HALF = D / C::NWG;  // the group's columns of the output
  constexpr int W = 16;
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 7, at = threadIdx.x & 127, quarter = at >> 5;
  const uint32_t lanes = (uint32_t)quarter << 21;
  const uint32_t own_o = tmem + C::O_COL + group * D + lanes, other_o = tmem + C::O_COL + (group ^ 1) * D + lanes;
  const float sl2 = p.scale_log2;
  const bool live = lane < it.rows;
  const int end = live ? seen_to(p, it, lane) : it.lo;
  float ref = -INFINITY, sum = 0.f;
  int i = C::NWG == 2 ? group : 0;
  const bool any = i < it.tiles;
  for (; i < it.tiles; i += C::NWG) {
    const int buf = i & 1;
    const uint32_t s_at = tmem + C::S_COL + buf * C::TN + lanes;
    if (!wait_for(smem_addr(&sh.s_full[buf]), (parities >> buf) & 1, &sh.give_up)) return false;
    parities ^= 1u << buf;
    tc_fence_after();
    uint32_t x[N];
    tmem_load(x, s_at + quarter * N);
    tmem_loaded(x);
    const uint32_t none[N / 2] = {};
#pragma unroll
    for (int k = 1; k < 4; ++k) tmem_store(s_at + (quarter + k) % 4 * (N / 2), none);
    const int t0 = it.t0 + i * C::TN + quarter * N, c0 = it.lo - t0, c1 = end - t0;  // columns [c0, c1) are seen
    if (!__all_sync(0xffffffffu, !live || (c0 <= 0 && c1 >= N))) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j < c0 || j >= c1) x[j] = 0xff800000u;
    }
    float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      most[0] = fmaxf(fmaxf(most[0], __uint_as_float(x[j])), __uint_as_float(x[j + 1]));
      most[1] = fmaxf(fmaxf(most[1], __uint_as_float(x[j + 2])), __uint_as_float(x[j + 3]));
    }
    const float top = fmaxf(most[0], most[1]) * sl2 - C::kLift;
    const bool raise = live && top > ref + C::kSlack;
    if (__any_sync(0xffffffffu, raise)) {
      const float now = raise ? top : ref;
      const float f = now == -INFINITY ? 1.f : exp2_approx(ref - now);
      ref = now;
      sum *= f;
      if (i >= C::NWG) {  // the accumulator of the steps before
        const int last = C::NWG == 2 ? buf : buf ^ 1;
        if (!wait_for(smem_addr(&sh.pv_done[last]), (parities >> last & 1) ^ (C::NWG == 2 ? 0 : 1), &sh.give_up))
          return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += W) {
          uint32_t o[W];
          tmem_load(o, own_o + c);
          tmem_loaded(o);
#pragma unroll
          for (int j = 0; j < W; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_store(own_o + c, o);
        }
      }
    }
    const float sub = ref == -INFINITY ? 0.f : -ref;
    const float2 by = make_float2(sl2, sl2), plus = make_float2(sub, sub);
    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t w[N / 2];
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      float2 e = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), by, plus);
      e.x = exp2_approx(e.x);
      e.y = exp2_approx(e.y);
      part[(j / 2) & 1] = add2(part[(j / 2) & 1], e);
      w[j / 2] = pack2<TM>(e.x, e.y);
    }
    tmem_store(s_at + quarter * (N / 2), w);
    const float2 both = add2(part[0], part[1]);
    sum += both.x + both.y;
    tmem_stored();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[buf]));
  }

  if (!place_next()) return false;  // while the last product runs

  // ---- the states of a row, of four warps in each group
  if (any) {
    const int last = C::NWG == 2 ? group : (it.tiles - 1) & 1;
    if (!wait_for(smem_addr(&sh.pv_done[last]), (parities >> last & 1) ^ 1, &sh.give_up)) return false;
  }
  sh.state[group][at] = make_float2(ref, sum);
  if (!meet(sh, parities)) return false;
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4 * C::NWG; ++k) m = fmaxf(m, sh.state[k >> 2][(k & 3) * 32 + lane].x);
  auto factor = [&](float of) { return of == -INFINITY ? 0.f : exp2_approx(of - m); };
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < 4 * C::NWG; ++k) {
    const float2 y = sh.state[k >> 2][(k & 3) * 32 + lane];
    sum += y.y * factor(y.x);
  }
  const float f_own = factor(ref), f_other = C::NWG == 2 ? factor(sh.state[group ^ 1][at].x) : 0.f;

  // ---- the rows: the warps' parts are added through the item's query tile, which no product reads any
  // more: [warp][row][column], the group's columns or half of them, 16-byte chunks swizzled by the row
  const bool whole = it.dest == kDirect, by_row = it.dest == kRowShared || it.dest == kRowOwn;
  const float mul = whole ? (sum == 0.f ? 0.f : p.v_scale / sum) : p.v_scale;
  const size_t first_slot = ((size_t)blockIdx.x * 2 + (it.dest == kSlotFirst ? 1 : 0)) * p.slot_rows;
  auto of_call = [&](int r) {  // the row's place among the call's
    const int tok = div_group(p, r);
    return (size_t)(it.tok + tok) * p.Hq + it.kvh * p.G + r - tok * p.G;
  };
  auto of_partials = [&](int r) {
    return by_row ? (it.dest == kRowOwn ? (size_t)p.T * p.Hq : 0) + of_call(r) : first_slot + r;
  };
  if (!whole && live && group == 0 && quarter == 0)
    (by_row ? p.row_ml : p.slot_ml)[of_partials(lane)] = make_float2(m, sum);
  static_assert(C::NWG * 4 * 16 * HALF * 4 == C::QTILE, "16 rows of all columns");
  const bool few = it.rows <= 16;
  const int room = few ? 16 : 32, cols = few ? HALF : HALF / 2;
  const uint32_t area = smem_addr(q_tiles) + (C::kQInTmem ? 0 : parities >> 3 & 1) * C::QTILE + group * (C::QTILE / C::NWG);
  for (int c0 = 0; c0 < HALF; c0 += cols) {
    if (c0 > 0 && !meet(sh, parities)) return false;
#pragma unroll 1
    for (int c = 0; c < cols; c += W) {
      uint32_t o[W], o2[W];
      tmem_load(o, own_o + group * HALF + c0 + c);
      if constexpr (C::NWG == 2) {
        tmem_load(o2, other_o + group * HALF + c0 + c);
        tmem_loaded(o2);
      }
      tmem_loaded(o);
      const uint32_t to = area + (quarter * room + lane) * cols * 4;
#pragma unroll
      for (int j = 0; j < W; j += 4) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // an accumulator that saw no token may hold anything
          float a = f_own > 0.f ? __uint_as_float(o[j + k]) * f_own : 0.f;
          if constexpr (C::NWG == 2) a += f_other > 0.f ? __uint_as_float(o2[j + k]) * f_other : 0.f;
          w[k] = __float_as_uint(a * mul);
        }
        if (live) sts128(to + (((c + j) / 4 ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    if (!meet(sh, parities)) return false;
    const int shift = few ? ilog2(HALF / 8) : ilog2(HALF / 16);
    for (int u = at; u < it.rows << shift; u += 128) {  // 8 columns of a row
      const int r = u >> shift, c = u - (r << shift);
      float e[8] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = lds128(area + (k * room + r) * cols * 4 + ((2 * c + h ^ (r & 7)) << 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) e[4 * h + j] += __uint_as_float(word_of(x, j));
        }
      const int column = group * HALF + c0 + 8 * c;
      if (whole) {
        *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + of_call(r) * D + column) =
            make_uint4(pack2<T>(e[0], e[1]), pack2<T>(e[2], e[3]), pack2<T>(e[4], e[5]), pack2<T>(e[6], e[7]));
      } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(e[j]);
        store32((by_row ? p.row_acc : p.slot_acc) + of_partials(r) * D + column, w);
      }
    }
  }
  async_proxy_fence();  // the next copy of queries comes after these reads
  // accumulators, states and the tile are read before the next ones come
  if (!meet(sh, parities)) return false;
  if (!C::kQInTmem && threadIdx.x == 0) mbar_arrive(smem_addr(&sh.q_empty[parities >> 3 & 1]));
  return true;
}

// One thread per row of a row tile.
template <typename C, typename T, int D, bool ZERO_V>
__device__ __forceinline__ void softmax_role(const AttendParams& p, AttendShared<C>& sh, uint8_t* q_tiles,
                                             uint8_t* stages, uint32_t tmem) {
  using TM = typename C::TM;
  constexpr int W = C::CHUNK, NC = C::TN / W;
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 7, at = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;  // 32 (warp % 4) in the upper half
  const uint32_t own_o = tmem + C::O_COL + group * D + lanes;
  const float sl2 = p.scale_log2;
  // Registers are short here (a spilled one comes back from L2): the item stays in its slot of the
  // ring, and what is needed of it after its steps is read again; parities are bits of one word, 0 and
  // 1 the score buffers', 2 the pair barrier's; 3 is the query tile of the next item of one row tile.
  uint32_t count = 0, parities = 0, tiles_before = 0;
  // The queries of item n, if there is one, into tensor memory: when no product reads those of the item
  // before any more. A negative scale negates them.
  auto place_queries = [&](uint32_t n) -> bool {
    if (!wait_for(smem_addr(&sh.item_full[n % C::ITEMS]), (n / C::ITEMS) & 1, &sh.give_up)) return false;
    if (sh.items[n % C::ITEMS].tiles == 0) return true;
    if (!wait_for(smem_addr(&sh.q_full[0]), n & 1, &sh.give_up)) return false;
    const uint32_t row = smem_addr(q_tiles) + (spread_rows<C>(p, sh.items[n % C::ITEMS]) ? lane : at) * 128, sign = p.negate ? 0x80008000u : 0u;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 8; c += 4) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = lds128(row + (c >> 3) * (128 * 128) + ((((c & 7) + j) ^ (at & 7)) << 4));
        w[4 * j] = x.x ^ sign;
        w[4 * j + 1] = x.y ^ sign;
        w[4 * j + 2] = x.z ^ sign;
        w[4 * j + 3] = x.w ^ sign;
      }
      tmem_store(tmem + C::Q_COL + 4 * c + lanes, w);
    }
    tmem_stored();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_addr(&sh.q_tmem));
      if (!C::kSpread) mbar_arrive(smem_addr(&sh.q_empty[0]));
    }
    return true;
  };
  auto end_item = [&](bool two) {
    if (!two) parities ^= 8;
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_addr(&sh.item_empty[count % C::ITEMS]));
      if (C::kQInTmem && C::kSpread) mbar_arrive(smem_addr(&sh.q_empty[0]));
    }
  };
  if constexpr (C::kQInTmem) {
    if (!place_queries(0)) return;
    // later ones when the item before is out, which may need the tile to add its rows' parts
    if (C::kSpread && lane == 0) mbar_arrive(smem_addr(&sh.q_empty[0]));
  }
  for (;; ++count) {
    const Item& it = sh.items[count % C::ITEMS];
    PA_WAIT(sh.item_full[count % C::ITEMS], (count / C::ITEMS) & 1);
    const int tiles = it.tiles;
    if (tiles == 0) return;
    if constexpr (C::kSpread) {
      if (spread_rows<C>(p, it)) {
        if (!spread_item<C, T, D>(p, sh, it, q_tiles, tmem, parities,
                                  [&] { return !C::kQInTmem || place_queries(count + 1); }))
          return;
        end_item(false);
        continue;
      }
    }
    const int tile_rows = p.tile_tokens * p.G;
    const bool two = two_row_tiles<C>(p, it);
    const int dup = two ? 1 : 0;
    const int r = (two ? group * tile_rows : 0) + at;  // the item's row of this thread
    const bool live = at < tile_rows && r < it.rows;
    const bool warp_live = at - lane < tile_rows && r - lane < it.rows;
    const int lo = it.lo;
    const int end = live ? seen_to(p, it, r) : lo;  // this row sees tokens in [lo, end)
    float ref = -INFINITY, sum = 0.f;
    int t0 = it.t0;
    int i = C::NWG == 2 ? group : 0;
    const bool any = i < tiles << dup;  // a step for this group
    if (C::NWG == 2 && !dup) t0 += group * C::TN;
    for (; i < tiles << dup; i += C::NWG, t0 += C::NWG == 2 && !dup ? 2 * C::TN : C::TN) {
      const int buf = C::NWG == 2 ? group : i & 1;
      const uint32_t s_at = tmem + C::S_COL + buf * C::TN + lanes;
      PA_WAIT(sh.s_full[buf], (parities >> buf) & 1);
      parities ^= 1u << buf;
      if (warp_live) {
        tc_fence_after();
        const int c0 = lo - t0, c1 = end - t0;  // columns [c0, c1) are seen
        uint32_t x[2][W];
        if (!__all_sync(0xffffffffu, !live || (c0 <= 0 && c1 >= C::TN))) {
          // scores of tokens that the row does not see become -inf, whatever they are
          const int all = __reduce_min_sync(0xffffffffu, live ? c1 : C::TN), none = __reduce_max_sync(0xffffffffu, c1);
#pragma unroll 1
          for (int c = 0; c < C::TN; c += W) {
            if (c >= c0 && c + W <= all) continue;
            if (c >= none) {  // not read either
#pragma unroll
              for (int j = 0; j < W; ++j) x[0][j] = 0xff800000u;
              tmem_store(s_at + c, x[0]);
              continue;
            }
            tmem_load(x[0], s_at + c);
            tmem_loaded(x[0]);
#pragma unroll
            for (int j = 0; j < W; ++j)
              if (c + j < c0 || c + j >= c1) x[0][j] = 0xff800000u;
            tmem_store(s_at + c, x[0]);
          }
          tmem_stored();
        }
        // the largest score, scaled
        float most[2] = {-INFINITY, -INFINITY};
        tmem_load(x[0], s_at);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t(&y)[W] = x[c & 1];
          tmem_loaded(y);
          tmem_load(x[(c + 1) & 1], s_at + W * ((c + 1) % NC));  // the last one: the first columns again
#pragma unroll
          for (int j = 0; j < W; j += 4) {
            most[0] = fmaxf(fmaxf(most[0], __uint_as_float(y[j])), __uint_as_float(y[j + 1]));
            most[1] = fmaxf(fmaxf(most[1], __uint_as_float(y[j + 2])), __uint_as_float(y[j + 3]));
          }
        }
        const float top = fmaxf(most[0], most[1]) * sl2 - C::kLift;
        const bool raise = top > ref + C::kSlack;
        if (__any_sync(0xffffffffu, raise)) {
          const float now = raise ? top : ref;
          const float f = now == -INFINITY ? 1.f : exp2_approx(ref - now);
          ref = now;
          sum *= f;
          if (i >= C::NWG) {  // the accumulator of the steps before
            const int last = C::NWG == 2 ? buf : buf ^ 1;
            PA_WAIT(sh.pv_done[last], (parities >> last & 1) ^ (C::NWG == 2 ? 0 : 1));
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += W) {
              uint32_t o[W];
              tmem_load(o, own_o + c);
              tmem_loaded(o);
#pragma unroll
              for (int j = 0; j < W; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_store(own_o + c, o);
            }
            tmem_load(x[NC & 1], s_at);  // read again rather than kept across the wait
          }
        }
        const float sub = ref == -INFINITY ? 0.f : -ref;
        const float2 by = make_float2(sl2, sl2), plus = make_float2(sub, sub);
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          uint32_t(&y)[W] = x[(NC + c) & 1];
          tmem_loaded(y);
          if (c + 1 < NC) tmem_load(x[(NC + c + 1) & 1], s_at + W * (c + 1));
#pragma unroll
          for (int k = 0; k < W; k += 16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float2 e = fma2(make_float2(__uint_as_float(y[k + j]), __uint_as_float(y[k + j + 1])), by, plus);
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              part[(j / 2) & 1] = add2(part[(j / 2) & 1], e);
              w[j / 2] = pack2<TM>(e.x, e.y);
            }
            // over columns of scores that are in registers already
            tmem_store(s_at + (W * c + k) / 2, w);
          }
        }
        const float2 both = add2(part[0], part[1]);
        sum += both.x + both.y;
        tmem_stored();
      }
      if constexpr (ZERO_V) {
        // V rows outside the context hold whatever the cache or an earlier tile left: zeros there,
        // so that weights of 0 meet 0. (Eight lanes a row: with a row for each lane, eight lanes met in a bank,
        // and six packed prompts of 128-token tiles took 89 us instead of 84.)
        if ((t0 < lo || t0 + C::TN > it.hi) && !(dup && group)) {
          const uint32_t n = tiles_before + place_v(i >> dup, lead_of<C>(p, it), tiles);
          PA_WAIT(sh.kv_full[n % C::NS], (n / C::NS) & 1);
          const uint32_t tile = smem_addr(stages) + (n % C::NS) * C::STAGE + at * 16;
          const int from = lo - t0 - (at >> 3), to = it.hi - t0 - (at >> 3);
#pragma unroll
          for (int row = 0; row < C::TN; row += 16)
            if (row < from || row >= to)
#pragma unroll
              for (int c = 0; c < C::PANELS; ++c) sts128_zero(tile + c * (C::TN * 128) + row * 128);
          async_proxy_fence();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[buf]));
    }
    tiles_before += 2 * tiles;
    if constexpr (C::kQInTmem)  // while the last product runs
      if (!place_queries(count + 1)) return;

    // ---- the item's rows: O / sum, or (reference, sum, O) of a piece
    if (any) {
      const int last = C::NWG == 2 ? group : (tiles - 1) & 1;
      PA_WAIT(sh.pv_done[last], (parities >> last & 1) ^ 1);
    }
    tc_fence_after();
    const bool joint = C::NWG == 2 && !two;  // two states of the same rows
    float f_own = 1.f, f_other = 0.f;
    if constexpr (C::NWG == 2) {
      if (joint) {
        sh.state[group][at] = make_float2(ref, sum);
        if (!meet(sh, parities)) return;
        const float2 other = sh.state[group ^ 1][at];
        const float m = fmaxf(ref, other.x);
        f_own = ref == -INFINITY ? 0.f : exp2_approx(ref - m);
        f_other = other.x == -INFINITY ? 0.f : exp2_approx(other.x - m);
        sum = sum * f_own + other.y * f_other;
        ref = m;
      }
    }
    if (warp_live) {
      const bool whole = it.dest == kDirect;
      // a row that sees no token is zero (and whatever its accumulator holds); one with a NaN is NaN
      const float mul = whole ? (sum == 0.f ? 0.f : p.v_scale / sum) : p.v_scale;
      const int tok = it.tok + div_group(p, r), head = it.kvh * p.G + r - div_group(p, r) * p.G;
      const size_t row = live ? (size_t)tok * p.Hq + head : 0;
      size_t part = 0;  // row of the partials
      float* acc = nullptr;
      float2* ml = nullptr;
      if (!whole) {
        if (it.dest == kRowShared || it.dest == kRowOwn) {
          part = (it.dest == kRowOwn ? (size_t)p.T * p.Hq : 0) + row;
          acc = p.row_acc;
          ml = p.row_ml;
        } else {
          part = ((size_t)blockIdx.x * 2 + (it.dest == kSlotFirst ? 1 : 0)) * p.slot_rows + r;
          acc = p.slot_acc;
          ml = p.slot_ml;
        }
        if (live && !(joint && group)) ml[part] = make_float2(ref, sum);
      }
      // joint groups take half of the columns each
      const int from = joint ? group * (D / 2) : 0, to = joint ? from + D / 2 : D;
      const uint32_t other_o = tmem + C::O_COL + (group ^ 1) * D + lanes;
#pragma unroll 1
      for (int c = from; c < to; c += W) {
        uint32_t o[W];
        tmem_load(o, own_o + c);
        tmem_loaded(o);
        if (joint) {
          uint32_t o2[W];
          tmem_load(o2, other_o + c);
          tmem_loaded(o2);
#pragma unroll
          for (int j = 0; j < W; ++j) {  // an accumulator that saw no token may hold anything
            const float a = f_own > 0.f ? __uint_as_float(o[j]) * f_own : 0.f;
            const float b = f_other > 0.f ? __uint_as_float(o2[j]) * f_other : 0.f;
            o[j] = __float_as_uint(a + b);
          }
        }
        if (live) {
          if (whole) {
            T* dst = static_cast<T*>(p.out) + row * D + c;
#pragma unroll
            for (int j = 0; j < W; j += 16) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float a = __uint_as_float(o[j + 2 * i]), b = __uint_as_float(o[j + 2 * i + 1]);
                w[i] = pack2<T>(sum == 0.f ? 0.f : a * mul, sum == 0.f ? 0.f : b * mul);
              }
              if (p.out_wide) {
                store32(dst + j, w);
              } else {
                *reinterpret_cast<uint4*>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(dst + j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          } else {
            float* dst = acc + part * D + c;
#pragma unroll
            for (int j = 0; j < W; j += 8) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(o[j + i]) * mul);
              store32(dst + j, w);
            }
          }
        }
      }
    }
    if constexpr (C::NWG == 2)
      if (joint && !meet(sh, parities)) return;  // both accumulators are read before either group's next weights
    end_item(two);
  }
}

// ------------------------------------------------------------------ kernel
template <typename T, int D, AttendLoad LOAD>
__global__ void __launch_bounds__(AttendCfg<T, D, LOAD>::THREADS, 1)
    attend_kernel(const AttendParams p, const __grid_constant__ AttendMaps maps) {
  using C = AttendCfg<T, D, LOAD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023) {  // the swizzle counts on it
    pdl_wait();
    if (threadIdx.x == 0) {
      atomicOr(p.err, PA_DEVERR_COPY);
      p.split[blockIdx.x].pieces = 0;
      if (blockIdx.x == 0) p.plan[0] = 0;  // nothing to merge
    }
    return;
  }
  uint8_t *q_tiles = smem, *stages = smem + C::OFF_STAGE, *raw = smem + C::OFF_RAW;
  AttendShared<C>& sh = *reinterpret_cast<AttendShared<C>*>(smem + C::OFF_SYNC);
  static_assert(sizeof(AttendShared<C>) <= C::SYNC_BYTES, "barriers and items");
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    auto init = [](uint64_t* bars, int n, int count) {
      for (int i = 0; i < n; ++i) mbar_init_count(smem_addr(bars + i), count);
    };
    init(sh.kv_full, C::NS, LOAD == kLoadTensor ? 2 : 4);
    init(sh.kv_empty, C::NS, 1);
    init(sh.q_raw, C::NQ, 1);
    init(sh.q_full, C::NQ, 1);
    init(sh.q_empty, C::NQ, C::kQInTmem ? 4 : 1);
    init(&sh.q_tmem, 1, 4);
    init(sh.s_full, 2, 1);
    init(sh.p_full, 2, 4);
    init(sh.pv_done, 2, 1);
    init(sh.item_full, C::ITEMS, 1);
    init(sh.item_empty, C::ITEMS, C::READERS);
    init(&sh.pair, 1, C::NSW);
    init(&sh.drain, 1, 1);
    sh.give_up.now = 0;
    sh.give_up.after = kGiveUpAfter;
    mbar_init_fence();
    tensor_prefetch(&maps.q);
    if constexpr (LOAD == kLoadTensor) {
      tensor_prefetch(&maps.k);
      tensor_prefetch(&maps.v);
    }
  }
  if (warp == C::W_MMA) tmem_alloc(smem_addr(&sh.tmem));
  tc_fence_before();
  // inputs may come from the kernel before in the stream
  pdl_wait();
  plan_work<C, D>(p, sh, reinterpret_cast<Group*>(stages));
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp < C::NSW)
    softmax_role<C, T, D, LOAD == kLoadTensor>(p, sh, q_tiles, stages, tmem);
  else if (warp == C::W_MMA)
    product_role<C, D>(p, sh, q_tiles, stages, tmem);
  else if (warp == C::W_PLAN)
    plan_role<C, D>(p, sh);
  else if (warp == C::W_Q)
    query_role<C, T, D>(p, maps, sh, q_tiles);
  else if constexpr (LOAD == kLoadTensor)
    tensor_load_role<C, D>(p, warp < C::W_LOAD + 2 ? &maps.k : &maps.v, warp < C::W_LOAD + 2,
                           (warp - C::W_LOAD) & 1, sh, stages);
  else if constexpr (LOAD == kLoadFp8)
    fp8_load_role<C, D>(p, warp < C::W_LOAD + 4, (warp - C::W_LOAD) & 3, sh, stages, raw);
  else
    row_load_role<C, D>(p, warp < C::W_LOAD + 4, (warp - C::W_LOAD) & 3, sh, stages);

  __syncwarp();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (sh.give_up.now) {
    // some wait took too long: copies and products in flight are waited for, with a limit,
    // before the CTA gives its memory back
    if (threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_COPY);
    if (warp == C::W_MMA) {
      mma_commit(elected(), smem_addr(&sh.drain));
      __syncwarp();
    }
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 100000000ull && !(warp == C::W_MMA && mbar_try(smem_addr(&sh.drain), 0)))
      ;
    __syncthreads();
  }
  tc_fence_after();
  if (warp == C::W_MMA) tmem_free(tmem);
}

// ------------------------------------------------------------------ merge
// The pieces of a row, weighed by 2^(reference - largest), their sums and outputs added in order; a
// warp per row. at(i) gives the addresses of piece i's (reference, sum) and output. BATCH pieces at
// a time, their states and outputs in one round trip.
template <int D>
struct Merged {
  static constexpr int V = D / 128;  // 16-byte vectors of a lane
  float top = -INFINITY, sum = 0.f;
  float4 v[V];
  __device__ Merged() {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  template <int BATCH, typename At>
  __device__ __forceinline__ void load(float2 (&x)[BATCH], float4 (&y)[BATCH][V], int first, int n, const At& at) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      x[i] = make_float2(-INFINITY, 0.f);
      if (first + i < n) {
        const float2* ml;
        const float* acc;
        at(first + i, &ml, &acc);
        x[i] = __ldcg(ml);
#pragma unroll
        for (int j = 0; j < V; ++j) y[i][j] = __ldcg(reinterpret_cast<const float4*>(acc + 128 * j + 4 * lane));
      }
    }
  }
  template <int BATCH>
  __device__ __forceinline__ void add(const float2 (&x)[BATCH], const float4 (&y)[BATCH][V]) {
    float most = top;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) most = fmaxf(most, x[i].x);
    const float f = top == -INFINITY ? 0.f : exp2_approx(top - most);
    top = most;
    sum *= f;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = make_float4(v[j].x * f, v[j].y * f, v[j].z * f, v[j].w * f);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (x[i].y == 0.f) continue;  // none, or it saw no token of the row: its output may be anything
      const float w = exp2_approx(x[i].x - top);
      sum += w * x[i].y;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j].x += w * y[i][j].x;
        v[j].y += w * y[i][j].y;
        v[j].z += w * y[i][j].z;
        v[j].w += w * y[i][j].w;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* out) const {
    const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < V; ++j)
      *reinterpret_cast<uint2*>(out + 128 * j + 4 * (threadIdx.x & 31)) =
          make_uint2(pack2<T>(v[j].x * f, v[j].y * f), pack2<T>(v[j].z * f, v[j].w * f));
  }
};
template <typename T, int D, int BATCH, typename At>
__device__ __forceinline__ void merge_pieces(int n, const At& at, T* out) {
  Merged<D> m;
  for (int first = 0; first < n; first += BATCH) {
    float2 x[BATCH];
    float4 y[BATCH][Merged<D>::V];
    m.load(x, y, first, n, at);
    m.add(x, y);
  }
  m.store(out);
}

// Rows with one context: grid (CTAs, parts of an item's rows), the item that CTA blockIdx.x begins and
// others end. A warp takes ROWS rows at a time: one where items have few rows but many pieces, two, their
// first pieces loaded together, where they have many, and then enough rows that every block is resident
// (each starts with a round trip to find its item).
constexpr int kMergeParts = 4;
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(256) merge_items_kernel(const AttendParams p) {
  constexpr int BATCH = ROWS == 1 ? (D == 128 ? 8 : 4) : 2;
  const int c = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int4 x = __ldcg(reinterpret_cast<const int4*>(p.split + c));
  const SplitItem it{x.x, x.y, x.z, x.w};
  if (it.pieces == 0) return;
  for (int r0 = blockIdx.y * 8 * ROWS + (threadIdx.x >> 5); r0 < it.rows; r0 += gridDim.y * 8 * ROWS) {
    Merged<D> m[ROWS];
    for (int first = 0; first < it.pieces; first += BATCH) {
      float2 ml[ROWS][BATCH];
      float4 acc[ROWS][BATCH][Merged<D>::V];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int r = r0 + 8 * k;
        m[k].load(ml[k], acc[k], first, r < it.rows ? it.pieces : 0, [&](int i, const float2** a, const float** b) {
          const size_t at = ((size_t)(c + i) * 2 + (i == 0 ? 1 : 0)) * p.slot_rows + r;
          *a = p.slot_ml + at;
          *b = p.slot_acc + at * D;
        });
      }
#pragma unroll
      for (int k = 0; k < ROWS; ++k) m[k].add(ml[k], acc[k]);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int r = r0 + 8 * k, tok = div_group(p, r);
      if (r < it.rows)
        m[k].store(static_cast<T*>(p.out) + ((size_t)(it.tok + tok) * p.Hq + it.kvh * p.G + r - tok * p.G) * D);
    }
  }
}

// Rows with two contexts, and others: every row finds its pieces.
template <typename T, int D>
__global__ void __launch_bounds__(256) merge_rows_kernel(const AttendParams p) {
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (row >= (long long)p.T * p.Hq) return;
  const int tok = (int)(row / p.Hq), head = (int)(row - (long long)tok * p.Hq);
  const int kvh = head / p.G, b = p.R == 1 ? tok : tok / p.R;
  auto record = [&](int s) -> SegmentRecord {
    union {
      int4 x[2];
      SegmentRecord r;
    } y;
    y.x[0] = __ldcg(reinterpret_cast<const int4*>(p.segments + s));
    y.x[1] = __ldcg(reinterpret_cast<const int4*>(p.segments + s) + 1);
    return y.r;
  };
  const long long per = __ldcg(p.plan);
  if (per == 0) return;
  const SegmentRecord own = record(p.N + b);
  // the pieces of this row in a segment: CTAs from .. to
  struct Pieces {
    int from, to, r;  // r: the row in the item
  };
  auto pieces_of = [&](const SegmentRecord& g) -> Pieces {
    const Shape z = shape_of<D>(p, g.tiles, g.n);
    const int tokens = p.tile_tokens * attend_row_tiles(D), i = (tok - g.tok0) / tokens;
    const long long u = g.first + units_before(z, kvh, i);
    Pieces y;
    y.from = (int)quotient(u, per);
    y.to = (int)quotient(u + (long long)(i == z.items - 1 ? z.last : z.full) * (z.tiles - 1), per);
    y.r = (tok - g.tok0 - i * tokens) * p.G + head - kvh * p.G;
    return y;
  };
  const Pieces po = pieces_of(own);
  if (own.group < 0 && po.from == po.to) return;  // written by the attention grid
  Pieces ps{0, -1, 0};
  if (own.group >= 0) ps = pieces_of(record(own.group));
  const int n_shared = ps.to - ps.from + 1, n = n_shared + po.to - po.from + 1;
  merge_pieces<T, D, D == 128 ? 8 : 4>(
      n,
      [&](int i, const float2** ml, const float** acc) {
        const bool mine = i >= n_shared;
        const int from = mine ? po.from : ps.from, c = mine ? from + i - n_shared : from + i;
        if (from == (mine ? po.to : ps.to)) {  // a whole item
          const size_t k = (mine ? (size_t)p.T * p.Hq : 0) + row;
          *ml = p.row_ml + k;
          *acc = p.row_acc + k * D;
        } else {
          const size_t k = ((size_t)c * 2 + (c == from ? 1 : 0)) * p.slot_rows + (mine ? po.r : ps.r);
          *ml = p.slot_ml + k;
          *acc = p.slot_acc + k * D;
        }
      },
      static_cast<T*>(p.out) + row * D);
}

// ------------------------------------------------------------------ launch
template <typename T, int D, AttendLoad LOAD>
cudaError_t launch_attend_load(const AttendParams& p, const AttendMaps& maps, cudaStream_t st) {
  using C = AttendCfg<T, D, LOAD>;
  auto kern = attend_kernel<T, D, LOAD>;
  // the opt-in to this much shared memory is per device
  static unsigned long long done_mask = 0ull;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, bit, __ATOMIC_ACQ_REL);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  e = cudaLaunchKernelEx(&cfg, kern, p, maps);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (!p.shared) {
    const int parts = (p.slot_rows + 7) / 8;
    cfg.gridDim = dim3(p.ctas, p.slot_rows > 64 ? kMergeParts : parts);
    return p.slot_rows > 64 ? cudaLaunchKernelEx(&cfg, merge_items_kernel<T, D, 2>, p)
                            : cudaLaunchKernelEx(&cfg, merge_items_kernel<T, D, 1>, p);
  }
  cfg.gridDim = dim3((unsigned)(((long long)p.T * p.Hq + 7) / 8));
  return cudaLaunchKernelEx(&cfg, merge_rows_kernel<T, D>, p);
}
template <typename T, int D>
cudaError_t launch_attend(const AttendParams& p, const AttendMaps& maps, AttendLoad load, cudaStream_t st) {
  return load == kLoadTensor ? launch_attend_load<T, D, kLoadTensor>(p, maps, st)
         : load == kLoad16   ? launch_attend_load<T, D, kLoad16>(p, maps, st)
                             : launch_attend_load<T, D, kLoadFp8>(p, maps, st);
}

}  // namespace pa
