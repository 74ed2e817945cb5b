// Decode arithmetic on 4-bit cache rows (layout: PA_INT4_ROW_BYTES in pa.h), per warp.
//
// With value = minimum + step * n (n = 0..15) per group g of 32 elements, a score is
//
//   q . k_t = sum_g step_tg (sum_{d in g} q_d n_td) + sum_g minimum_tg (sum_{d in g} q_d)
//
// and an output element d of group g is
//
//   sum_t p_t v_td = sum_t (p_t step_tg) n_td + sum_t p_t minimum_tg,
//
// so the codes themselves are MMA operands and no element is scaled on its own. The codes
// become fp16 without arithmetic: a nibble in the low mantissa bits of an fp16 word is the
// subnormal n * 2^-24 (bits 0-3) or n * 2^-20 (bits 4-7), which the tensor cores multiply
// exactly, so eight codes cost four AND and one shift. The powers of two leave through
// fp32 factors (scores) and through the final scaling of the accumulators (outputs).
//
// K: one accumulator per group, weighed by the step of its row in fp32. The minima are
// one more MMA, against the sums of the query over each group (exact to 22 bits as two
// fp16 terms). V: the weights are multiplied by the steps of their tokens, one packed
// multiplication per group and token pair; the minima are one more MMA whose rows are
// the groups. (Sums from alternating ends of the codes: see int4_pv.)
//
// Shared-memory order. Row i of the score MMA (and with it column i of the V MMA) is
// token row_of(i) of its 16: rows of 80 bytes four apart start 64 bytes apart modulo 128,
// so the eight 16-byte words of a quarter warp fall in distinct banks.
#pragma once

#include "pa_device.cuh"

namespace pa {

// Token (0..7) of row i (0..7) of an MMA row block's half; the other half adds 8.
__device__ __forceinline__ int int4_row_of(int i) { return (i >> 1) + 4 * (i & 1); }

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Two 8x8 16-bit matrices, transposed; lanes 0-7 and 8-15 give their row addresses.
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t mul2_half(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// c = a b with a zero accumulator (fp16 in, fp32 out).
__device__ __forceinline__ void mma16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int D>
struct Int4Row {
  static constexpr int G = D / 32;             // groups
  static constexpr int CODES = D / 2;          // bytes of codes; the steps follow
  static constexpr int MINS = CODES + 2 * G;   // byte offset of the minima
  static constexpr int BYTES = MINS + 2 * G;
  static constexpr int W = G / 4;              // 16-byte words of one octet of all groups
  static constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
};

// The steps (at = CODES) or minima (at = MINS) of the row at `row`, packed two groups a word.
template <int D>
__device__ __forceinline__ void int4_meta(uint32_t (&w)[D / 64], uint32_t row, int at) {
  if constexpr (D == 128) {
    const uint2 v = lds64(row + at);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = lds128(row + at);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// Query fragments for the codes' order and range, from the raw words loaded in the
// prologue (eight consecutive elements 32 g + 8 tig .. + 7 per group g, in qf[2g][0],
// qf[2g][1], qf[2g+1][0], qf[2g+1][1]). The column is scaled by a power of two that puts
// its largest magnitude in [2^9, 2^10): exact, whatever the query's range, with 24 binades
// left below and room for the sum over a group. Element j of the eight meets the code in
// nibble j: nibbles 0, 4 | 2, 6 in the first k-step, 1, 5 | 3, 7 (sixteen times larger as
// fp16 words, so the query is divided by 16) in the second. qs: the B fragment of the
// minima's MMA, the group sums as high and low fp16 terms. Returns the column's factor
// 2^k to be taken out of its scores.
template <typename T, int D>
__device__ __forceinline__ float int4_query(uint32_t (&qf)[D / 16][2], uint32_t (&qs)[2], int tig) {
  using R = Int4Row<D>;
  float amax = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v = unpack2<T>(qf[kk][i]);
      amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // 2^e <= amax < 2^(e+1); both 2^(9-e) and its inverse stay normal fp32 numbers
  const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
  const float up = __uint_as_float((uint32_t)(127 + 9 - e) << 23);
  const float down = __uint_as_float((uint32_t)(127 - 9 + e) << 23);
  uint32_t hi[R::G / 2], lo[R::G / 2];  // group sums of two groups a word
#pragma unroll
  for (int g = 0; g < R::G; ++g) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<T>(qf[2 * g + i / 2][i % 2]);
      x[2 * i] = v.x * up;
      x[2 * i + 1] = v.y * up;
    }
    const uint32_t a = pack2<__half>(x[0], x[4]), b = pack2<__half>(x[2], x[6]);
    const uint32_t c = pack2<__half>(x[1], x[5]), d = pack2<__half>(x[3], x[7]);
    const float2 fa = unpack2<__half>(a), fb = unpack2<__half>(b);
    const float2 fc = unpack2<__half>(c), fd = unpack2<__half>(d);
    float sum = ((fa.x + fa.y) + (fb.x + fb.y)) + ((fc.x + fc.y) + (fd.x + fd.y));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    qf[2 * g][0] = a;
    qf[2 * g][1] = b;
    qf[2 * g + 1][0] = pack2<__half>(fc.x * 0.0625f, fc.y * 0.0625f);
    qf[2 * g + 1][1] = pack2<__half>(fd.x * 0.0625f, fd.y * 0.0625f);
    const uint32_t h = pack2<__half>(sum, 0.f);  // low half: the high term
    const uint32_t l = pack2<__half>(sum - unpack2<__half>(h).x, 0.f);
    hi[g / 2] = (g & 1) ? (hi[g / 2] | (h << 16)) : (h & 0xffffu);
    lo[g / 2] = (g & 1) ? (lo[g / 2] | (l << 16)) : (l & 0xffffu);
  }
  // rows k of the B operand: high terms of the groups, then low terms (D 128: k = 0-3 and
  // 4-7; D 256: 0-7 and 8-15); the A operand repeats the minima over both ranges
  qs[0] = qs[1] = 0u;
#pragma unroll
  for (int i = 0; i < R::G / 2; ++i) {
    if constexpr (D == 128) {
      if (tig == i) qs[0] = hi[i];
      if (tig == i + 2) qs[0] = lo[i];
    } else {
      if (tig == i) {
        qs[0] = hi[i];
        qs[1] = lo[i];
      }
    }
  }
  return down;
}

// The query fragments of a CTA's columns: in registers, or (SHARED) in shared memory as eight
// bytes per column tile, k-step and lane, where the registers serve more warps better.
template <int D, int NT, bool SHARED>
struct Int4Query {
  uint32_t r[SHARED ? 1 : NT][SHARED ? 1 : D / 16][2];
  uint32_t at;  // SHARED: this lane's words of the first fragment
  __device__ __forceinline__ uint2 operator()(int nt, int ks) const {
    if constexpr (SHARED) return lds64(at + (nt * (D / 16) + ks) * 256);
    return make_uint2(r[nt][ks][0], r[nt][ks][1]);
  }
};

// Scores of 16 MT tokens from `rows` (their first row in shared memory) with NT column tiles:
// s[mt][nt] = sum_g step_g (q . n) * 2^-24 and sm[mt][nt] = sum_g minimum_g (sum of q).
template <int D, int NT, int MT, bool SHARED>
__device__ __forceinline__ void int4_scores(float (&s)[MT][NT][4], float (&sm)[MT][NT][4], uint32_t rows,
                                            const Int4Query<D, NT, SHARED>& q,
                                            const uint32_t (&qs)[NT][2], int gid, int tig) {
  using R = Int4Row<D>;
  uint4 k0[MT][R::W], k1[MT][R::W];
  uint32_t st0[MT][R::G / 2], st1[MT][R::G / 2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const uint32_t r0 = rows + (16 * mt + int4_row_of(gid)) * R::BYTES, r1 = r0 + 8 * R::BYTES;
#pragma unroll
    for (int i = 0; i < R::W; ++i) {
      k0[mt][i] = lds128(r0 + 16 * R::W * tig + 16 * i);
      k1[mt][i] = lds128(r1 + 16 * R::W * tig + 16 * i);
    }
    int4_meta<D>(st0[mt], r0, R::CODES);
    int4_meta<D>(st1[mt], r1, R::CODES);
    uint32_t a[4];
    a[0] = lds32(r0 + R::MINS + 4 * (tig & (R::G / 2 - 1)));
    a[1] = lds32(r1 + R::MINS + 4 * (tig & (R::G / 2 - 1)));
    a[2] = a[0];
    a[3] = a[1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma16816_zero(sm[mt][nt], a, qs[nt][0], qs[nt][1]);
  }
#pragma unroll
  for (int g = 0; g < R::G; ++g) {
    uint2 b0[NT], b1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      b0[nt] = q(nt, 2 * g);
      b1[nt] = q(nt, 2 * g + 1);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint32_t w0 = word_of(k0[mt][g / 4], g % 4), w1 = word_of(k1[mt][g / 4], g % 4);
      const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
      const uint32_t a0[4] = {w0 & R::LO, w1 & R::LO, h0 & R::LO, h1 & R::LO};
      const uint32_t a1[4] = {w0 & R::HI, w1 & R::HI, h0 & R::HI, h1 & R::HI};
      const float2 u0 = unpack2<__half>(st0[mt][g / 2]), u1 = unpack2<__half>(st1[mt][g / 2]);
      const float f0 = (g & 1) ? u0.y : u0.x, f1 = (g & 1) ? u1.y : u1.x;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[4];
        mma16816_zero(acc, a0, b0[nt].x, b0[nt].y);
        mma16816<__half>(acc, a1, b1[nt].x, b1[nt].y);
        float(&d)[4] = s[mt][nt];
        d[0] = g == 0 ? f0 * acc[0] : fmaf(f0, acc[0], d[0]);
        d[1] = g == 0 ? f0 * acc[1] : fmaf(f0, acc[1], d[1]);
        d[2] = g == 0 ? f1 * acc[2] : fmaf(f1, acc[2], d[2]);
        d[3] = g == 0 ? f1 * acc[3] : fmaf(f1, acc[3], d[3]);
      }
    }
  }
}

// o += V^T P^T over the 16 tokens at `rows` (rows past the context have zero steps and
// minima there; any code is finite). Accumulator o[nt][2g + i]: rows gid and gid + 8 are
// elements 32 g + 4 gid + i and + 2, times 2^-24, for i = 0; for i = 1 the A operand is the
// whole byte (the nibble of i = 1 above that of i = 0), which takes one mask less, so that
// the accumulator holds 16 times the element's sum plus that of i = 0 until int4_finish.
//
// Every other 16 tokens are summed from the other end of the codes (DOWN): value =
// maximum - step * (15 - n), with 15 - n the complement of the nibble. Summed from the
// minimum alone, the codes' sums and the minima's grow with the context and cancel, and
// the truncation of the tensor cores' fp32 sums is not lost in them: 4e-3 of the output
// over 32K tokens in one split. From alternating ends both sums stay near the result.
//
// The steps of two tokens, for the multiplication of the weights, come from a transposing
// load of the tokens' steps and minima: lane 4 g + tig then holds those of group g and
// tokens 2 tig, 2 tig + 1 (of the MMA's order), and a shuffle hands them to the others.
// om[nt][0..1], row gid: the sum of the minima (maxima) of group gid. A maximum is the minimum,
// plus 16 steps, minus one: rounded to fp16 it cost 4.4e-4 of the output's norm, as three
// exact products nothing. The MMAs of the three lie apart, since they add to one accumulator
// (GB300, us per call, one rounded product / three in a row / three apart: 32/8 heads of 128,
// 32 sequences of 16K 125.1 / 129.1 / 127.0, 4 query rows of 8 of 16K 55.4 / 55.3 / 55.1, 8 rows
// 133.9 / 140.9 / 138.2; 24/4 of 256, 2 rows of 8 of 8K 35.4 / 35.9 / 35.6). The minus one in the
// idle rows of the first MMA, with accumulators of its own: 127.1, 56.4, 139.1 and 36.5.
template <int D, int NT, bool DOWN>
__device__ __forceinline__ void int4_pv(float (&o)[NT][D / 16][4], float (&om)[NT][4], uint32_t rows,
                                        const uint32_t (&pb)[NT][2], int lane) {
  using R = Int4Row<D>;
  const int gid = lane >> 2, tig = lane & 3;
  uint4 w[4][R::W];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // the tokens of k = 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
    const uint32_t row = rows + (tig + 4 * (j & 1) + 8 * (j >> 1)) * R::BYTES;
#pragma unroll
    for (int i = 0; i < R::W; ++i) w[j][i] = lds128(row + 16 * R::W * (gid >> 1) + 16 * i);
  }
  uint32_t st[2], mn[2];  // steps and minima of group gid (D 128: gid < 4), tokens of k < 8 and >= 8
  {
    const uint32_t row = rows + (int4_row_of(lane & 7) + (lane & 8)) * R::BYTES + R::CODES;
    if constexpr (D == 128) {
      ldmatrix_x2_trans(st, row);  // eight 16-bit columns: four steps, four minima
      mn[0] = __shfl_sync(0xffffffffu, st[0], lane + 16);
      mn[1] = __shfl_sync(0xffffffffu, st[1], lane + 16);
    } else {
      uint32_t m[4];
      ldmatrix_x4<true>(m, row + (lane & 16));
      st[0] = m[0];
      st[1] = m[1];
      mn[0] = m[2];
      mn[1] = m[3];
    }
  }
  {
    const uint32_t a[4] = {mn[0], 0u, mn[1], 0u};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma16816<__half>(om[nt], a, pb[nt][0], pb[nt][1]);
  }
  if (DOWN) {
    st[0] ^= 0x80008000u;
    st[1] ^= 0x80008000u;
  }
  const uint32_t sel = (gid & 1) ? 0x7632u : 0x5410u;  // the half of the octet's word
#pragma unroll
  for (int g = 0; g < R::G; ++g) {
    const uint32_t x0 = __byte_perm(word_of(w[0][g / 4], g % 4), word_of(w[1][g / 4], g % 4), sel);
    const uint32_t x1 = __byte_perm(word_of(w[2][g / 4], g % 4), word_of(w[3][g / 4], g % 4), sel);
    const uint32_t h0 = __byte_perm(x0, 0u, 0x4341), h1 = __byte_perm(x1, 0u, 0x4341);  // upper bytes
    constexpr uint32_t kBytes = 0x00ff00ffu;
    auto lo = [](uint32_t x) { return (DOWN ? ~x : x) & R::LO; };
    const uint32_t a0[4] = {lo(x0), lo(h0), lo(x1), lo(h1)};
    const uint32_t a1[4] = {(DOWN ? ~x0 : x0) & kBytes, DOWN ? h0 ^ kBytes : h0,
                            (DOWN ? ~x1 : x1) & kBytes, DOWN ? h1 ^ kBytes : h1};
    const uint32_t s0 = __shfl_sync(0xffffffffu, st[0], 4 * g + tig);
    const uint32_t s1 = __shfl_sync(0xffffffffu, st[1], 4 * g + tig);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the weights times the steps, rounded to fp16 once more
      const uint32_t b0 = mul2_half(pb[nt][0], s0), b1 = mul2_half(pb[nt][1], s1);
      mma16816<__half>(o[nt][2 * g], a0, b0, b1);
      mma16816<__half>(o[nt][2 * g + 1], a1, b0, b1);
    }
    if (DOWN && g == R::G / 2) {  // st is negative here: plus 16 steps ..
      const uint32_t a[4] = {st[0], 0u, st[1], 0u};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma16816<__half>(om[nt], a, mul2_half(pb[nt][0], 0xcc00cc00u), mul2_half(pb[nt][1], 0xcc00cc00u));
    }
  }
  if (DOWN) {  // .. minus one
    const uint32_t a[4] = {st[0], 0u, st[1], 0u};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma16816<__half>(om[nt], a, pb[nt][0], pb[nt][1]);
  }
}

// The codes' powers of two out of the accumulators, and the minima's sums in.
template <int D, int NT>
__device__ __forceinline__ void int4_finish(float (&o)[NT][D / 16][4], const float (&om)[NT][4], int tig) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
      const float m0 = __shfl_sync(0xffffffffu, om[nt][0], 4 * g + tig);
      const float m1 = __shfl_sync(0xffffffffu, om[nt][1], 4 * g + tig);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = o[nt][2 * g][i] * 16777216.f;                   // 2^24
        const float hi = (o[nt][2 * g + 1][i] - o[nt][2 * g][i]) * 1048576.f;  // 2^20
        const float mn = (i & 1) ? m1 : m0;
        o[nt][2 * g][i] = lo + mn;
        o[nt][2 * g + 1][i] = hi + mn;
      }
    }
}

}  // namespace pa
