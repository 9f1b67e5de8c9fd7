// Score modification of the tile kernels: tanh cap, distance bias, document
// and position masks (spattn_score).
//
//   z = c tanh(x / c) - slope |pos_q - pos_k|,   x = scale q.k   (no cap: z = x - ...)
//   allowed iff the plan's masks say so, k_pos <= q_last and q_doc == k_doc >= 0.
//
// The column side of a step (positions, documents, and their range over the
// step) is written into shared memory by the warp that loads the step's tiles.
// A row warp holds the range of its own rows, so a step that the two ranges show
// to be fully allowed or fully masked costs it a few compares; pairs are compared
// only in the others.  The lines become visible to the rows with the barrier
// that announces the step's scores: the issuer of the products has waited
// for the tiles, whose announcement follows the lines, and adds an arrival of its
// own to that of the products.
#pragma once

#include "tile.cuh"

namespace spattn {
namespace dev {

// Forms of a scored kernel.
//   kScoreNone   the plain kernel
//   kScoreMask   masks and bias
//   kScoreCap    the same with a cap
//   kScoreFixed  (paged) a cap within kCapFixedMax: a fixed softmax reference
enum : int { kScoreNone = 0, kScoreMask = 1, kScoreCap = 2, kScoreFixed = 3 };

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// NaN stays NaN (fminf would drop it)
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// s (raw products) -> z = c log2(e) tanh(s scale / c) in place; with GRAD also
// d *= 1 - tanh^2.
//
// While every score of the warp's step is at most half the cap, tanh is its
// polynomial: z = s (a0 + a1 w + ... + a4 w^4), w = s^2, the coefficients of
// tanh(u) / u on |u| <= 1/2 (relative error 1.5e-8) with scale, cap and log2(e)
// folded in by the host: five FMA-pipe operations per pair more than a plain
// score.  Beyond that it is 1 - 2 / (1 + e^2u) with two special-function
// operations per pair, of which the softmax already spends one.  Scores well
// inside the cap are the ordinary case; a warp decides per step.  `votes`: whether
// this thread's scores count for that.  Those of rows without a pair do not: they
// may be whatever stood in tensor memory, and the two branches differ in their last bits.
constexpr float kTanhExpMax = 126.0f;  // e^2u held at 2^126: 1 - tanh^2 = 4 r (e r), r = 1 / (1 + e), stays finite
template <bool GRAD, int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], uint32_t (&d)[N], const CapArgs& c, bool votes) {
  auto pair = [&](int i) { return f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])); };
  constexpr bool kKeep = N <= 16;  // wider rows form the squares twice rather than hold them
  uint64_t sq[kKeep ? N / 2 : 1];
  float mx[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float a, b;
    const uint64_t w = f2_mul(pair(i), pair(i));
    if constexpr (kKeep) sq[i] = w;
    f2_unpack(w, a, b);
    mx[i & 1] = fmax3(mx[i & 1], a, b);  // a NaN drops out here and keeps its NaN in either form
  }
  if (__builtin_expect(!__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > (votes ? c.w_max : INFINITY)), 1)) {
    const uint64_t a0 = c.a[0], a1 = c.a[1], a2 = c.a[2], a3 = c.a[3], a4 = c.a[4], ng = c.ng, one = f2_pack(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint64_t x = pair(i), w = kKeep ? sq[kKeep ? i : 0] : f2_mul(x, x);
      const uint64_t z = f2_mul(x, f2_fma(f2_fma(f2_fma(f2_fma(a4, w, a3), w, a2), w, a1), w, a0));
      float a, b;
      f2_unpack(z, a, b);
      s[2 * i] = __float_as_uint(a);
      s[2 * i + 1] = __float_as_uint(b);
      if constexpr (GRAD) {
        // 1 - tanh^2 = 1 - (z / (c log2 e))^2
        const uint64_t g = f2_fma(f2_mul(z, ng), z, one);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), g), a, b);
        d[2 * i] = __float_as_uint(a);
        d[2 * i + 1] = __float_as_uint(b);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = ex2(min_nan(__uint_as_float(s[i]) * c.k2, kTanhExpMax));
      const float r = rcp_approx(1.f + e);
      s[i] = __float_as_uint(fmaf(-2.f * c.cap2, r, c.cap2));
      if constexpr (GRAD) d[i] = __float_as_uint(__uint_as_float(d[i]) * (4.f * r * (e * r)));
    }
  }
}

// s - slope * |row - col| in place, col[i] the fp32 positions of the N columns
// in shared memory (16-byte aligned).  Scores that are multiplied later (no cap)
// come with the slope divided by that factor.
template <int N>
__device__ __forceinline__ void bias_scores(uint32_t (&s)[N], const float* col, float row, float slope) {
  const uint64_t nr = f2_pack(-row, -row);
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(col + i);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float d0, d1;
      f2_unpack(f2_add(j ? f2_pack(c.z, c.w) : f2_pack(c.x, c.y), nr), d0, d1);
      s[i + j] = __float_as_uint(fmaf(-slope, fabsf(d0), __uint_as_float(s[i + j])));
      s[i + j + 1] = __float_as_uint(fmaf(-slope, fabsf(d1), __uint_as_float(s[i + j + 1])));
    }
  }
}

// s * mul + col[i] in place (col: N fp32 values in shared memory).
template <int N>
__device__ __forceinline__ void add_columns(uint32_t (&s)[N], const float* col, float mul) {
  const uint64_t m2 = f2_pack(mul, mul);
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(col + i);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float a, b;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 1])), m2,
                       j ? f2_pack(c.z, c.w) : f2_pack(c.x, c.y)),
                a, b);
      s[i + j] = __float_as_uint(a);
      s[i + j + 1] = __float_as_uint(b);
    }
  }
}

// dS of one row, N columns, and its weights: w = 2^x (x = log2 of the weight, in
// `s`), ds = w d, both in bf16; `out` holds dS, or with 2 N / 2 words the weights
// and then dS.  Columns whose bit is clear get zeros, and dS is dropped where the
// weight rounds to one (live_weight).
__device__ __forceinline__ bool live_weight(float p);
template <int N, int W>
__device__ __forceinline__ void weights_and_ds(uint32_t (&s)[N], uint32_t (&d)[N], uint32_t bits, uint32_t (&out)[W]) {
  static_assert(W == N / 2 || W == N, "dS, or weights and dS");
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = __float_as_uint(ex2(__uint_as_float(s[i])));
  if (__builtin_expect(bits != (N == 32 ? 0xFFFFFFFFu : (1u << (N & 31)) - 1u), 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool on = (bits >> i) & 1u;
      if (!on || !live_weight(__uint_as_float(s[i]))) d[i] = 0u;
      if (!on) s[i] = 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float p0 = __uint_as_float(s[2 * i]), p1 = __uint_as_float(s[2 * i + 1]);
    float s0, s1;
    f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]))), s0, s1);
    if constexpr (W == N) out[i] = pack_bf16(p0, p1);
    out[W - N / 2 + i] = pack_bf16(s0, s1);
  }
}

// Whether a pair of weight p has a gradient: not when masked (p = 0), and not
// when p rounds to one.  With p = 1 - e every other weight of the row is at most
// e, so |dS| <= 2 e max |dP|, below 2^-15 of dP for e < 2^-16, while Delta (from O
// rounded to bf16, summed in another order than dP) is off by more; a query
// with a single key gets the exact 0.  Used where a step's mask has holes, as
// the mask of a query with one key always has in the query-owned pass.
__device__ __forceinline__ bool live_weight(float p) { return p != 0.f && p < 1.0f - 1.52587890625e-5f; }

// Range of the positions (or last positions) and documents of the live columns
// of a step or half step: {min, max} of each.  No live column leaves the
// range empty (min above max).
__device__ __forceinline__ int4 column_range(bool live, int pos, int doc) {
  constexpr int kLow = static_cast<int>(0x80000000), kHigh = 0x7FFFFFFF;
  return make_int4(__reduce_min_sync(0xffffffffu, live ? pos : kHigh), __reduce_max_sync(0xffffffffu, live ? pos : kLow),
                   __reduce_min_sync(0xffffffffu, live ? doc : kHigh), __reduce_max_sync(0xffffffffu, live ? doc : kLow));
}
// The same of two columns per lane, which halves the reductions.  (Leaving out
// those that no mask asks for puts branches between them: 2% slower on 12289
// tokens; so are ranges of 64 columns in the dQ kernel, 573 -> 587 us on the video
// layout, where more steps then count as mixed.)
__device__ __forceinline__ int4 columns_range(const bool (&live)[2], const int (&pos)[2], const int (&doc)[2]) {
  constexpr int kLow = static_cast<int>(0x80000000), kHigh = 0x7FFFFFFF;
  return make_int4(__reduce_min_sync(0xffffffffu, min(live[0] ? pos[0] : kHigh, live[1] ? pos[1] : kHigh)),
                   __reduce_max_sync(0xffffffffu, max(live[0] ? pos[0] : kLow, live[1] ? pos[1] : kLow)),
                   __reduce_min_sync(0xffffffffu, min(live[0] ? doc[0] : kHigh, live[1] ? doc[1] : kHigh)),
                   __reduce_max_sync(0xffffffffu, max(live[0] ? doc[0] : kLow, live[1] ? doc[1] : kLow)));
}

// Range of a warp's rows: of last positions (query rows) or positions (key rows),
// and of documents.  Rows without a segment are left out.
__device__ __forceinline__ int4 row_range(bool real, int pos, int doc) { return column_range(real, pos, doc); }

// Query rows `w` against key columns `c`: none allowed / every pair allowed.
__device__ __forceinline__ bool query_none(const ScoreArgs& sc, int4 c, int4 w) {
  return (sc.q_last && c.x > w.y) || (sc.q_doc && (w.w < 0 || w.w < c.z || w.z > c.w));
}
__device__ __forceinline__ bool query_all(const ScoreArgs& sc, int4 c, int4 w) {
  return (!sc.q_last || c.y <= w.x) && (!sc.q_doc || (c.z == c.w && w.z == w.w && c.z == w.z && w.z >= 0));
}
// Key rows `w` against query columns `c`.
__device__ __forceinline__ bool key_none(const ScoreArgs& sc, int4 c, int4 w) {
  return (sc.q_last && w.x > c.y) || (sc.q_doc && (w.w < 0 || w.w < c.z || w.z > c.w));
}
__device__ __forceinline__ bool key_all(const ScoreArgs& sc, int4 c, int4 w) {
  return (!sc.q_last || w.y <= c.x) && (!sc.q_doc || (c.z == c.w && w.z == w.w && c.z == w.z && w.z >= 0));
}

// A warp whose rows differ asks each of them (its own range being a point): a row
// with nothing loses its bits, and true comes back if it has to be compared.
__device__ __forceinline__ bool mixed_row(uint32_t& bits, bool none, bool all) {
  if (none) bits = 0u;
  return !none && !all && bits != 0u;
}

// Bits of N columns for one row.  KEYS: the columns are keys (position <=
// `mine`), else queries (`mine` <= their last position).
template <bool KEYS, int N>
__device__ __forceinline__ uint32_t column_bits(bool use_pos, bool use_doc, const int* pos, const int* doc, int mine,
                                             int my_doc) {
  uint32_t bits = 0xFFFFFFFFu;
  if (use_pos) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int4 c = *reinterpret_cast<const int4*>(pos + i);
      b |= (KEYS ? c.x <= mine : mine <= c.x) ? 1u << i : 0u;
      b |= (KEYS ? c.y <= mine : mine <= c.y) ? 2u << i : 0u;
      b |= (KEYS ? c.z <= mine : mine <= c.z) ? 4u << i : 0u;
      b |= (KEYS ? c.w <= mine : mine <= c.w) ? 8u << i : 0u;
    }
    bits = b;
  }
  if (use_doc) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int4 c = *reinterpret_cast<const int4*>(doc + i);
      b |= c.x == my_doc ? 1u << i : 0u;
      b |= c.y == my_doc ? 2u << i : 0u;
      b |= c.z == my_doc ? 4u << i : 0u;
      b |= c.w == my_doc ? 8u << i : 0u;
    }
    bits &= my_doc >= 0 ? b : 0u;
  }
  return bits;
}

// ----------------------------------------------------------------------------
// Softmax of one step with two threads per row
// ----------------------------------------------------------------------------
// Group g (0, 1) has 32 of the step's 64 columns, so that four row warps per
// scheduler (two CTAs) cover each other's latency and a thread's code is half as
// long.  That needs a reference of the weights that is known beforehand: with a
// running maximum the two threads would exchange their halves' maxima every step,
// which cost more than the second thread gave (943 us -> 1421 on 12289 causal
// tokens x 16 heads).  They meet once, at the end.  Four threads per row would have 56
// registers each and were slower again (981 -> 1235 us with a cap and a prefix).
struct SoftRow {
  float l = 0.f;   // sum of this thread's weights
  float lr = 0.f;  // the same of the weights rounded to bf16
};

// Sums of weights within these leave fp32 2^46 on either side, for the values and for
// the smaller keys; a row outside (an LSE beyond +-55 of its reference) needs its maximum.
constexpr float kSumLow = 8.271806125530277e-25f, kSumHigh = 1.2089258196146292e24f;  // 2^-80, 2^80

// Meeting of the two warps of a row pair (a barrier of 64 arrivals), the n-th.  A
// bounded wait, so that a warp that gave up cannot strand its partner; false
// when the CTA is aborting.
__device__ __forceinline__ bool pair_sync(uint64_t* bar, int n, const Abort& ab) {
  mbar_arrive(bar);
  return __all_sync(0xffffffffu, mbar_wait(bar, n & 1, ab));
}

// Weights 2^(s mul - ref) of this thread's 32 columns to P (bf16, TMEM) and their sums.
__device__ __forceinline__ void soft_weights(const uint32_t (&s)[32], float mul, float ref, SoftRow& r, uint32_t p_addr) {
  const uint64_t m2 = f2_pack(mul, mul), n2 = f2_pack(-ref, -ref);
  uint64_t sum[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)}, sumr[2] = {sum[0], sum[1]};
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), m2, n2), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    sum[i & 1] = f2_add(sum[i & 1], f2_pack(p0, p1));
    pk[i] = pack_bf16(p0, p1);
    sumr[i & 1] = f2_add(sumr[i & 1], f2_pack(__uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xFFFF0000u)));
  }
  tmem_st16(p_addr, pk);
  float a0, a1, b0, b1;
  f2_unpack(sum[0], a0, a1);
  f2_unpack(sum[1], b0, b1);
  r.l += (a0 + a1) + (b0 + b1);
  f2_unpack(sumr[0], a0, a1);
  f2_unpack(sumr[1], b0, b1);
  r.lr += (a0 + a1) + (b0 + b1);
}

// Sums of both threads of the row (xsum: this row's entries of [4][128] floats).
// `l`, the divisor of O, sums the rounded weights: no weight need be 1 here, so a
// row with few keys would keep its weights' rounding otherwise.  l_true is
// the sum in LSE.
__device__ __forceinline__ bool soft_total(const SoftRow& r, float* xsum, int grp, uint64_t* bar, int n,
                                           const Abort& ab, float& l, float& l_true) {
  xsum[128 * grp] = r.l;
  xsum[256 + 128 * grp] = r.lr;
  if (!pair_sync(bar, n, ab)) return false;
  l_true = xsum[0] + xsum[128];
  l = xsum[256] + xsum[256 + 128];
  return true;
}

// The row's maximum over both threads (-inf: no key).
__device__ __forceinline__ float local_max(const uint32_t (&s)[32]) {
  float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    mx[0] = fmax3(mx[0], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    mx[1] = fmax3(mx[1], __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
  }
  return fmaxf(mx[0], mx[1]);
}

}  // namespace dev
}  // namespace spattn
