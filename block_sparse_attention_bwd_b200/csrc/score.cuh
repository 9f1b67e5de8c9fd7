// Score modification of the tile kernels: tanh cap, distance bias, document
// and position masks (spattn_score).
//
//   z = c tanh(x / c) - slope |pos_q - pos_k|,   x = scale q.k   (no cap: z = x - ...)
//   allowed iff the plan's masks say so, k_pos <= q_last and q_doc == k_doc >= 0.
//
// A lane holds the position and document of one or two columns of the step
// (loaded a step ahead); a row's thread reads them by shuffle when it has to
// compare, and as fp32 from a warp's own shared-memory line for the bias, which
// touches every pair.  Comparison per pair happens only in steps where some row of the
// warp is neither fully allowed nor fully masked by the range of the
// step's positions and documents.
#pragma once

#include "tile.cuh"

namespace spattn {
namespace dev {

// tanh for |u| <= 1/2: u + u v Q(v), v = u^2, Q the minimax cubic of
// (tanh(u) / u - 1) / v on [0, 1/4] (relative error 1.5e-8), all on the FMA
// pipe.  Outside, 1 - 2 / (1 + e^2u) with two special-function operations.
// A warp takes the first form when all of its scores of the step allow it:
// scores well inside the cap are the ordinary case, and the softmax already
// spends a special-function operation per pair.
constexpr float kTanhPolyMax = 0.5f;
constexpr float kTq0 = -0.33333149552345276f, kTq1 = 0.1332598626613617f, kTq2 = -0.05305291339755058f,
                kTq3 = 0.017256902530789375f;
// e^2u is held at 2^100 so that 1 - tanh^2 = 4 e r^2 (r = 1 / (1 + e)) stays finite
constexpr float kTanhExpMax = 100.0f;

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

// s (raw products) -> cap2 * tanh(s * k1), in place; k1 = scale / cap, cap2 =
// cap * log2(e).  With GRAD also d *= 1 - tanh^2.
template <bool GRAD>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[32], uint32_t (&d)[32], float k1, float cap2) {
  float mx[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    mx[0] = fmax3(mx[0], fabsf(__uint_as_float(s[i])), fabsf(__uint_as_float(s[i + 1])));
    mx[1] = fmax3(mx[1], fabsf(__uint_as_float(s[i + 2])), fabsf(__uint_as_float(s[i + 3])));
  }
  const bool wide = fmaxf(mx[0], mx[1]) * fabsf(k1) > kTanhPolyMax;  // a NaN score keeps its NaN in either form
  if (!__any_sync(0xffffffffu, wide)) {
    const uint64_t k = f2_pack(k1, k1), c2 = f2_pack(cap2, cap2);
    const uint64_t q0 = f2_pack(kTq0, kTq0), q1 = f2_pack(kTq1, kTq1), q2 = f2_pack(kTq2, kTq2), q3 = f2_pack(kTq3, kTq3);
    const uint64_t one = f2_pack(1.f, 1.f), m1 = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint64_t u = f2_mul(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), k);
      const uint64_t v = f2_mul(u, u);
      const uint64_t q = f2_fma(f2_fma(f2_fma(q3, v, q2), v, q1), v, q0);
      const uint64_t t = f2_fma(f2_mul(u, v), q, u);
      float a, b;
      f2_unpack(f2_mul(t, c2), a, b);
      s[i] = __float_as_uint(a);
      s[i + 1] = __float_as_uint(b);
      if constexpr (GRAD) {
        const uint64_t g = f2_fma(f2_mul(t, m1), t, one);
        f2_unpack(f2_mul(f2_pack(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), g), a, b);
        d[i] = __float_as_uint(a);
        d[i + 1] = __float_as_uint(b);
      }
    }
  } else {
    const float k2 = k1 * (2.f * kLog2e);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float e = ex2(min_nan(__uint_as_float(s[i]) * k2, kTanhExpMax));
      const float r = rcp_approx(1.f + e);
      s[i] = __float_as_uint(fmaf(-2.f * cap2, r, cap2));
      if constexpr (GRAD) d[i] = __float_as_uint(__uint_as_float(d[i]) * (4.f * r * (e * r)));
    }
  }
}

// s * mul - slope2 * |row - col| in place, col[i] the fp32 positions of 32
// columns in shared memory (16-byte aligned); slope_lo is the slope of
// columns 0..15, slope_hi that of 16..31 (the two pages may belong to two heads).
__device__ __forceinline__ void bias_scores(uint32_t (&s)[32], const float* col, float row, float mul, float slope_lo,
                                            float slope_hi) {
  const uint64_t m2 = f2_pack(mul, mul), nr = f2_pack(-row, -row);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float sl = i < 16 ? -slope_lo : -slope_hi;
    const uint64_t ns = f2_pack(sl, sl);
    const float4 c = *reinterpret_cast<const float4*>(col + i);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float d0, d1, a, b;
      f2_unpack(f2_add(j ? f2_pack(c.z, c.w) : f2_pack(c.x, c.y), nr), d0, d1);
      f2_unpack(f2_fma(f2_pack(fabsf(d0), fabsf(d1)), ns,
                       f2_mul(f2_pack(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 1])), m2)),
                a, b);
      s[i + j] = __float_as_uint(a);
      s[i + j + 1] = __float_as_uint(b);
    }
  }
}

// s * mul - col[i] in place (col: 32 fp32 values in shared memory).
__device__ __forceinline__ void sub_columns(uint32_t (&s)[32], const float* col, float mul) {
  const uint64_t m2 = f2_pack(mul, mul);
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(col + i);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      float a, b;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 1])), m2,
                       j ? f2_pack(-c.z, -c.w) : f2_pack(-c.x, -c.y)),
                a, b);
      s[i + j] = __float_as_uint(a);
      s[i + j + 1] = __float_as_uint(b);
    }
  }
}

// Whether a pair of weight p has a gradient: not when masked (p = 0), and not
// when p rounds to one.  With p = 1 - e every other weight of the row is at most
// e, so |dS| <= 2 e max |dP|, below 2^-15 of dP for e < 2^-16, while Delta (from O
// rounded to bf16, summed in another order than dP) is off by more; a row with
// a single key gets the exact 0.  Used where a step's mask has holes, which a
// row with one key always has.
__device__ __forceinline__ bool live_weight(float p) { return p != 0.f && p < 1.0f - 1.52587890625e-5f; }

// Position and document of one key column (lanes hold one each).  A column
// behind the list or the tensor is left out of the ranges; the plan's masks
// already exclude it.
struct KeyCol {
  int pos, doc;
  bool live;
  __device__ __forceinline__ void clear() {
    pos = 0;
    doc = -1;
    live = false;
  }
};

__device__ __forceinline__ KeyCol load_key_col(const ScoreArgs& sc, int64_t batch_off, bool listed, int32_t ref, int r,
                                               int64_t slots) {
  KeyCol k;
  k.clear();
  const int64_t slot = pref_slot(ref, r);
  k.live = listed && slot < slots;
  if (k.live) {
    if (sc.k_pos) k.pos = __ldg(sc.k_pos + batch_off + slot);
    if (sc.k_doc) k.doc = __ldg(sc.k_doc + batch_off + slot);
  }
  return k;
}

// What a query row allows.
struct RowRule {
  int last, doc;  // doc: -1 attends nothing when documents are in use
};

// Range of positions and documents over the live columns of a warp's lanes.
struct ColRange {
  int pos_min, pos_max, doc_min, doc_max;
  __device__ __forceinline__ void reset() {
    pos_min = doc_min = 0x7FFFFFFF;
    pos_max = doc_max = static_cast<int>(0x80000000);
  }
  __device__ __forceinline__ void add(const KeyCol& k) {
    if (!k.live) return;
    pos_min = min(pos_min, k.pos);
    pos_max = max(pos_max, k.pos);
    doc_min = min(doc_min, k.doc);
    doc_max = max(doc_max, k.doc);
  }
  __device__ __forceinline__ void reduce() {
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    pos_max = __reduce_max_sync(0xffffffffu, pos_max);
    doc_min = __reduce_min_sync(0xffffffffu, doc_min);
    doc_max = __reduce_max_sync(0xffffffffu, doc_max);
  }
};

// One query column of the key-owned pass: what it allows, and its LSE.
struct QueryCol {
  int last, doc;
  float pos, lse2, slope2;
  bool live;
};

// Range of the live columns' rules over a warp's lanes.
struct QueryRange {
  int last_min, last_max, doc_min, doc_max;
  __device__ __forceinline__ void of(const QueryCol& q) {
    last_min = __reduce_min_sync(0xffffffffu, q.live ? q.last : 0x7FFFFFFF);
    last_max = __reduce_max_sync(0xffffffffu, q.live ? q.last : static_cast<int>(0x80000000));
    doc_min = __reduce_min_sync(0xffffffffu, q.live ? q.doc : 0x7FFFFFFF);
    doc_max = __reduce_max_sync(0xffffffffu, q.live ? q.doc : static_cast<int>(0x80000000));
  }
};

// Columns (of 32, one per lane) that may attend this thread's key row.
__device__ __forceinline__ uint32_t query_bits(const QueryCol& q, bool use_pos, int pos, bool use_doc, int doc) {
  uint32_t bits = 0xFFFFFFFFu;
  if (use_pos) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (pos <= __shfl_sync(0xffffffffu, q.last, i)) b |= 1u << i;
    bits = b;
  }
  if (use_doc) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (__shfl_sync(0xffffffffu, q.doc, i) == doc) b |= 1u << i;
    bits &= doc >= 0 ? b : 0u;
  }
  return bits;
}

// Columns (of 32, one per lane) that the row of this thread may attend: bit i
// set iff column i's position is at most `last` and its document is `doc`.
__device__ __forceinline__ uint32_t key_bits(const KeyCol& k, bool use_pos, int last, bool use_doc, int doc) {
  uint32_t bits = 0xFFFFFFFFu;
  if (use_pos) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (__shfl_sync(0xffffffffu, k.pos, i) <= last) b |= 1u << i;
    bits = b;
  }
  if (use_doc) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (__shfl_sync(0xffffffffu, k.doc, i) == doc) b |= 1u << i;
    bits &= doc >= 0 ? b : 0u;
  }
  return bits;
}

}  // namespace dev
}  // namespace spattn
