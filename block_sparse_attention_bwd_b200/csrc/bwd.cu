// Backward kernels: K2 (Delta = rowsum(dO * O); scored forms: K2b, from the
// weights in rows of few keys), K3 (dK, dV owned per key tile, no atomics) and
// K4 (dQ owned per query tile, no atomics).
//
// Method (KPage abstract, "KPage: block-sparse attention for partially
// occupied 3D blocks", zhuanzhiai.com, abstract paragraph): the backward pass
// keeps the sparse graph exact by letting the K/V side own its pages.  Here
// the key side packs its valid 16-row pages into 128-row owned tiles exactly
// as the query side does in the forward pass; each key tile walks the query
// pages that reach it (the transposed lists), so dK and dV are accumulated
// in TMEM and written once.  dQ is computed by a second, query-owned pass
// over the forward page lists.  The gradient formulas are the standard ones
// for softmax attention: P = exp(S - LSE), dV = P^T dO, dP = dO V^T,
// dS = P * (dP - Delta), dK = scale dS^T Q, dQ = scale dS K.
//
// Both tile kernels use 12 warps: warps 0 and 11 are TMA producers (one per
// column tensor), warp 1 allocates TMEM and issues the two products of each
// step that read the column tiles, warp 10 issues the accumulating products,
// and warps 2..9 turn each step's scores into P / dS, one tile row per lane,
// two warp groups per step (32 columns each).
//
// Scored forms (spattn_score): P from the modified scores z, dS = P (dP - Delta)
// (1 - tanh^2), four warp groups of 16 columns, -LSE, positions and documents of the
// columns in lines beside the stages.  Bound: the row threads' instructions and the
// latency of a step (tensor pipe busy 0.39 in dK / dV and 0.30 in dQ; with 96 registers a
// thread the D = 128 forms of dK / dV spill, 80 bytes of stores and 52 of loads).  12289
// causal tokens with a prefix and a cap of 50, 16 heads over 4, D = 128: dK / dV 1740 us
// and dQ 1475 in a long run (1695 and 1435 in a short one; there masks alone take 1455
// and 1040, unmodified 1240 and 905).
#include <algorithm>
#include <type_traits>

#include "kernels.cuh"
#include "score.cuh"
#include "tile.cuh"

namespace spattn {
namespace {

using namespace dev;

// ----------------------------------------------------------------------------
// K2: Delta
// ----------------------------------------------------------------------------
template <int D>
__global__ void delta_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ d_o,
                             float* __restrict__ delta, int64_t rows) {
  constexpr int TPR = D / 8;  // threads per row, 8 bf16 (16 B) each
  const int64_t total = rows * TPR;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;  // multiple of 32
  const int lane = threadIdx.x & 31;
  // warp-uniform loop so that the group shuffles below always see full warps
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + (threadIdx.x & ~31); t0 < total; t0 += stride) {
    const int64_t t = t0 + lane;
    const int64_t row = t / TPR;
    const int part = static_cast<int>(t % TPR);
    float acc = 0.f;
    if (t < total) {
      const uint4 a = *reinterpret_cast<const uint4*>(o + row * D + part * 8);
      const uint4 b = *reinterpret_cast<const uint4*>(d_o + row * D + part * 8);
      const __nv_bfloat162* pa = reinterpret_cast<const __nv_bfloat162*>(&a);
      const __nv_bfloat162* pb = reinterpret_cast<const __nv_bfloat162*>(&b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 fa = __bfloat1622float2(pa[i]);
        const float2 fb = __bfloat1622float2(pb[i]);
        acc = fmaf(fa.x, fb.x, acc);
        acc = fmaf(fa.y, fb.y, acc);
      }
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off, TPR);
    if (t < total && part == 0) delta[row] = acc;
  }
}

// ----------------------------------------------------------------------------
// Start of a scored backward
// ----------------------------------------------------------------------------
// In one launch: the scan for rows of few keys (see K2b below), Delta, the work-item counter
// of the dK / dV kernel, and the zero rows that no work item writes.  n_scan blocks scan
// one query-owned item each, n_delta form Delta, one warp-row group per pass as above, and
// the others take (fill entry, batch*head) pairs.  The first two take turns, so that the
// scan's waits and Delta's bytes meet on an SM.
constexpr int kFewKeys = 127;   // (255 took dQ of documents from 0.239% to 0.238% and their backward from 685 to 748 us)
constexpr int kFewPages = 16;   // pages per pass of the scan

struct PrepArgs {
  const __nv_bfloat16* o;
  const __nv_bfloat16* d_o;
  float* delta;
  int64_t rows;
  int64_t n_scan;
  int short_entries;  // items of no more are not scanned
  int n_delta;
  int* sched;
  FillArgs q, k;  // dQ; dK and dV
  // the scan's side
  const int32_t* work;
  const int32_t* pages;
  const uint64_t* masks;
  int64_t q_slots, kv_slots;
  int heads;
  const int32_t* order;
  FewList few;
  ScoreArgs sc;
};

// Range over the 16 lanes of a half warp.
__device__ __forceinline__ int2 half_range(bool live, int lo, int hi) {
  if (!live) lo = 0x7FFFFFFF, hi = static_cast<int>(0x80000000);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  return make_int2(lo, hi);
}

// One item: thread r < 128 counts row r's allowed keys over the item's list, sixteen
// pages at a time, until every row has more than kFewKeys or the list ends; most rows
// leave in the first pass.  Pairs are compared one by one only in pages that their range
// leaves open.
__device__ void scan_few_keys(const PrepArgs& a, int64_t item) {
  __shared__ __align__(16) int s_pos[kFewPages * 16];  // positions and documents of a pass, a thread each
  __shared__ __align__(16) int s_doc[kFewPages * 16];
  __shared__ int4 s_rng[kFewPages];
  __shared__ uint4 s_mask[kFewPages];
  const ScoreArgs& sc = a.sc;
  const Work wk = load_work(a.work, a.order ? __ldg(a.order + item) : item);
  const int n_cols = wk.e1 - wk.e0;
  if (n_cols <= a.short_entries) return;
  const int row = threadIdx.x, lane = lane_id();
  const int64_t k_off = (wk.bh / a.heads) * sc.k_batch;
  const bool masked = sc.q_last || sc.q_doc;
  auto page_of = [&](int e) { return masked && e < n_cols ? __ldg(a.pages + wk.e0 + e) : 0; };
  auto mask_of = [&](int e) {
    return row < kFewPages && e < n_cols
               ? __ldg(reinterpret_cast<const uint4*>(a.masks + 2 * (static_cast<int64_t>(wk.e0) + e)))
               : make_uint4(0, 0, 0, 0);
  };
  int page = page_of(row >> 4);
  uint4 words = mask_of(row);
  const bool own = row < 16 * wk.n_own;
  const uint32_t code = own ? wk.row_code(row) : 15u;
  const int64_t slot = own ? pref_slot(wk.own_page(row >> 4), row & 15) : a.q_slots;
  const bool real = code < 8u && slot < a.q_slots;
  bool open = real;  // the row may yet turn out to have few keys
  int last = 0, doc = -1, n = 0, first_e = 0, last_e = 0;
  uint64_t seen = 0;  // entries with an allowed key, from the first one on
  if (open) {
    const int64_t off = (wk.bh / a.heads) * sc.q_batch + slot;
    if (sc.q_last) last = __ldg(sc.q_last + off);
    if (sc.q_doc) doc = __ldg(sc.q_doc + off);
  }
  const int4 mine = make_int4(last, last, doc, doc);
  for (int e0 = 0; e0 < n_cols; e0 += kFewPages) {
    if (!__syncthreads_or(open)) break;
    if (masked) {
      const int e = e0 + (row >> 4);
      const int64_t ks = pref_slot(page, row & 15);
      const bool live = e < n_cols && ks < a.kv_slots;
      const int64_t off = k_off + (live ? ks : 0);
      const int pos = sc.q_last ? __ldg(sc.k_pos + off) : 0, kd = sc.q_doc ? __ldg(sc.k_doc + off) : 0;
      s_pos[row] = pos;
      s_doc[row] = kd;
      const int2 rp = half_range(live, pos, pos), rd = half_range(live, kd, kd);
      if ((lane & 15) == 0) s_rng[row >> 4] = make_int4(rp.x, rp.y, rd.x, rd.y);
      page = page_of(e + kFewPages);
    }
    if (row < kFewPages) s_mask[row] = words;
    words = mask_of(e0 + kFewPages + row);
    __syncthreads();
    for (int j = 0; open && j < min(kFewPages, n_cols - e0); ++j) {
      uint32_t m = reinterpret_cast<const uint16_t*>(&s_mask[j])[code];
      if (m == 0u) continue;
      if (masked) {
        const int4 rg = s_rng[j];
        if (query_none(sc, rg, mine)) continue;
        if (!query_all(sc, rg, mine)) m &= column_bits<true, 16>(sc.q_last, sc.q_doc, s_pos + 16 * j, s_doc + 16 * j, last, doc);
        if (m == 0u) continue;
      }
      if (n == 0) first_e = e0 + j;
      last_e = e0 + j;
      if (last_e - first_e < 64) seen |= 1ull << (last_e - first_e);
      n += __popc(m);
      open = n <= kFewKeys;
    }
  }
  if (row >= kRows) return;
  const bool few = real && open && n > 0;
  const uint32_t bits = __ballot_sync(0xffffffffu, few);
  const int2 span = half_range(few, first_e, last_e);
  const bool far = span.y - span.x >= 64;
  uint64_t x = few && !far ? seen << (first_e - span.x) : 0;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) x |= __shfl_xor_sync(0xffffffffu, x, off);
  const uint32_t rows = (bits >> (lane & 16)) & 0xFFFFu;
  if ((lane & 15) == 0 && rows != 0u) {
    FewPage p;
    p.page = static_cast<int>(a.order ? __ldg(a.order + item) : item) * 8 + (row >> 4);
    p.rows = far ? rows | kFewFar : rows;
    p.first = span.x;
    p.pad = 0;
    p.entries = x;
    p.pad2 = 0;
    const int i = atomicAdd(a.few.counts, 1);
    if (i < a.few.cap) a.few.pages[i] = p;
  }
}

template <int D>
__global__ void __launch_bounds__(256) prep_kernel(const PrepArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // Delta of rows with few keys waits on its own
  const int64_t turns = 2 * min(a.n_scan, static_cast<int64_t>(a.n_delta));
  const bool scan = blockIdx.x < turns ? (blockIdx.x & 1) == 0 : blockIdx.x - turns / 2 < a.n_scan;
  if (scan) return scan_few_keys(a, blockIdx.x < turns ? blockIdx.x / 2 : blockIdx.x - turns / 2);
  const int64_t block = blockIdx.x < turns ? blockIdx.x / 2 : blockIdx.x - a.n_scan;  // of those that form Delta
  if (block >= a.n_delta) {
    const int64_t first = block - a.n_delta, step = gridDim.x - a.n_scan - a.n_delta;
    for (int64_t i = first; i < a.q.n * a.q.bh; i += step) fill_rows<D>(a.q, i % a.q.n, i / a.q.n);
    for (int64_t i = first; i < a.k.n * a.k.bh; i += step) fill_rows<D>(a.k, i % a.k.n, i / a.k.n);
    return;
  }
  if (block == 0 && threadIdx.x == 0) *a.sched = 0;
  constexpr int TPR = D / 8;
  const int64_t total = a.rows * TPR, stride = static_cast<int64_t>(a.n_delta) * blockDim.x;
  const int lane = threadIdx.x & 31;
  for (int64_t t0 = block * blockDim.x + (threadIdx.x & ~31); t0 < total; t0 += stride) {
    const int64_t t = t0 + lane;
    float acc = 0.f;
    if (t < total) {
      const uint4 x = *reinterpret_cast<const uint4*>(a.o + t * 8);
      const uint4 y = *reinterpret_cast<const uint4*>(a.d_o + t * 8);
      const __nv_bfloat162* px = reinterpret_cast<const __nv_bfloat162*>(&x);
      const __nv_bfloat162* py = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 fx = __bfloat1622float2(px[i]), fy = __bfloat1622float2(py[i]);
        acc = fmaf(fx.x, fy.x, acc);
        acc = fmaf(fx.y, fy.y, acc);
      }
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off, TPR);
    if (t < total && t % TPR == 0) a.delta[t / TPR] = acc;
  }
}

// ----------------------------------------------------------------------------
// K2b: Delta of rows with few keys (scored forms)
// ----------------------------------------------------------------------------
// Delta = dO.O inherits the rounding of O, 2^-9 of |dO| |O| or so.  In a row of very many
// keys O is small against V and that is lost in the rounding of dS; in a row of few,
// dP - Delta is a difference of like numbers.  Simulated at D = 128 with scores of
// deviation 1.5, dQ is off by 0.43% with 2 keys, 0.29% with 8, 0.265% with 16, 0.25% with 64
// and 0.245% with 256, of which its own roundings are 0.235%.  So a row with up to 127
// allowed keys, masks included, gets
//   Delta_i = sum_j P_ij dP_ij / sum_j P_ij
// from the weights themselves, in fp32.  Items of short lists get that as a whole, in 128-row
// tiles (dq_kernel's DELTA form); here are the rows of longer items, such as a
// document's first ones behind the pages of another.
//
// The scan lists the 16-row owned pages that hold such rows, in any order, and warps take
// them from a counter, since they are few, stand together and differ in cost.  A warp walks
// the entries of the list that have a key of its page's rows, alone, so that a row's sums
// have one order whatever else the call holds.  S and dP of 16 rows x 16 keys are m16n8k16
// products whose operands come from global memory in 16-byte pieces (the order of the
// inner dimension is free as long as both sides have the same).  A tile for tcgen05 would
// be 128 rows, of which a page is an eighth and its neighbours have other keys; here the
// loads' latency decides, not the products.
//
// 16 heads, D = 128: 18 us on 16384 tokens in documents of 900 (the scan takes 10 beside
// Delta's 28; the backward went from 664 to 685), 4 where no row has few keys (12289
// tokens with a prefix: 3090 to 3120).
struct FewArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* d_o;
  const float* lse;
  float* delta;
  const int32_t* work;
  const int32_t* pages;
  const uint64_t* masks;
  FewList few;
  int64_t q_slots, kv_slots;
  int heads, kv_group;
  float scale;
  ScoreArgs sc;
};

// d += a b, 16 x 8 x 16, bf16 in, fp32 out
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kFewThreads = 128;

template <int D>
__global__ void __launch_bounds__(kFewThreads, 3) few_keys_kernel(const FewArgs a) {
  constexpr int NC = D / 32;  // 64-byte pieces of a row, 16 bytes of each per lane
  const ScoreArgs& sc = a.sc;
  const int lane = lane_id();
  const int quad = lane >> 2, part = lane & 3;  // this lane's rows are quad and quad + 8, its keys 2 part, 2 part + 1 (+ 8)
  const int mine = lane & 15;                   // the row (or column) whose arrays this lane holds
  // (the pass over short items, which waits for the end of this kernel)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the list and every row's Delta are there when the kernel before has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int count = min(*reinterpret_cast<volatile int*>(a.few.counts), a.few.cap);
  if (count == 0) return;
  for (;;) {
    int next = 0;
    if (lane == 0) next = atomicAdd(a.few.counts + 1, 1);
    next = __shfl_sync(0xffffffffu, next, 0);
    if (next >= count) break;
    const FewPage rec = a.few.pages[next];
    const uint32_t few = rec.rows;
    const bool far = (few & kFewFar) != 0u;
    const int first = rec.first;
    const Work wk = load_work(a.work, rec.page >> 3);
    const int pg = rec.page & 7;
    const int batch = wk.bh / a.heads;
    const int kv_bh = batch * (a.heads / a.kv_group) + (wk.bh % a.heads) / a.kv_group;
    const int own = wk.own_page(pg);
    // this lane's row of the page; rows that are not asked for read the first one that is
    const bool asked = (few >> mine) & 1u;
    const int64_t slot = min(pref_slot(own, asked ? mine : __ffs(few) - 1), a.q_slots - 1);
    const int64_t row = static_cast<int64_t>(wk.bh) * a.q_slots + slot;
    const int seg = asked ? static_cast<int>(wk.row_code(16 * pg + mine)) : 0;
    const int64_t q_off = batch * sc.q_batch + slot;
    const int last = sc.q_last ? __ldg(sc.q_last + q_off) : 0, doc = sc.q_doc ? __ldg(sc.q_doc + q_off) : 0;
    const float pos = sc.slopes ? static_cast<float>(__ldg(sc.q_pos + q_off)) : 0.f, lse = __ldg(a.lse + row);
    const float slope = sc.slopes ? __ldg(sc.slopes + wk.bh % a.heads) : 0.f;
    uint4 q[2][NC], d_o[2][NC];
    float row_pos[2], row_lse[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = __shfl_sync(0xffffffffu, row, quad + 8 * h);
      row_pos[h] = __shfl_sync(0xffffffffu, pos, quad + 8 * h);
      row_lse[h] = __shfl_sync(0xffffffffu, lse, quad + 8 * h);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        q[h][c] = __ldg(reinterpret_cast<const uint4*>(a.q + r * D) + 4 * c + part);
        d_o[h][c] = __ldg(reinterpret_cast<const uint4*>(a.d_o + r * D) + 4 * c + part);
      }
    }
    float sum[2] = {0.f, 0.f}, dsum[2] = {0.f, 0.f};
    auto entry = [&](int e, int page) {
      const int64_t ks = pref_slot(page, mine);  // this lane's column
      const int64_t k_off = batch * sc.k_batch + (ks < a.kv_slots ? ks : 0);
      const float k_pos = sc.slopes ? static_cast<float>(__ldg(sc.k_pos + k_off)) : 0.f;
      const int cp = sc.q_last ? __ldg(sc.k_pos + k_off) : 0, cd = sc.q_doc ? __ldg(sc.k_doc + k_off) : 0;
      uint32_t m = asked ? __ldg(reinterpret_cast<const uint16_t*>(a.masks + 2 * (static_cast<int64_t>(wk.e0) + e)) + seg) : 0u;
      uint4 kk[2][NC], vv[2][NC];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int64_t kr = static_cast<int64_t>(kv_bh) * a.kv_slots + min(pref_slot(page, quad + 8 * t), a.kv_slots - 1);
#pragma unroll
        for (int c = 0; c < NC; ++c) kk[t][c] = __ldg(reinterpret_cast<const uint4*>(a.k + kr * D) + 4 * c + part);
#pragma unroll
        for (int c = 0; c < NC; ++c) vv[t][c] = __ldg(reinterpret_cast<const uint4*>(a.v + kr * D) + 4 * c + part);
      }
      // this lane's row's allowed columns
      if (sc.q_last) {
        uint32_t ok = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) ok |= __shfl_sync(0xffffffffu, cp, i) <= last ? 1u << i : 0u;
        m &= ok;
      }
      if (sc.q_doc) {
        uint32_t ok = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) ok |= __shfl_sync(0xffffffffu, cd, i) == doc ? 1u << i : 0u;
        m &= doc >= 0 ? ok : 0u;
      }
      const uint32_t bits[2] = {__shfl_sync(0xffffffffu, m, quad), __shfl_sync(0xffffffffu, m, quad + 8)};
      float s[2][4] = {}, dp[2][4] = {};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma_16x8x16(s[t], q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y, kk[t][c].x, kk[t][c].y);
          mma_16x8x16(s[t], q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w, kk[t][c].z, kk[t][c].w);
          mma_16x8x16(dp[t], d_o[0][c].x, d_o[1][c].x, d_o[0][c].y, d_o[1][c].y, vv[t][c].x, vv[t][c].y);
          mma_16x8x16(dp[t], d_o[0][c].z, d_o[1][c].z, d_o[0][c].w, d_o[1][c].w, vv[t][c].z, vv[t][c].w);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 8 * t + 2 * part + j;
          const float kp = __shfl_sync(0xffffffffu, k_pos, col);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float z = s[t][2 * h + j] * a.scale;
            if (sc.cap > 0.f) {
              const float u = z / sc.cap;
              if (!(fabsf(u) < 1e-4f)) z = sc.cap * tanhf(u);  // (tanh u = u to 3e-9 there, and u may leave fp32's normals)
            }
            if (sc.slopes) z -= slope * fabsf(row_pos[h] - kp);
            const float p = (bits[h] >> col) & 1u ? expf(z - row_lse[h]) : 0.f;
            sum[h] += p;
            if (p != 0.f) dsum[h] = fmaf(p, dp[t][2 * h + j], dsum[h]);
          }
        }
      }
    };
    const int n_cols = wk.e1 - wk.e0;
    for (int w = first; w < (far ? n_cols : min(n_cols, first + 1)); w += 64) {
      uint64_t left = (far ? ~0ull : rec.entries) & ~0ull >> max(0, 64 - (n_cols - w));
      int e = w + __ffsll(left) - 1;
      int page = left != 0 ? __ldg(a.pages + wk.e0 + e) : 0;
      while (left != 0) {
        left &= left - 1;
        const int e_next = w + __ffsll(left) - 1;
        const int page_next = left != 0 ? __ldg(a.pages + wk.e0 + e_next) : 0;
        entry(e, page);
        e = e_next;
        page = page_next;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 1; off < 4; off *= 2) {
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], off);
        dsum[h] += __shfl_xor_sync(0xffffffffu, dsum[h], off);
      }
      const int r = quad + 8 * h;
      const int64_t at = __shfl_sync(0xffffffffu, row, r);
      if (part == 0 && ((few >> r) & 1u) && sum[h] > 0.f) a.delta[at] = dsum[h] / sum[h];  // (NaN scores: dO.O, which is NaN)
    }
  }
  // the last CTA leaves the counts at zero for the next call
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.few.counts + 2, 1) == static_cast<int>(gridDim.x) - 1) {
      a.few.counts[0] = a.few.counts[1] = a.few.counts[2] = 0;
    }
  }
}

// ----------------------------------------------------------------------------
// K3: dK, dV (key-owned tiles, query pages as columns, 64 columns per step)
// ----------------------------------------------------------------------------
// TMEM columns: one fp32 staging set (S^T at 0, dP^T at 64), two packed
// bf16 operand sets (P^T at 128 + 64p, dS^T at 160 + 64p), dV at 256, dK at
// 256 + D.  The staging set is free again as soon as the row threads have
// loaded it, so the S^T / dP^T MMAs of step c+1 run while the row threads
// compute step c; the packed set of step c is reused two steps later, after
// the dV / dK MMAs that read it.
//
// Column tiles arrive in stages of one 64-column MMA step (dK / dV) or two
// (dQ, 128 rows, one 32 KB box): a TMA request holds its issuing thread for
// a long time whatever its size, so larger stages keep a producer ahead of the
// tensor core, while more stages give more slack between a stage's release
// and its reuse; dK / dV have room for four 64-row stages per tensor only.
//
// The per-column terms of the backward pass are folded into the two MMAs
// with one extra K = 16 slice each, so the row threads read nothing but
// TMEM: with x = LSE / scale of query column c, split into three bf16 terms
// x = h + m + l (exact to about 2^-27 relative),
//   [K | 1 1 1 0..] . [Q | -h -m -l 0..]^T = S^T - x,  sl2 * (S^T - x) = log2 P^T,
//   [V | 1 1 1 0..] . [dO | -Delta split]^T = dP^T - Delta,
// both accumulated in fp32.  The slices are 16 bf16 wide, in the plain
// (unswizzled) K-major layout: a 128-row block of ones shared by both MMAs,
// and one block per Q / dO stage that the producer writes.
constexpr int kBwdStepPages = 4;                  // 64 columns per MMA step
constexpr int kHalfStage = 64 * 128;              // offset of a two-step stage's second step in a chunk
constexpr int kOnesBytes = 128 * 32;              // 128 rows x 16 bf16, plain layout

// Byte offset of row r (first 8 of its 16 elements) in a plain K-major
// 16-wide block: 8-row core matrices of 256 bytes, the second K half 128 B on.
__device__ __forceinline__ uint32_t aug_row_off(int r) { return static_cast<uint32_t>((r >> 3) * 256 + (r & 7) * 16); }

// First 8 elements of an augmented row: -x as three bf16 terms, then zeros.
__device__ __forceinline__ uint4 aug_row(float x) {
  const float h = __bfloat162float(__float2bfloat16_rn(x));
  const float r1 = x - h;
  const float m = __bfloat162float(__float2bfloat16_rn(r1));
  const float l = r1 - m;
  return make_uint4(pack_bf16(-h, -m), pack_bf16(-l, 0.f), 0u, 0u);
}

template <int D>
struct DkvCfg {
  static constexpr int kNch = D / 64;
  static constexpr int kTile = kNch * kChunkBytes;     // owned 128-row tile
  static constexpr int kStagePages = 4;                  // one step per stage
  static constexpr int kStageChunk = kStagePages * 16 * 128;  // one 64-column chunk of a stage
  static constexpr int kStageTile = kNch * kStageChunk;
  static constexpr int kAugStage = kStagePages * 16 * 32;     // plain-layout slice of a stage
  static constexpr int kQStages = (D == 128) ? 4 : 6;
  static constexpr int kDStages = (D == 128) ? 4 : 6;
  static constexpr int kSmem = 2 * kTile + (kQStages + kDStages) * (kStageTile + kAugStage) + kOnesBytes + 1024 + 512;
  // scored forms, per stage: -LSE, last position, document and fp32 position of
  // its 64 query columns, the slopes of its pages, and the ranges of its halves.
  // The producers write them (the dO producer the positions); they are rewritten
  // when the tiles are, after the dV / dK products of the step, which wait for
  // every row thread.
  static constexpr int kColBytes = 4 * 64 * 4 + 16 + 32;
  static constexpr int kScoreBytes = kQStages * kColBytes;
  static_assert(kQStages == kDStages, "both producers fill the same line");
};

// 12 warps: 0 and 11 = TMA producers, 1 = TMEM owner and issuer of the MMAs
// that read the step's column tiles into TMEM (S^T/dP^T or S/dP), 2..9 = two
// groups of row threads, 10 = issuer of the accumulating MMAs (dV/dK or dQ).
// Row group g (warps 2+4g .. 5+4g) handles columns 32g .. 32g+31 of every
// 64-column step (warp w reaches TMEM lanes of quarter w%4).  The tensor
// core accepts only a couple of MMAs ahead of the one it runs, so a single
// issuing warp idles it whenever that warp waits; with two issuers one keeps
// it busy while the other waits.
//
// The scored forms do several times the arithmetic per pair; two row warps per
// scheduler left most of its latency in the open (issue slots 0.38 busy), so they
// split a step over four groups of 16 columns (16 row warps): dK / dV of 12289
// causal tokens 2817 -> 2112 us.
// The producer of the second column tensor (dO stages for dK / dV, V stages for
// dQ; warp 0 produces the Q or K stages) is the last warp: a TMA request holds
// its issuing thread for hundreds of cycles, so one producer for both column
// tensors would set the step time.
template <bool SCORED>
struct BwdWarps {
  static constexpr int kGroups = SCORED ? 4 : 2;
  static constexpr int kRowThreads = 128 * kGroups;
  static constexpr int kAcc = 2 + 4 * kGroups;        // issuer of the accumulating products
  static constexpr int kProd2 = kAcc + 1;
  static constexpr int kThreads = 32 * (kProd2 + 1);
  static constexpr int kItemReaders = 3 + 4 * kGroups;  // warps 1, kAcc, kProd2 and the row warps
};

// Persistent form: one CTA per SM takes work items from a device counter in
// list order (longest first per head), so each SM keeps its rings and TMEM
// across items.  Warp 0 fetches the next item and publishes it in a 4-deep
// queue in shared memory; every other role reads the queue.  Stage, step and
// item counters run across items, so every barrier keeps advancing one phase
// at a time.  At an item boundary the producers load the next item's owned
// K / V (once the last S^T / dP^T products of the previous item have read
// them) and its first stages, and the first S^T / dP^T products of the next
// item run while the row threads finish the previous item and write its dK /
// dV; the accumulating products of the next item wait until those
// accumulators have been read.
constexpr int kItemQueue = 4;

// SC: the scored forms (score.cuh).  A cap has to be applied to the bare
// products, so LSE is not folded into S^T there: the row threads read it per
// column, with the columns' positions and documents, from lines in shared memory
// that the producers fill with each stage (the Delta slice stays).
template <int D, int SC>
__global__ void __launch_bounds__(BwdWarps<SC != kScoreNone>::kThreads, 1)
    dkdv_kernel(const __grid_constant__ TmaPages tm_k, const __grid_constant__ TmaPages tm_v,
                const __grid_constant__ TmaPages tm_q, const __grid_constant__ TmaPages tm_do,
                const int32_t* __restrict__ work, int64_t n_work, int* __restrict__ sched,
                const int32_t* __restrict__ col_pages, const uint64_t* __restrict__ col_masks,
                const float* __restrict__ lse, const float* __restrict__ delta, __nv_bfloat16* __restrict__ out_dk,
                __nv_bfloat16* __restrict__ out_dv, int64_t kv_slots, int64_t q_slots, float sl2, float scale,
                int heads, int kv_heads, int kv_group, const uint16_t* __restrict__ col_heads, int* err,
                const ScoreArgs sc, const int32_t* __restrict__ order) {
  using C = DkvCfg<D>;
  constexpr bool kScored = SC != kScoreNone;
  using W = BwdWarps<kScored>;
  constexpr int QS = C::kQStages, DS = C::kDStages, NP = kBwdStepPages, SP = C::kStagePages;
  static_assert(SP == NP, "one MMA step per stage");
  constexpr int NH = SP * 16 / 32;  // stage columns per producer lane
  constexpr int kStageChunk = C::kStageChunk, kAugStage = C::kAugStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTile;
  uint8_t* sQ = smem + 2 * C::kTile;                 // Q stage s at sQ + s*kStageTile
  uint8_t* sDO = sQ + QS * C::kStageTile;            // dO stage s at sDO + s*kStageTile
  uint8_t* sQa = sDO + DS * C::kStageTile;           // -LSE/scale slice of Q stage s at sQa + s*kAugStage
  uint8_t* sDa = sQa + QS * kAugStage;               // -Delta slice of dO stage s at sDa + s*kAugStage
  uint8_t* sOnes = sDa + DS * kAugStage;             // ones slice of the owned K / V rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOnes + kOnesBytes);
  uint64_t* own_full = bars;          // the item's owned K / V rows have landed
  uint64_t* own_free = own_full + 1;  // the item's last S^T / dP^T products have read them
  uint64_t* q_full = own_free + 1;
  uint64_t* q_empty = q_full + QS;
  uint64_t* do_full = q_empty + QS;
  uint64_t* do_empty = do_full + DS;
  uint64_t* st_full = do_empty + DS;  // S^T, dP^T of a step are in the staging set
  uint64_t* st_free = st_full + 1;    // the row threads have loaded the staging set
  uint64_t* pt_full = st_free + 1;    // [2] P^T, dS^T of a step are in packed set p
  uint64_t* acc_done = pt_full + 2;   // the item's dV, dK products have finished
  uint64_t* acc_free = acc_done + 1;  // the row threads have read the item's dV, dK
  uint64_t* acc_b = acc_free + 1;     // [2] dV, dK MMAs of the steps using packed set p finished
  uint64_t* drain = acc_b + 2;        // [2] one per issuing warp
  uint64_t* item_full = drain + 2;    // [kItemQueue]
  uint64_t* item_empty = item_full + kItemQueue;  // [kItemQueue]
  int32_t* items = reinterpret_cast<int32_t*>(item_empty + kItemQueue);  // [kItemQueue]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(items + kItemQueue);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  const Abort ab{abort_flag, err};
  const int warp = warp_id(), lane = lane_id();
  // column lines of stage s (scored forms)
  uint8_t* score_smem = reinterpret_cast<uint8_t*>(bars) + 512;
  auto col_lse = [&](int s) { return reinterpret_cast<float*>(score_smem + s * C::kColBytes); };
  auto col_posf = [&](int s) { return col_lse(s) + 64; };
  auto col_last = [&](int s) { return reinterpret_cast<int*>(col_lse(s) + 128); };
  auto col_doc = [&](int s) { return reinterpret_cast<int*>(col_lse(s) + 192); };
  auto col_slope = [&](int s) { return col_lse(s) + 256; };                             // [4]
  auto col_rng = [&](int s) { return reinterpret_cast<int4*>(col_lse(s) + 260); };     // [2]

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(own_full, 1);
    mbar_init(own_free, 1);
    mbar_init(&acc_b[0], 1);
    mbar_init(&acc_b[1], 1);
    mbar_init(&drain[1], 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < DS; ++s) {
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    mbar_init(st_full, kScored ? 2 : 1);  // the products' commit; scored forms: and their issuer
    mbar_init(st_free, W::kRowThreads);
    for (int b = 0; b < 2; ++b) mbar_init(&pt_full[b], W::kRowThreads);
    mbar_init(acc_done, 1);
    mbar_init(acc_free, W::kRowThreads);
    mbar_init(drain, 1);
    for (int s = 0; s < kItemQueue; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], W::kItemReaders);
    }
    fence_barrier_init();
  }
  {
    // Slices: the ones block holds 1 1 1 0.. in every row; the Q / dO slices
    // start at zero (their second K half is never written again).
    uint4* sl = reinterpret_cast<uint4*>(sQa);
    constexpr int kN16 = ((QS + DS) * kAugStage + kOnesBytes) / 16;
    constexpr int kOnes0 = (QS + DS) * kAugStage / 16;
    for (int i = threadIdx.x; i < kN16; i += W::kThreads) {
      const bool one = i >= kOnes0 && ((i - kOnes0) & 15) < 8;  // first K half of a ones row
      sl[i] = one ? make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tDV = tmem + 256, tDK = tmem + 256 + D;
  // The scored dQ kernel needs nothing from this one: once every CTA is here (all
  // are resident), its CTAs may take the SMs that are free or become so.
  if constexpr (kScored) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Item k of this CTA (k = 0, 1, ...): the readers wait for its queue slot,
  // read it and release the slot; -1 ends the loop (also on abort).
  auto read_item = [&](int k) -> int {
    const int s = k % kItemQueue;
    if (!__all_sync(0xffffffffu, mbar_wait(&item_full[s], (k / kItemQueue) & 1, ab))) return -1;
    const int idx = *reinterpret_cast<volatile int32_t*>(&items[s]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[s]);
    return idx;
  };

  if (warp == 0 || warp == W::kProd2) {
    // ---------------- producers (whole warps): warp 0 = Q stages, warp 11 = dO stages ----------------
    // Warp 0 also owns the item queue and loads each item's owned K / V rows.
    // Lane j < n owns page j of a stage: it holds the page id (fetched one
    // stage ahead) and issues that page's TMA boxes; every lane also writes
    // the augmented slice rows of two of the stage's 64 query columns.
    const bool is_q = warp == 0;
    const int NS = is_q ? QS : DS;
    uint8_t* stage0 = is_q ? sQ : sDO;
    uint8_t* aug0 = is_q ? sQa : sDa;
    uint64_t* full = is_q ? q_full : do_full;
    uint64_t* empty = is_q ? q_empty : do_empty;
    const TmaPages& tm = is_q ? tm_q : tm_do;
    const float* terms = is_q ? lse : delta;
    const float inv_scale = 1.0f / scale;
    if (lane == 0) {
      tma_prefetch_desc(&tm.m64w);
      tma_prefetch_desc(&tm.m64);
      if (is_q) {
        tma_prefetch_desc(&tm_k.m64);
        tma_prefetch_desc(&tm_v.m64);
      }
    }
    int T = 0;  // stages issued by this warp over all items
    int own_loads = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      int idx;
      if (is_q) {
        const int s = k % kItemQueue;
        if (k >= kItemQueue && !__all_sync(0xffffffffu, mbar_wait(&item_empty[s], ((k / kItemQueue) - 1) & 1, ab)))
          break;
        int v = 0;
        if (lane == 0) {
          v = atomicAdd(sched, 1);
          v = v < n_work ? (kScored && order ? __ldg(order + v) : v) : -1;
          items[s] = v;
          mbar_arrive(&item_full[s]);
        }
        idx = __shfl_sync(0xffffffffu, v, 0);
      } else {
        idx = read_item(k);
      }
      if (idx < 0) break;
      const Work wk = load_work(work, idx);
      const int n_cols = wk.e1 - wk.e0;
      if (is_q) {
        // owned K / V rows: their buffers are free once the previous item's
        // last S^T / dP^T products have read them
        if (k >= 1 && !__all_sync(0xffffffffu, mbar_wait(own_free, (k - 1) & 1, ab))) break;
        if (lane == 0) mbar_arrive_expect_tx(own_full, 2 * wk.n_own * C::kNch * 2048);
        __syncwarp();
        const int own_pid = lane < wk.n_own ? wk.own_page(lane) : 0;
        load_page_runs<C::kNch>(sK, kChunkBytes, tm_k, own_pid, wk.n_own, wk.bh, own_full);
        load_page_runs<C::kNch>(sV, kChunkBytes, tm_v, own_pid, wk.n_own, wk.bh, own_full);
        own_loads = k + 1;
      }
      // Lane j holds the page id of column page j of stages t and t+1, and the
      // per-column term (LSE for Q, Delta for dO) of columns lane + 32h of
      // stage t.  Both are fetched one stage ahead, and the fetched values are
      // used only in the next iteration, so their global-load latency overlaps
      // the waits and TMA issue of the current one instead of stalling it.
      const int n_stages = (n_cols + SP - 1) / SP;
      auto page_id = [&](int t) {
        return (t < n_stages && lane < min(SP, n_cols - t * SP)) ? __ldg(col_pages + wk.e0 + t * SP + lane) : 0;
      };
      // Query head of a column page: the item's K/V head owns the query heads
      // q_base .. q_base + kv_group - 1 (grouped-query attention); each entry
      // names its offset.
      const int q_base = (wk.bh / kv_heads) * heads + (wk.bh % kv_heads) * kv_group;
      auto col_bh = [&](int t) {
        return q_base + ((col_heads && t < n_stages && lane < min(SP, n_cols - t * SP))
                             ? static_cast<int>(__ldg(col_heads + wk.e0 + t * SP + lane))
                             : 0);
      };
      // Raw loads only (nothing here reads the loaded registers); a dead
      // column (beyond the stage or the tensor) loads a valid address and is
      // zeroed where the value is used, through its bit in `live`.
      auto fetch_terms = [&](int t, int pg_lane, int bh_lane, float (&x)[NH], uint32_t& live) {
        const int n_t = min(SP, n_cols - t * SP);
        live = 0u;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const int idx2 = lane + 32 * h;  // column of the stage
          const int pg = __shfl_sync(0xffffffffu, pg_lane, idx2 >> 4);
          const int cb = __shfl_sync(0xffffffffu, bh_lane, idx2 >> 4);
          const int64_t slot = pref_slot(pg, idx2 & 15);
          const bool okc = t < n_stages && (idx2 >> 4) < n_t && slot < q_slots;
          x[h] = __ldg(terms + static_cast<int64_t>(cb) * q_slots + (okc ? slot : 0));
          live |= okc ? (1u << h) : 0u;
        }
      };
      // Augmented row of a column: -LSE / scale for Q (a column that attends
      // nothing, LSE = -inf, is masked everywhere, like a dead one: zeros; a NaN stays),
      // or -Delta for dO.
      auto term_row = [&](float t, bool okr) {
        const float x = is_q ? t * inv_scale : t;
        return aug_row(okr && fabsf(x) != INFINITY ? x : 0.f);
      };
      int pid = page_id(0), pid_next = page_id(1);
      int cbh = col_bh(0), cbh_next = col_bh(1);
      float xc[NH];
      uint32_t livec;
      fetch_terms(0, pid, cbh, xc, livec);
      // scored forms: the Q producer, which has no slice to write there, also holds
      // the last positions and documents of columns lane + 32h and the slopes of
      // the pages, the dO producer the positions
      int xpos[NH], xlast[NH], xdoc[NH];
      float xslope = 0.f;
      const bool masked = kScored && (sc.q_last || sc.q_doc);
      const bool fetches = kScored && (is_q ? masked || sc.slopes : sc.slopes != nullptr);
      const int64_t q_off = (wk.bh / kv_heads) * sc.q_batch;
      const int head0 = (wk.bh / kv_heads) * heads;
      auto fetch_cols = [&](int t, int pg_lane, int bh_lane) {
        if constexpr (kScored) {
          if (!fetches) return;
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const int idx2 = lane + 32 * h;
            const int64_t slot = pref_slot(__shfl_sync(0xffffffffu, pg_lane, idx2 >> 4), idx2 & 15);
            const bool okc = t < n_stages && (idx2 >> 4) < min(SP, n_cols - t * SP) && slot < q_slots;
            const int64_t off = q_off + (okc ? slot : 0);
            if (!is_q) {
              xpos[h] = __ldg(sc.q_pos + off);
            } else {
              xlast[h] = sc.q_last ? __ldg(sc.q_last + off) : 0;
              xdoc[h] = sc.q_doc ? __ldg(sc.q_doc + off) : -1;
            }
          }
          if (is_q && sc.slopes) xslope = __ldg(sc.slopes + bh_lane - head0);
        }
      };
      if constexpr (kScored) fetch_cols(0, pid, cbh);
      for (int t = 0; t < n_stages; ++t, ++T) {
        const int s = T % NS;
        const int n = min(SP, n_cols - t * SP);
        const int pid_next2 = page_id(t + 2);
        const int cbh_next2 = col_bh(t + 2);
        float xn[NH];
        uint32_t liven;
        fetch_terms(t + 1, pid_next, cbh_next, xn, liven);
        if (T >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((T / NS) - 1) & 1, ab))) {
          ok = false;
          break;
        }
        if (!kScored || !is_q) {
#pragma unroll
          for (int h = 0; h < NH; ++h)
            *reinterpret_cast<uint4*>(aug0 + s * kAugStage + aug_row_off(lane + 32 * h)) =
                term_row(xc[h], (livec >> h) & 1u);
          fence_proxy_async_smem();
        }
        if (kScored && is_q) {
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const bool okc = (livec >> h) & 1u;
            // -LSE; -inf for a column behind the list and for a query that attends
            // nothing: its weights are 2^-inf = 0 whatever its scores
            col_lse(s)[lane + 32 * h] = okc && xc[h] != -INFINITY ? -xc[h] * kLog2e : -INFINITY;
            if (masked) {
              col_last(s)[lane + 32 * h] = xlast[h];
              col_doc(s)[lane + 32 * h] = xdoc[h];
              const int4 rg = column_range(okc, xlast[h], xdoc[h]);
              if (lane == 0) col_rng(s)[h] = rg;
            }
          }
          // (before a score is multiplied by sl2, where there is no cap)
          if (sc.slopes && lane < SP) col_slope(s)[lane] = xslope * (SC == kScoreCap ? kLog2e : inv_scale);
        } else if (kScored && sc.slopes) {
#pragma unroll
          for (int h = 0; h < NH; ++h) col_posf(s)[lane + 32 * h] = static_cast<float>(xpos[h]);
        }
        if constexpr (kScored) fetch_cols(t + 1, pid_next, cbh_next);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[s], n * C::kNch * 2048);
        __syncwarp();
        load_page_runs<C::kNch>(stage0 + s * C::kStageTile, kStageChunk, tm, pid, n, cbh, &full[s]);
        pid = pid_next;
        pid_next = pid_next2;
        cbh = cbh_next;
        cbh_next = cbh_next2;
        livec = liven;
#pragma unroll
        for (int h = 0; h < NH; ++h) xc[h] = xn[h];
      }
    }
    // no copy may still be landing in shared memory when the CTA exits
    if (lane == 0) {
      for (int t = max(0, T - NS); t < T; ++t) mbar_wait_drain(&full[t % NS], (t / NS) & 1);
      if (is_q && own_loads > 0) mbar_wait_drain(own_full, (own_loads - 1) & 1);
    }
  } else if (warp == 1) {
    // ---------------- S^T, dP^T issuer (warp-wide; one elected lane issues) ----------------
    const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dv0 = sdesc_sw128(smem_u32(sV), 16, 1024);
    const uint64_t dqk = sdesc_sw128(smem_u32(sQ), 16, 1024);             // Q stages, K-major
    const uint64_t ddk = sdesc_sw128(smem_u32(sDO), 16, 1024);            // dO stages, K-major
    const uint64_t d_ones = sdesc_plain(smem_u32(sOnes), 128, 256);
    const uint64_t d_qa = sdesc_plain(smem_u32(sQa), 128, 256);
    const uint64_t d_da = sdesc_plain(smem_u32(sDa), 128, 256);
    int G = 0;  // steps over all items
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int idx = read_item(k);
      if (idx < 0) break;
      const Work wk = load_work(work, idx);
      const int n_cols = wk.e1 - wk.e0;
      const int n_steps = (n_cols + NP - 1) / NP;
      ok = __all_sync(0xffffffffu, mbar_wait(own_full, k & 1, ab));
      tc_fence_after();
      for (int st = 0; ok && st < n_steps; ++st, ++G) {
        const int qs = G % QS, ds = G % DS;
        const int n = min(NP, n_cols - st * NP);
        const uint32_t idesc_s = idesc_bf16(128, 16 * n, false, false);
        // the staging set is free once the row threads have loaded step G-1
        // (scored forms wait for the tiles first: what follows st_free is the time
        // that the row threads wait for)
        bool w;
        if constexpr (kScored)
          w = mbar_wait_warp(&q_full[qs], (G / QS) & 1, ab) && mbar_wait_warp(&do_full[ds], (G / DS) & 1, ab) &&
              (G < 1 || mbar_wait_warp(st_free, (G - 1) & 1, ab));
        else
          w = (G < 1 || mbar_wait(st_free, (G - 1) & 1, ab)) && mbar_wait(&q_full[qs], (G / QS) & 1, ab);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        const uint64_t bq = sdesc_add(dqk, qs * C::kStageTile);
        const uint64_t bd = sdesc_add(ddk, ds * C::kStageTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_w(tmem, sdesc_add(dk0, (kk >> 2) * kChunkBytes + (kk & 3) * 32),
                    sdesc_add(bq, (kk >> 2) * kStageChunk + (kk & 3) * 32), idesc_s, kk > 0);
        if constexpr (!kScored) umma_ss_w(tmem, d_ones, sdesc_add(d_qa, qs * kAugStage), idesc_s, 1u);
        if constexpr (!kScored) {
          if (!__all_sync(0xffffffffu, mbar_wait(&do_full[ds], (G / DS) & 1, ab))) { ok = false; break; }
          tc_fence_after();
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_w(tmem + 64, sdesc_add(dv0, (kk >> 2) * kChunkBytes + (kk & 3) * 32),
                    sdesc_add(bd, (kk >> 2) * kStageChunk + (kk & 3) * 32), idesc_s, kk > 0);
        umma_ss_w(tmem + 64, d_ones, sdesc_add(d_da, ds * kAugStage), idesc_s, 1u);
        umma_commit_w(st_full);
        if (kScored && lane == 0) mbar_arrive(st_full);
      }
      // the owned K / V buffers are free once these products have read them
      umma_commit_w(own_free);
    }
    umma_commit_w(&drain[0]);
    mbar_wait_drain(&drain[0], 0);
  } else if (warp == W::kAcc) {
    // ---------------- dV, dK issuer (warp-wide; one elected lane issues) ----------------
    const uint64_t dqm = sdesc_sw128(smem_u32(sQ), kStageChunk, 1024);    // Q stages, MN-major
    const uint64_t ddm = sdesc_sw128(smem_u32(sDO), kStageChunk, 1024);   // dO stages, MN-major
    const uint32_t idesc_acc = idesc_bf16(128, D, false, true);
    // P^T of page j of packed set b at 128 + 64b + 8j and dS^T 32 columns on; scored
    // forms: side by side, one store of a row thread
    constexpr uint32_t kPk = kScored ? 16 : 8;
    int G = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int idx = read_item(k);
      if (idx < 0) break;
      const Work wk = load_work(work, idx);
      const int n_cols = wk.e1 - wk.e0;
      const int n_steps = (n_cols + NP - 1) / NP;
      // the accumulators hold the previous item until its row threads read them
      if (k >= 1 && !__all_sync(0xffffffffu, mbar_wait(acc_free, (k - 1) & 1, ab))) break;
      tc_fence_after();
      for (int st = 0; st < n_steps; ++st, ++G) {
        const int b = G & 1, qs = G % QS, ds = G % DS;
        if (!(kScored ? mbar_wait_warp(&pt_full[b], (G >> 1) & 1, ab)
                      : __all_sync(0xffffffffu, mbar_wait(&pt_full[b], (G >> 1) & 1, ab)))) { ok = false; break; }
        tc_fence_after();
        const int n = min(NP, n_cols - st * NP);
        const uint64_t bq = sdesc_add(dqm, qs * C::kStageTile);
        const uint64_t bd = sdesc_add(ddm, ds * C::kStageTile);
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (j < n)
            umma_ts_w(tDV, tmem + 128 + 64 * b + kPk * j, sdesc_add(bd, j * 2048), idesc_acc, (st > 0 || j > 0) ? 1u : 0u);
        umma_commit_w(&do_empty[ds]);
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (j < n)
            umma_ts_w(tDK, tmem + 128 + 64 * b + (kScored ? 8 : 32) + kPk * j, sdesc_add(bq, j * 2048), idesc_acc,
                      (st > 0 || j > 0) ? 1u : 0u);
        umma_commit_w(&q_empty[qs]);
        umma_commit_w(&acc_b[b]);
      }
      if (ok) umma_commit_w(acc_done);  // every item, with or without steps
    }
    umma_commit_w(&drain[1]);
    mbar_wait_drain(&drain[1], 0);
  } else if constexpr (kScored) {
    // ---------------- scored P^T, dS^T (one key row per thread, one page of columns per group) + epilogue ----------------
    constexpr int CW = 64 / W::kGroups;  // 16: group g's columns are page g of the step
    const int grp = (warp - 2) >> 2;
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    int G = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int idx = read_item(k);
      if (idx < 0) break;
      const Work wk = load_work(work, idx);
      const int n_cols = wk.e1 - wk.e0;
      const int n_steps = (n_cols + NP - 1) / NP;
      const uint32_t code = wk.row_code(row);
      const int seg = code < 8 ? static_cast<int>(code) : -1;
      int key_pos = 0, key_doc = -1;
      {
        const int64_t slot = row < 16 * wk.n_own ? pref_slot(wk.own_page(row >> 4), row & 15) : kv_slots;
        if (slot < kv_slots) {
          const int64_t off = (wk.bh / kv_heads) * sc.k_batch + slot;
          if (sc.k_pos) key_pos = __ldg(sc.k_pos + off);
          if (sc.k_doc) key_doc = __ldg(sc.k_doc + off);
        }
      }
      const int4 rows = row_range(seg >= 0, key_pos, key_doc), mine = make_int4(key_pos, key_pos, key_doc, key_doc);
      // this row's mask of the group's page, fetched a step ahead; `left`: entries
      // from the group's page of this step on (a row without a segment has none to read)
      const uint16_t* mask = reinterpret_cast<const uint16_t*>(col_masks + 2 * (static_cast<int64_t>(wk.e0) + grp)) + max(seg, 0);
      int left = n_cols - grp;
      uint32_t m_next = seg >= 0 && left > 0 ? __ldg(mask) : 0u;
      for (int st = 0; st < n_steps; ++st, ++G) {
        const int b = G & 1, qs = G % QS;
        const bool active = left > 0;
        uint32_t m = m_next;
        left -= NP;
        mask += 8 * NP;
        if (seg >= 0 && left > 0) m_next = __ldg(mask);
        ok = mbar_wait_warp(st_full, G & 1, ab);
        if (!ok) break;
        tc_fence_after();
        uint32_t a[CW], d[CW], pk[CW];  // pk: P^T, then dS^T, in bf16
        if (active) {
          tmem_ld16(tmem + lane_off + grp * CW, a);
          tmem_ld16(tmem + 64 + lane_off + grp * CW, d);
          tmem_wait_ld();
        }
        tc_fence_before();
        mbar_arrive(st_free);
        if (active) {
          if (sc.q_last || sc.q_doc) {
            const int4 rg = col_rng(qs)[grp >> 1];
            if (key_none(sc, rg, rows))
              m = 0u;
            else if (__builtin_expect(!key_all(sc, rg, rows), 0) &&
                     __any_sync(0xffffffffu, mixed_row(m, key_none(sc, rg, mine), key_all(sc, rg, mine))))
              m &= column_bits<false, CW>(sc.q_last, sc.q_doc, col_last(qs) + CW * grp, col_doc(qs) + CW * grp, key_pos, key_doc);
          }
          // d = dP^T - Delta (from the augmented product); a = S^T -> log2 P^T
          if constexpr (SC == kScoreCap) cap_scores<true>(a, d, sc.c, m != 0u);
          constexpr bool kCap = SC == kScoreCap;
          if (sc.slopes) bias_scores(a, col_posf(qs) + CW * grp, static_cast<float>(key_pos), col_slope(qs)[grp]);
          add_columns(a, col_lse(qs) + CW * grp, kCap ? 1.0f : sl2);
          weights_and_ds(a, d, m, pk);
        }
        // Packed set b still feeds dV(G-2) / dK(G-2).  Every row thread waits, active
        // or not, so that no arrival for step G can land in the pt_full phase of G-2.
        if (G >= 2 && !mbar_wait_warp(&acc_b[b], ((G - 2) >> 1) & 1, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          tmem_st16(tmem + 128 + 64 * b + lane_off + grp * CW, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&pt_full[b]);
      }
      if (!ok) break;
      // acc_done completes once per item, after the item's last dV / dK products
      ok = __all_sync(0xffffffffu, mbar_wait(acc_done, k & 1, ab));
      if (!ok) break;
      tc_fence_after();
      {
        // groups 0, 1 write the halves of dV, groups 2, 3 those of scale * dK
        const bool owned = code != 15u && row < 16 * wk.n_own;
        const int64_t slot = owned ? pref_slot(wk.own_page(row >> 4), row & 15) : 0;
        const bool write = owned && slot < kv_slots;
        const int half = (grp & 1) * (D / 2);
        const int64_t base = (static_cast<int64_t>(wk.bh) * kv_slots + slot) * D + half;
        const uint32_t tacc = (grp < 2 ? tDV : tDK) + half;
        __nv_bfloat16* out = grp < 2 ? out_dv : out_dk;
        const float mul = grp < 2 ? 1.0f : scale;
#pragma unroll
        for (int pc = 0; pc < D / 64; ++pc) {
          uint32_t r[32] = {};
          if (n_steps > 0) {
            tmem_ld32(tacc + lane_off + pc * 32, r);
            tmem_wait_ld();
          }
          if (write) store_row32(out + base + pc * 32, r, mul, n_steps == 0);
        }
      }
      // the next item's dV / dK products may overwrite the accumulators
      tc_fence_before();
      mbar_arrive(acc_free);
    }
  } else {
    // ---------------- P^T, dS^T (one key row per thread) + epilogue ----------------
    const int grp = (warp - 2) >> 2;  // column half of each step
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    int G = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int idx = read_item(k);
      if (idx < 0) break;
      const Work wk = load_work(work, idx);
      const int n_cols = wk.e1 - wk.e0;
      const int n_steps = (n_cols + NP - 1) / NP;
      const uint32_t code = wk.row_code(row);
      const int seg = code < 8 ? static_cast<int>(code) : -1;
      StepMasks<NP> raw;
      if (n_steps > 0) raw.fetch(col_masks, wk.e0, min(NP, n_cols), seg);
      for (int st = 0; st < n_steps; ++st, ++G) {
        const int b = G & 1;
        const int N = 16 * min(NP, n_cols - st * NP);
        const bool active = grp * 32 < N;
        uint32_t mw[2];
        raw.bits(mw);
        // mask words of the next step load while this one computes
        if (st + 1 < n_steps) raw.fetch(col_masks, wk.e0 + (st + 1) * NP, min(NP, n_cols - (st + 1) * NP), seg);
        ok = __all_sync(0xffffffffu, mbar_wait(st_full, G & 1, ab));
        if (!ok) break;
        tc_fence_after();
        uint32_t a[32], d[32];
        if (active) {
          tmem_ld32(tmem + lane_off + grp * 32, a);
          tmem_ld32(tmem + 64 + lane_off + grp * 32, d);
          tmem_wait_ld();
        }
        tc_fence_before();
        mbar_arrive(st_free);
        // a = S^T - LSE/scale, d = dP^T - Delta (fp32, from the augmented MMAs)
        uint32_t pp[16], pd[16];
        if (active) {
          const uint32_t m = grp ? mw[1] : mw[0];
          if (m == 0xFFFFFFFFu) {
            // every column allowed: no masking, all values finite
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1, s0, s1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])), sl2x2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]))), s0,
                        s1);
              pp[i] = pack_bf16(p0, p1);
              pd[i] = pack_bf16(s0, s1);
            }
          } else if (m == 0u) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              pp[i] = 0u;
              pd[i] = 0u;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1, s0, s1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])), sl2x2), x0, x1);
              float p0 = ex2(x0), p1 = ex2(x1);
              if (!((m >> (2 * i)) & 1u)) p0 = 0.f;
              if (!((m >> (2 * i + 1)) & 1u)) p1 = 0.f;
              f2_unpack(f2_mul(f2_pack(p0, p1), f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]))), s0,
                        s1);
              pp[i] = pack_bf16(p0, p1);
              // masked entries: p = 0 exactly, so dS = 0 unless dP - Delta is not finite
              pd[i] = pack_bf16(p0 != 0.f ? s0 : 0.f, p1 != 0.f ? s1 : 0.f);
            }
          }
        }
        // Packed set b still feeds dV(G-2) / dK(G-2).  Every row thread
        // waits, active or not, so that no arrival for step G can land in
        // the pt_full phase of step G-2.
        if (G >= 2 && !__all_sync(0xffffffffu, mbar_wait(&acc_b[b], ((G - 2) >> 1) & 1, ab))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          tmem_st16(tmem + 128 + 64 * b + lane_off + grp * 16, pp);
          tmem_st16(tmem + 160 + 64 * b + lane_off + grp * 16, pd);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&pt_full[b]);
      }
      if (!ok) break;
      // acc_done completes once per item, after the item's last dV / dK products
      ok = __all_sync(0xffffffffu, mbar_wait(acc_done, k & 1, ab));
      if (!ok) break;
      tc_fence_after();
      {
        // group 0 writes dV, group 1 writes scale * dK
        const bool owned = code != 15u && row < 16 * wk.n_own;
        const int64_t slot = owned ? pref_slot(wk.own_page(row >> 4), row & 15) : 0;
        const bool write = owned && slot < kv_slots;
        const int64_t base = (static_cast<int64_t>(wk.bh) * kv_slots + slot) * D;
        const uint32_t tacc = grp == 0 ? tDV : tDK;
        __nv_bfloat16* out = grp == 0 ? out_dv : out_dk;
        const float mul = grp == 0 ? 1.0f : scale;
#pragma unroll
        for (int pc = 0; pc < D / 32; ++pc) {
          uint32_t r[32] = {};
          if (n_steps > 0) {
            tmem_ld32(tacc + lane_off + pc * 32, r);
            tmem_wait_ld();
          }
          if (write) store_row32(out + base + pc * 32, r, mul, n_steps == 0);
        }
      }
      // the next item's dV / dK products may overwrite the accumulators
      tc_fence_before();
      mbar_arrive(acc_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------------------
// K4: dQ (query-owned tiles, key pages as columns; the forward lists)
// ----------------------------------------------------------------------------
// TMEM columns: the owned Q rows as bf16 pairs at 0 (the A operand of
// S = Q K^T, so that MMA reads only K from shared memory), two fp32 staging
// sets (S at 64 + 64b, dP at 192 + 64b), two packed bf16 dS sets at 320 + 32p,
// dQ at 384.  A staging set is free as soon as the row threads have loaded
// it; a packed set is reused after the dQ MMAs of two steps back.
template <int D>
struct DqCfg {
  static constexpr int kNch = D / 64;
  static constexpr int kTile = kNch * kChunkBytes;        // dO tile (128 rows)
  static constexpr int kStagePages = 8;                   // two steps per stage
  static constexpr int kStageChunk = kStagePages * 16 * 128;
  static constexpr int kStageTile = kNch * kStageChunk;   // 128-row K / V stage
  static constexpr int kKStages = (D == 128) ? 3 : 5;
  static constexpr int kVStages = (D == 128) ? 3 : 5;
  static constexpr int kSmem = kTile + (kKStages + kVStages) * kStageTile + 1024 + 512;
  // scored forms: fp32 positions of each K stage's 128 columns and the ranges of
  // its four half steps.  The positions are all that fits at head_dim 128, so the
  // ranges share the barriers' 512 bytes there.
  static constexpr int kRangeBytes = kKStages * 64;
  static constexpr int kScoreBytes = kKStages * 128 * 4 + (D == 64 ? kRangeBytes : 0);
};

// SC: the scored forms (score.cuh).
//
// DELTA: no dQ, but Delta_i = sum_j P_ij dP_ij for the rows of an item, from the
// weights themselves (see K2b, which does that for single rows of longer items).
// Items of up to 256 listed keys get this pass, every row of them having few; it costs
// a few steps each (9 of 84 us for two rows of 777 tokens with 4 heads) and overwrites
// what Delta = dO.O gave.
template <int D, int SC, bool DELTA>
__global__ void __launch_bounds__(BwdWarps<SC != kScoreNone>::kThreads, 1)
    dq_kernel(const __nv_bfloat16* __restrict__ q, const __grid_constant__ TmaPages tm_do,
              const __grid_constant__ TmaPages tm_k, const __grid_constant__ TmaPages tm_v,
              const int32_t* __restrict__ work, const int32_t* __restrict__ col_pages,
              const uint64_t* __restrict__ col_masks, const float* __restrict__ lse, const float* __restrict__ delta,
              __nv_bfloat16* __restrict__ out_dq, int64_t q_slots, float sl2, float scale, int heads, int kv_group,
              int* err, const ScoreArgs sc, int64_t kv_slots, const int32_t* __restrict__ order, int short_entries,
              float* __restrict__ out_delta) {
  using C = DqCfg<D>;
  constexpr bool kScored = SC != kScoreNone, kCap = SC == kScoreCap;
  using W = BwdWarps<kScored>;
  constexpr int KS = C::kKStages, VS = C::kVStages, NP = kBwdStepPages, SP = C::kStagePages;
  constexpr int SPS = SP / NP;  // steps per stage
  constexpr int kStageChunk = C::kStageChunk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sDO = smem;
  uint8_t* sK = smem + C::kTile;           // K stage s at sK + s*kStageTile
  uint8_t* sV = sK + KS * C::kStageTile;   // V stage s at sV + s*kStageTile
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + VS * C::kStageTile);
  uint64_t* own_full = bars;
  uint64_t* q_ready = own_full + 1;  // Q rows stored into TMEM by the row threads
  uint64_t* k_full = q_ready + 1;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + VS;
  uint64_t* sd_full = v_empty + VS;  // [2] S and dP of a step are in staging set b
  uint64_t* s_free = sd_full + 2;    // [2] the row threads have loaded staging set b
  uint64_t* ds_full = s_free + 2;    // [2] dS of a step is in packed set p
  uint64_t* dq_done = ds_full + 2;   // [2] dQ MMAs of the steps using packed set p finished
  uint64_t* acc_done = dq_done + 2;
  uint64_t* drain = acc_done + 1;    // [2] one per issuing warp
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  const Abort ab{abort_flag, err};
  // column lines of K stage s (scored forms); a stage's are rewritten when its
  // tile is, after the dQ products of its steps, which wait for every row thread
  auto col_posf = [&](int s) { return reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 512) + 128 * s; };
  static_assert(D == 64 || (13 + 2 * (KS + VS)) * 8 + 8 + C::kRangeBytes <= 512, "barriers and ranges share 512 bytes");
  auto col_rng = [&](int s) {  // [4]
    uint8_t* base = reinterpret_cast<uint8_t*>(bars) + 512;
    return reinterpret_cast<int4*>(D == 64 ? base + KS * 512 : base - C::kRangeBytes) + 4 * s;
  };
  const bool use_cols = kScored && (sc.q_last || sc.q_doc || sc.slopes);

  const Work wk = load_work(work, kScored && order ? __ldg(order + blockIdx.x) : blockIdx.x);
  // K/V head of this item's query head (grouped-query attention)
  const int kv_bh = (wk.bh / heads) * (heads / kv_group) + (wk.bh % heads) / kv_group;
  const int n_cols = wk.e1 - wk.e0;
  const int n_steps = (n_cols + NP - 1) / NP;
  const int warp = warp_id(), lane = lane_id();
  if constexpr (DELTA) {
    if (n_cols > short_entries || n_cols == 0) {  // (a row without keys keeps its 0)
      asm volatile("griddepcontrol.wait;" ::: "memory");
      return;
    }
  }

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(own_full, 1);
    mbar_init(q_ready, W::kRowThreads);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sd_full[b], kScored ? 2 : 1);  // the products' commit; scored forms: and their issuer
      mbar_init(&s_free[b], W::kRowThreads);
      mbar_init(&ds_full[b], W::kRowThreads);
      mbar_init(&dq_done[b], 1);
    }
    mbar_init(acc_done, 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tQ = tmem, tDQ = tmem + 384;
  auto tS = [&](int b) { return tmem + 64 + 64 * b; };
  auto tDP = [&](int b) { return tmem + 192 + 64 * b; };
  auto tPk = [&](int p) { return tmem + 320 + 32 * p; };

  if (warp == 0 || warp == W::kProd2) {
    // ---------------- producers (whole warps): warp 0 = K stages, warp 11 = V stages ----------------
    // Lane j owns page j of a 128-row stage; page ids are fetched one stage
    // ahead.
    const bool is_k = warp == 0;
    const int NS = is_k ? KS : VS;
    uint8_t* stage0 = is_k ? sK : sV;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    const TmaPages& tm = is_k ? tm_k : tm_v;
    if (is_k) {
      if (lane == 0) {
        tma_prefetch_desc(&tm_do.m64);
        mbar_arrive_expect_tx(own_full, wk.n_own * C::kNch * 2048);
      }
      __syncwarp();
      load_page_runs<C::kNch>(sDO, kChunkBytes, tm_do, lane < wk.n_own ? wk.own_page(lane) : 0, wk.n_own, wk.bh,
                              own_full);
    }
    if (lane == 0) {
      tma_prefetch_desc(&tm.m64w);
      tma_prefetch_desc(&tm.m64);
    }
    __syncwarp();
    const int n_stages = (n_cols + SP - 1) / SP;
    auto page_of = [&](int t) {
      return (t < n_stages && lane < min(SP, n_cols - t * SP)) ? __ldg(col_pages + wk.e0 + t * SP + lane) : 0;
    };
    int pid_next = page_of(0);
    // scored forms: the K producer's lane l also holds columns l + 32h of a stage,
    // loaded a stage ahead from page ids that are fetched two ahead
    int pid_next2 = 0;
    int cpos[4] = {0, 0, 0, 0}, cdoc[4] = {-1, -1, -1, -1};
    uint32_t clive = 0u;
    auto load_cols = [&](int t, int pid_lane) {
      clive = 0u;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int pg = (lane >> 4) + 2 * h;
        const int64_t slot = pref_slot(__shfl_sync(0xffffffffu, pid_lane, pg), lane & 15);
        const bool live = t < n_stages && t * SP + pg < n_cols && slot < kv_slots;
        const int64_t off = (wk.bh / heads) * sc.k_batch + (live ? slot : 0);
        cpos[h] = sc.k_pos ? __ldg(sc.k_pos + off) : 0;
        cdoc[h] = sc.k_doc ? __ldg(sc.k_doc + off) : -1;
        clive |= live ? 1u << h : 0u;
      }
    };
    const bool cols = use_cols && is_k;
    if (cols) {
      pid_next2 = page_of(1);
      load_cols(0, pid_next);
    }
    int issued = 0;
    for (int t = 0; t < n_stages; ++t) {
      const int s = t % NS;
      const int n = min(SP, n_cols - t * SP);
      const int pid = pid_next;
      if (cols) {
        pid_next = pid_next2;
        pid_next2 = page_of(t + 2);
      } else {
        pid_next = page_of(t + 1);
      }
      if (t >= NS && !__all_sync(0xffffffffu, mbar_wait(&empty[s], ((t / NS) - 1) & 1, ab))) break;
      if (cols) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          col_posf(s)[lane + 32 * h] = static_cast<float>(cpos[h]);
          const int4 rg = column_range((clive >> h) & 1u, cpos[h], cdoc[h]);
          if (lane == 0) col_rng(s)[h] = rg;
        }
        load_cols(t + 1, pid_next);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[s], n * C::kNch * 2048);
      __syncwarp();
      load_page_runs<C::kNch>(stage0 + s * C::kStageTile, kStageChunk, tm, pid, n, kv_bh, &full[s]);
      issued = t + 1;
    }
    if (lane == 0) {
      for (int t = max(0, issued - NS); t < issued; ++t) mbar_wait_drain(&full[t % NS], (t / NS) & 1);
      if (is_k) mbar_wait_drain(own_full, 0);
    }
  } else if (warp == 1) {
    // ---------------- S, dP issuer (warp-wide; one elected lane issues) ----------------
    const uint64_t ddo0 = sdesc_sw128(smem_u32(sDO), 16, 1024);
    const uint64_t dkk = sdesc_sw128(smem_u32(sK), 16, 1024);            // K stages, K-major
    const uint64_t dvk = sdesc_sw128(smem_u32(sV), 16, 1024);            // V stages, K-major
    bool ok = __all_sync(0xffffffffu, mbar_wait(own_full, 0, ab) && mbar_wait(q_ready, 0, ab));
    tc_fence_after();
    for (int st = 0; ok && st < n_steps; ++st) {
      const int b = st & 1, t = st / SPS, half = st % SPS, ks = t % KS, vs = t % VS;
      const bool stage_end = half == SPS - 1 || st + 1 == n_steps;
      const int n = min(NP, n_cols - st * NP);
      const uint32_t idesc_s = idesc_bf16(128, 16 * n, false, false);
      // staging set b is free once the row threads have loaded step st-2
      bool w;
      if constexpr (kScored)
        w = mbar_wait_warp(&k_full[ks], (t / KS) & 1, ab) && mbar_wait_warp(&v_full[vs], (t / VS) & 1, ab) &&
            (st < 2 || mbar_wait_warp(&s_free[b], ((st - 2) >> 1) & 1, ab));
      else
        w = (st < 2 || mbar_wait(&s_free[b], ((st - 2) >> 1) & 1, ab)) && mbar_wait(&k_full[ks], (t / KS) & 1, ab);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      tc_fence_after();
      const uint64_t bk = sdesc_add(dkk, ks * C::kStageTile + half * kHalfStage);
      const uint64_t bv = sdesc_add(dvk, vs * C::kStageTile + half * kHalfStage);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_ts_w(tS(b), tQ + 8 * kk, sdesc_add(bk, (kk >> 2) * kStageChunk + (kk & 3) * 32), idesc_s, kk > 0);
      if constexpr (!kScored) {
        if (!__all_sync(0xffffffffu, mbar_wait(&v_full[vs], (t / VS) & 1, ab))) { ok = false; break; }
        tc_fence_after();
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_ss_w(tDP(b), sdesc_add(ddo0, (kk >> 2) * kChunkBytes + (kk & 3) * 32),
                  sdesc_add(bv, (kk >> 2) * kStageChunk + (kk & 3) * 32), idesc_s, kk > 0);
      if (stage_end) umma_commit_w(&v_empty[vs]);
      umma_commit_w(&sd_full[b]);
      if (kScored && lane == 0) mbar_arrive(&sd_full[b]);
    }
    umma_commit_w(&drain[0]);
    mbar_wait_drain(&drain[0], 0);
  } else if (warp == W::kAcc) {
    // ---------------- dQ issuer (warp-wide; one elected lane issues) ----------------
    const uint64_t dkm = sdesc_sw128(smem_u32(sK), kStageChunk, 1024);   // K stages, MN-major
    const uint32_t idesc_acc = idesc_bf16(128, D, false, true);
    bool ok = true;
    for (int st = 0; ok && st < n_steps; ++st) {
      const int p = st & 1, t = st / SPS, half = st % SPS, ks = t % KS;
      const bool stage_end = half == SPS - 1 || st + 1 == n_steps;
      if (!(kScored ? mbar_wait_warp(&ds_full[p], (st >> 1) & 1, ab)
                    : __all_sync(0xffffffffu, mbar_wait(&ds_full[p], (st >> 1) & 1, ab)))) { ok = false; break; }
      tc_fence_after();
      const int n = min(NP, n_cols - st * NP);
      const uint64_t bk = sdesc_add(dkm, ks * C::kStageTile + half * kHalfStage);
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (!DELTA && j < n) umma_ts_w(tDQ, tPk(p) + 8 * j, sdesc_add(bk, j * 2048), idesc_acc, (st > 0 || j > 0) ? 1u : 0u);
      if (stage_end) umma_commit_w(&k_empty[ks]);
      umma_commit_w(&dq_done[p]);
    }
    if (ok && n_steps > 0) umma_commit_w(acc_done);
    umma_commit_w(&drain[1]);
    mbar_wait_drain(&drain[1], 0);
  } else if constexpr (kScored) {
    // ---------------- scored dS (one query row per thread, one page of columns per group) + epilogue ----------------
    constexpr int NG = W::kGroups, CW = 64 / NG;  // 16: group g's columns are page g of the step
    const int grp = (warp - 2) >> 2;
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t code = wk.row_code(row);
    const int seg = code < 8 ? static_cast<int>(code) : -1;
    const bool owned = code != 15u && row < 16 * wk.n_own;
    const int64_t slot = row < 16 * wk.n_own ? pref_slot(wk.own_page(row >> 4), row & 15) : 0;
    const bool loaded = row < 16 * wk.n_own && slot < q_slots;
    const bool valid_slot = owned && slot < q_slots;
    const int64_t roff = static_cast<int64_t>(wk.bh) * q_slots + slot;
    // Q row into TMEM as bf16 pairs: group g stores pair columns [g*D/8, (g+1)*D/8)
    {
      constexpr int kCols = D / 2 / NG;  // 32-bit TMEM columns per group
      uint32_t qr[kCols] = {};
      if (loaded) {
        const uint4* src = reinterpret_cast<const uint4*>(q + roff * D + grp * (D / NG));
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const uint4 v = __ldg(src + i);
          qr[4 * i] = v.x;
          qr[4 * i + 1] = v.y;
          qr[4 * i + 2] = v.z;
          qr[4 * i + 3] = v.w;
        }
      }
      if constexpr (kCols == 16)
        tmem_st16(tQ + lane_off + grp * kCols, qr);
      else
        tmem_st8(tQ + lane_off + grp * kCols, qr);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(q_ready);
    }
    const float lse_row = (valid_slot && seg >= 0) ? __ldg(lse + roff) : 0.f;
    const float nlse2 = lse_row == -INFINITY ? -INFINITY : -lse_row * kLog2e;  // -inf: no key, every weight 0
    const float dl = (!DELTA && valid_slot && seg >= 0) ? __ldg(delta + roff) : 0.f;
    float delta_sum = 0.f;  // DELTA: this group's part of the row's sum
    // this row's side of the masks and the bias
    int row_last = 0, row_doc = -1;
    float row_pos = 0.f, slope = 0.f;
    if (loaded) {
      const int64_t off = (wk.bh / heads) * sc.q_batch + slot;
      if (sc.q_last) row_last = __ldg(sc.q_last + off);
      if (sc.q_doc) row_doc = __ldg(sc.q_doc + off);
      if (sc.slopes) row_pos = static_cast<float>(__ldg(sc.q_pos + off));
    }
    const float mul = kCap ? 1.0f : sl2;  // after the cap the scores are in log2 units
    if (sc.slopes) slope = __ldg(sc.slopes + wk.bh % heads) * kLog2e / mul;
    const uint64_t m2 = f2_pack(mul, mul);
    const int4 rows = row_range(seg >= 0, row_last, row_doc), mine = make_int4(row_last, row_last, row_doc, row_doc);
    // Bits of this group's 16 columns of a step, compared pair by pair: lanes load
    // one column each (the stage's lines hold fp32 positions only).
    auto step_bits = [&](int st) -> uint32_t {
      const int e = st * NP + grp;
      const int64_t kslot = e < n_cols ? pref_slot(__ldg(col_pages + wk.e0 + e), lane & 15) : kv_slots;
      const int64_t off = (wk.bh / heads) * sc.k_batch + (kslot < kv_slots ? kslot : 0);
      uint32_t bits = (1u << CW) - 1u;
      if (sc.q_last) {
        const int p = __ldg(sc.k_pos + off);
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < CW; ++i) m |= __shfl_sync(0xffffffffu, p, i) <= row_last ? 1u << i : 0u;
        bits = m;
      }
      if (sc.q_doc) {
        const int dc = __ldg(sc.k_doc + off);
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < CW; ++i) m |= __shfl_sync(0xffffffffu, dc, i) == row_doc ? 1u << i : 0u;
        bits &= row_doc >= 0 ? m : 0u;
      }
      return bits;
    };
    // this row's mask of the group's page, fetched a step ahead; `left`: entries
    // from the group's page of this step on (a row without a segment has none to read)
    const uint16_t* mask = reinterpret_cast<const uint16_t*>(col_masks + 2 * (static_cast<int64_t>(wk.e0) + grp)) + max(seg, 0);
    int left = n_cols - grp;
    uint32_t m_next = seg >= 0 && left > 0 ? __ldg(mask) : 0u;
    const uint64_t ndl = f2_pack(-dl, -dl), nl2 = f2_pack(nlse2, nlse2);
    bool ok = true;
    for (int st = 0; st < n_steps; ++st) {
      const int b = st & 1, t = st / SPS, ks = t % KS;
      const bool active = left > 0;
      uint32_t m = m_next;
      left -= NP;
      mask += 8 * NP;
      if (seg >= 0 && left > 0) m_next = __ldg(mask);
      ok = mbar_wait_warp(&sd_full[b], (st >> 1) & 1, ab);
      if (!ok) break;
      if (active && (sc.q_last || sc.q_doc)) {
        const int4 rg = col_rng(ks)[2 * (st % SPS) + (grp >> 1)];
        if (query_none(sc, rg, rows))
          m = 0u;
        else if (__builtin_expect(!query_all(sc, rg, rows), 0) &&
                 __any_sync(0xffffffffu, mixed_row(m, query_none(sc, rg, mine), query_all(sc, rg, mine))))
          m &= step_bits(st);
      }
      tc_fence_after();
      uint32_t a[CW], d[CW], pd[CW / 2];
      if (active) {
        tmem_ld16(tS(b) + lane_off + grp * CW, a);
        tmem_ld16(tDP(b) + lane_off + grp * CW, d);
        tmem_wait_ld();
      }
      tc_fence_before();
      mbar_arrive(&s_free[b]);
      if (active) {
        if constexpr (!DELTA) {
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            float x0, x1;
            f2_unpack(f2_add(f2_pack(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), ndl), x0, x1);
            d[i] = __float_as_uint(x0);
            d[i + 1] = __float_as_uint(x1);
          }
        }
        if constexpr (kCap) cap_scores<!DELTA>(a, d, sc.c, m != 0u);
        if (sc.slopes) bias_scores(a, col_posf(ks) + 64 * (st % SPS) + CW * grp, row_pos, slope);
#pragma unroll
        for (int i = 0; i < CW; i += 2) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), m2, nl2), x0, x1);
          a[i] = __float_as_uint(x0);
          a[i + 1] = __float_as_uint(x1);
        }
        if constexpr (DELTA) {
#pragma unroll
          for (int i = 0; i < CW; ++i)
            if ((m >> i) & 1u) delta_sum = fmaf(ex2(__uint_as_float(a[i])), __uint_as_float(d[i]), delta_sum);
        } else {
          weights_and_ds(a, d, m, pd);
        }
      }
      // Packed set b still feeds dQ(st-2).  Every row thread waits, active or not:
      // dq_done(st-2) implies that ds_full finished the phase of step st-2.
      if (st >= 2 && !mbar_wait_warp(&dq_done[b], ((st - 2) >> 1) & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (!DELTA && active) {
        tmem_st8(tPk(b) + lane_off + grp * (CW / 2), pd);
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&ds_full[b]);
    }
    if (ok && n_steps > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(acc_done, 0, ab));
      tc_fence_after();
    }
    // (the dO tile's last readers, the products of the last step, are done)
    if constexpr (DELTA) reinterpret_cast<float*>(sDO)[128 * grp + row] = delta_sum;
    if (!DELTA && ok) {
      // group g writes columns [g*D/4, (g+1)*D/4) of dQ
      constexpr int kOut = D / NG;  // 32 or 16
      const int col = grp * kOut;
      uint32_t r[kOut] = {};
      if (n_steps > 0) {
        if constexpr (kOut == 32)
          tmem_ld32(tDQ + lane_off + col, r);
        else
          tmem_ld16(tDQ + lane_off + col, r);
        tmem_wait_ld();
      }
      if (valid_slot) store_row(out_dq + roff * D + col, r, scale, n_steps == 0);
    }
  } else {
    const int grp = (warp - 2) >> 2;  // column half of each step
    const int q4 = warp & 3;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t code = wk.row_code(row);
    const int seg = code < 8 ? static_cast<int>(code) : -1;
    const bool owned = code != 15u && row < 16 * wk.n_own;
    const int64_t slot = row < 16 * wk.n_own ? pref_slot(wk.own_page(row >> 4), row & 15) : 0;
    const bool loaded = row < 16 * wk.n_own && slot < q_slots;
    const bool valid_slot = owned && slot < q_slots;
    const int64_t roff = static_cast<int64_t>(wk.bh) * q_slots + slot;
    // Q row into TMEM as bf16 pairs: group g stores pair columns [g*D/4, (g+1)*D/4)
    {
      constexpr int kCols = D / 4;  // 32-bit TMEM columns per group
      uint32_t qr[32] = {};
      if (loaded) {
        const uint4* src = reinterpret_cast<const uint4*>(q + roff * D + grp * (D / 2));
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const uint4 v = __ldg(src + i);
          qr[4 * i] = v.x;
          qr[4 * i + 1] = v.y;
          qr[4 * i + 2] = v.z;
          qr[4 * i + 3] = v.w;
        }
      }
      if (kCols == 32) {
        tmem_st32(tQ + lane_off + grp * kCols, qr);
      } else {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = qr[i];
        tmem_st16(tQ + lane_off + grp * kCols, h);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(q_ready);
    }
    const float lse2 = (valid_slot && seg >= 0) ? __ldg(lse + roff) * kLog2e : 0.f;
    const float dl = (valid_slot && seg >= 0) ? __ldg(delta + roff) : 0.f;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    const uint64_t nl2 = f2_pack(-lse2, -lse2);
    const uint64_t ndl = f2_pack(-dl, -dl);
    bool ok = true;
    StepMasks<NP> raw;
    if (n_steps > 0) raw.fetch(col_masks, wk.e0, min(NP, n_cols), seg);
    for (int st = 0; st < n_steps; ++st) {
      const int b = st & 1;
      const int N = 16 * min(NP, n_cols - st * NP);
      const bool active = grp * 32 < N;
      uint32_t mw[2];
      raw.bits(mw);
      // mask words of the next step load while this one computes
      if (st + 1 < n_steps) raw.fetch(col_masks, wk.e0 + (st + 1) * NP, min(NP, n_cols - (st + 1) * NP), seg);
      ok = __all_sync(0xffffffffu, mbar_wait(&sd_full[b], (st >> 1) & 1, ab));
      if (!ok) break;
      tc_fence_after();
      uint32_t a[32], d[32];
      if (active) {
        tmem_ld32(tS(b) + lane_off + grp * 32, a);
        tmem_ld32(tDP(b) + lane_off + grp * 32, d);
        tmem_wait_ld();
      }
      tc_fence_before();
      mbar_arrive(&s_free[b]);
      uint32_t pd[16];
      if (active) {
        const uint32_t m = grp ? mw[1] : mw[0];
        if (m == 0xFFFFFFFFu) {
          // every column allowed: no masking, all values finite
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1, g0, g1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])), sl2x2, nl2), x0, x1);
            f2_unpack(f2_mul(f2_pack(ex2(x0), ex2(x1)),
                             f2_add(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), ndl)),
                      g0, g1);
            pd[i] = pack_bf16(g0, g1);
          }
        } else if (m == 0u) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pd[i] = 0u;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])), sl2x2, nl2), x0, x1);
            float p0 = ex2(x0), p1 = ex2(x1);
            if (!((m >> (2 * i)) & 1u)) p0 = 0.f;
            if (!((m >> (2 * i + 1)) & 1u)) p1 = 0.f;
            float g0, g1;
            f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])), ndl)),
                      g0, g1);
            pd[i] = pack_bf16(p0 != 0.f ? g0 : 0.f, p1 != 0.f ? g1 : 0.f);
          }
        }
      }
      // Packed set b still feeds dQ(st-2).  Every row thread waits, active or
      // not: dq_done(st-2) implies that ds_full finished the phase of step
      // st-2, so no thread can arrive for step st while that phase is open.
      if (st >= 2 && !__all_sync(0xffffffffu, mbar_wait(&dq_done[b], ((st - 2) >> 1) & 1, ab))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (active) {
        tmem_st16(tPk(b) + lane_off + grp * 16, pd);
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&ds_full[b]);
    }
    if (ok && n_steps > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(acc_done, 0, ab));
      tc_fence_after();
    }
    if (ok) {
      // group g writes columns [g*D/2, (g+1)*D/2) of dQ
      __nv_bfloat16* dst = out_dq + roff * D;
#pragma unroll
      for (int pc = 0; pc < D / 64; ++pc) {
        const int col = grp * (D / 2) + pc * 32;
        uint32_t r[32] = {};
        if (n_steps > 0) {
          tmem_ld32(tDQ + lane_off + col, r);
          tmem_wait_ld();
        }
        if (valid_slot) store_row32(dst + col, r, scale, n_steps == 0);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // launched beside the dK / dV kernel (DELTA: beside the one that writes every
  // row's Delta first): what follows in the stream waits for this kernel only, so
  // this one ends after that one
  if constexpr (kScored) asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (DELTA) {
    const int row = threadIdx.x;
    if (row < 16 * wk.n_own && wk.row_code(row) < 8u && !*abort_flag) {
      const int64_t slot = pref_slot(wk.own_page(row >> 4), row & 15);
      const float* part = reinterpret_cast<const float*>(sDO) + row;
      if (slot < q_slots)
        out_delta[static_cast<int64_t>(wk.bh) * q_slots + slot] = (part[0] + part[128]) + (part[256] + part[384]);
    }
  }
}

}  // namespace

cudaError_t launch_delta(int head_dim, const __nv_bfloat16* o, const __nv_bfloat16* d_o, float* delta, int64_t rows,
                         cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t threads = rows * (head_dim / 8);
  const int64_t blocks = std::min<int64_t>((threads + 255) / 256, 148 * 16);
  if (head_dim == 128)
    delta_kernel<128><<<static_cast<unsigned>(blocks), 256, 0, st>>>(o, d_o, delta, rows);
  else
    delta_kernel<64><<<static_cast<unsigned>(blocks), 256, 0, st>>>(o, d_o, delta, rows);
  return cudaGetLastError();
}

cudaError_t launch_prep(int head_dim, const __nv_bfloat16* o, const __nv_bfloat16* d_o, float* delta, int64_t rows,
                        const TileArgs& a, int64_t n_long, int short_entries, const ScoreArgs& sc, const FewList& few,
                        const FillArgs& q, const FillArgs& k, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((rows * (head_dim / 8) + 255) / 256, 148 * 16);
  const int n_delta = static_cast<int>(std::max<int64_t>(blocks, 1));
  const int64_t fills = std::min<int64_t>(std::max(q.n * q.bh, k.n * k.bh), 148 * 16);
  const PrepArgs p{o,      d_o,     delta,   rows,        n_long,      short_entries, n_delta, a.sched, q, k,
                   a.work, a.pages, a.masks, a.own_slots, a.col_slots, a.heads,       a.order, few,     sc};
  const unsigned grid = static_cast<unsigned>(n_long + n_delta + fills);
  if (head_dim == 128)
    prep_kernel<128><<<grid, 256, 0, st>>>(p);
  else
    prep_kernel<64><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D, int SC>
static cudaError_t launch_dkdv_t(const TmaPages& tk, const TmaPages& tv, const TmaPages& tq,
                                 const TmaPages& tdo, const TileArgs& a, const ScoreArgs& sc, const float* lse,
                                 const float* delta, __nv_bfloat16* dk, __nv_bfloat16* dv, cudaStream_t st) {
  using C = DkvCfg<D>;
  constexpr int kSmem = C::kSmem + (SC != kScoreNone ? C::kScoreBytes : 0);
  cudaError_t e = cudaFuncSetAttribute(dkdv_kernel<D, SC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess || a.n_work == 0) return e;
  // one persistent CTA per SM (at most one item each when there are fewer items)
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && SC == kScoreNone) e = cudaMemsetAsync(a.sched, 0, sizeof(int), st);  // else launch_prep's
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(a.n_work, std::max(sms, 1));
  dkdv_kernel<D, SC><<<static_cast<unsigned>(grid), BwdWarps<SC != kScoreNone>::kThreads, kSmem, st>>>(
      tk, tv, tq, tdo, a.work, a.n_work, a.sched, a.pages, a.masks, lse, delta, dk, dv, a.own_slots, a.col_slots,
      a.scale * kLog2e, a.scale, a.heads, a.kv_heads, a.kv_group, a.col_heads, a.err, sc, a.order);
  return cudaGetLastError();
}

template <int D, int SC, bool DELTA>
static cudaError_t launch_dq_t(const __nv_bfloat16* q, const TmaPages& tdo, const TmaPages& tk,
                               const TmaPages& tv, const TileArgs& a, const ScoreArgs& sc, const float* lse,
                               const float* delta, __nv_bfloat16* dq, int64_t n_items, int short_entries,
                               float* out_delta, cudaStream_t st) {
  using C = DqCfg<D>;
  constexpr int kSmem = C::kSmem + (SC != kScoreNone ? C::kScoreBytes : 0);
  cudaError_t e = cudaFuncSetAttribute(dq_kernel<D, SC, DELTA>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess || n_items == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_items));
  cfg.blockDim = dim3(BwdWarps<SC != kScoreNone>::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute beside = {};
  beside.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  beside.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &beside;
  cfg.numAttrs = a.beside ? 1 : 0;
  // short items are the last ones of the order
  const int32_t* order = DELTA && a.order ? a.order + (a.n_work - n_items) : a.order;
  return cudaLaunchKernelEx(&cfg, dq_kernel<D, SC, DELTA>, q, tdo, tk, tv, a.work, a.pages, a.masks, lse, delta, dq,
                            a.own_slots, a.scale * kLog2e, a.scale, a.heads, a.kv_group, a.err, sc, a.col_slots,
                            order, short_entries, out_delta);
}

// Calls `go` with the head size and the form of the scores as constants.
template <typename F>
static cudaError_t by_form(int head_dim, const ScoreArgs* sc, const F& go) {
  const int form = !sc ? kScoreNone : sc->cap > 0.f ? kScoreCap : kScoreMask;
  const auto pick = [&](auto d) {
    return form == kScoreNone   ? go(d, std::integral_constant<int, kScoreNone>{})
           : form == kScoreMask ? go(d, std::integral_constant<int, kScoreMask>{})
                                : go(d, std::integral_constant<int, kScoreCap>{});
  };
  return head_dim == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
}

cudaError_t launch_dkdv(int head_dim, const TmaPages& tk, const TmaPages& tv, const TmaPages& tq, const TmaPages& tdo,
                        const TileArgs& a, const ScoreArgs* sc, const float* lse, const float* delta,
                        __nv_bfloat16* dk, __nv_bfloat16* dv, cudaStream_t st) {
  const auto go = [&](auto d, auto form) {
    return launch_dkdv_t<decltype(d)::value, decltype(form)::value>(tk, tv, tq, tdo, a, sc ? *sc : ScoreArgs(), lse,
                                                                    delta, dk, dv, st);
  };
  return by_form(head_dim, sc, go);
}

cudaError_t launch_dq(int head_dim, const __nv_bfloat16* q, const TmaPages& tdo, const TmaPages& tk,
                      const TmaPages& tv, const TileArgs& a, const ScoreArgs* sc, const float* lse,
                      const float* delta, __nv_bfloat16* dq, cudaStream_t st) {
  const auto go = [&](auto d, auto form) {
    return launch_dq_t<decltype(d)::value, decltype(form)::value, false>(q, tdo, tk, tv, a, sc ? *sc : ScoreArgs(), lse,
                                                                         delta, dq, a.n_work, 0, nullptr, st);
  };
  return by_form(head_dim, sc, go);
}

cudaError_t launch_delta_exact(int head_dim, const __nv_bfloat16* q, const TmaPages& tdo, const TmaPages& tk,
                               const TmaPages& tv, const TileArgs& a, const ScoreArgs* sc, int64_t n_short,
                               int short_entries, const float* lse, float* delta, cudaStream_t st) {
  const auto go = [&](auto d, auto form) {
    constexpr int kForm = decltype(form)::value == kScoreNone ? kScoreMask : decltype(form)::value;  // always scored
    return launch_dq_t<decltype(d)::value, kForm, true>(q, tdo, tk, tv, a, *sc, lse, nullptr, nullptr,
                                                        a.order ? n_short : a.n_work, short_entries, delta, st);
  };
  return by_form(head_dim, sc, go);
}

cudaError_t launch_few_keys(int head_dim, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                            const __nv_bfloat16* d_o, const TileArgs& a, int64_t n_long, const ScoreArgs& sc,
                            const FewList& few, const float* lse, float* delta, cudaStream_t st) {
  if (n_long == 0) return cudaSuccess;
  const FewArgs f{q,       k,   v,           d_o,         lse,     delta,      a.work,  a.pages,
                  a.masks, few, a.own_slots, a.col_slots, a.heads, a.kv_group, a.scale, sc};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(8 * n_long, 148 * 3)));
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = st;
  cudaLaunchAttribute behind = {};
  behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &behind;
  cfg.numAttrs = a.beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, head_dim == 128 ? few_keys_kernel<128> : few_keys_kernel<64>, f);
}

}  // namespace spattn
