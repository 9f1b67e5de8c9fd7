// Attention of each sequence's new tokens over a paged K/V cache, from one
// token per sequence to long chunks, and the join of its split rows.
//
//   z = c tanh(x / c) - slope (p_q - p_k),  x = scale q.k,  allowed iff p_k <= p_q;
//   O = sum_k exp(z - LSE) v_k.
// Token i of a sequence with n new tokens and a cache of L slots (the new ones
// included) stands at position L - n + i.
//
// A CTA owns one tile of a sequence and a K/V head: 128 rows, the (token, query
// head) pairs of that head's group, token by token, so that a cached row is
// read once for all heads that share it.  The rest is the tile form of the
// plan's forward: 64 keys a step gathered by TMA, S = Q K^T and O += P V on
// tcgen05 with S double-buffered in TMEM, one or two threads per row, two CTAs
// per SM.  A page of the cache is a run of 16-slot pages; a run of consecutive
// ones takes one request per 64 rows, whole rows at a time (CachePages).  The
// TMA engine's time goes by requests: with one per 64-column chunk, 64 sequences in
// pages of 16 slots took 328 us, not 270.
//
// Bound: with few rows per tile the cache's bytes (one step moves 32 KB at
// head_dim 128 for 0.27 us of tensor work on an SM that gets 44 GB/s: memory
// sets the pace), with full tiles the softmax and the tensor core as in the
// plan's forward.  Long caches with few tiles are split along the keys into
// ranges of `chunk` keys; split rows go to a workspace in fp32 with their
// reference and sum, and paged_join_kernel adds them.
//
// Measured (head_dim 128, bounds equal to the lengths): 64 decoding sequences of 500 ..
// 9000 keys, 32 heads over 8, in 254 us of a long run (5.2 TB/s; 230 to 241 in short
// ones, before the board's power limit takes clocks); 2048 tokens over 131072 keys,
// 16 heads over 4, in 2450 us (0.9 PFLOP/s; 2185 in short runs); 777 keys of one sequence
// in 17 us, of which the launches and the host are most.  Ranges are sized from the
// bounds: with max_kv = 131072 the 64 sequences take 371 us (short runs), and one token
// over 8000 keys 41, not 20.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "kernels.cuh"
#include "score.cuh"
#include "spattn.h"

namespace spattn {
namespace {

using namespace dev;

constexpr int kStepKeys = 64;
constexpr int kStep16 = kStepKeys / 16;
constexpr float kRescale = 8.0f;  // rescale O when the running maximum grows by more than 2^8, as in the plan's forward

// FORM: kScoreMask (no cap) and kScoreCap run with a running maximum, one thread
// per row; kScoreFixed (a cap within kCapFixedMax) has a fixed reference and two
// threads per row (score.cuh).  Without a cap two threads and the plan's forward's
// passes for extreme rows were slower here, where no column lines are compared:
// 2420 us, not 2288, for 2048 tokens over 131072 keys.
// SMALL: tiles of at most 32 rows (decoding).  Memory sets the pace there, and in
// a long run the board's power: products of 128 rows, four of them live and the others
// whatever stood in shared memory, throttled the clocks to 1.57 GHz (64 sequences:
// 235 us in a short run, 280 in one of a second).  So the products have 64 rows, and
// most of the dead ones are zeros, which cost little (241 and 255 us).  Q takes 4 KB per
// chunk of 64 columns and 4 KB of zeros behind the last: rows 32 .. 63 of a chunk are what
// follows it, which for the first of two (head_dim 128) is the second's rows, live ones
// among them.  Products of those rows are never read.  The K and V rings are a stage deeper.
// Row r of an M = 64 product is TMEM lane r % 16 + 32 (r / 16).
template <int D, int FORM, bool SMALL>
struct PagedCfg {
  static constexpr int kNch = D / 64;
  static constexpr int kQChunk = SMALL ? 32 * 128 : kChunkBytes;
  static constexpr int kM = SMALL ? 64 : 128;  // rows of a product
  static constexpr int kWarpRows = kM / 4;
  static constexpr int kTile = kNch * kQChunk + (SMALL ? kQChunk : 0);
  static constexpr int kStage = kNch * kStepKeys * 128;
  static constexpr int kGroup = kNch * 1024;  // 8 rows of a stage
  static constexpr int kKStages = D == 128 ? (SMALL ? 3 : 2) : (SMALL ? 6 : 4);
  static constexpr int kVStages = kKStages;
  static constexpr int kRowThreads = FORM == kScoreFixed ? 256 : 128;
  static constexpr int kThreads = 64 + kRowThreads;
  static constexpr int kRamp = 384;   // barriers, TMEM slot and abort flag, then the ramp of a step's columns
  static constexpr int kBars = kRamp + kStepKeys * 4;
  static constexpr int kPairs = FORM == kScoreFixed ? 4 * 128 * 4 + 4 * 8 : 0;  // sums and barriers of the row pairs
  static constexpr int kSmem = kTile + (kKStages + kVStages) * kStage + 1024 + kBars + kPairs;
  static_assert((7 + 2 * (kKStages + kVStages) + 1) * 8 + 8 <= kRamp, "barriers end before the ramp");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct PagedArgs {
  const __nv_bfloat16* q;
  int64_t q_token, q_head;  // strides
  int64_t tokens;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* q_start;
  const int32_t* kv_len;
  __nv_bfloat16* o;
  float* lse;
  const float* slopes;
  float* part;  // [tile][split][tile_rows][D], then (reference, sum, divisor, 0) in the same order
  int64_t n_pages;
  int heads, kv_heads, group, page16;  // page16: 16-slot pages per page
  int max_q, max_kv, q_tiles, tile_rows, splits, chunk;
  int sms;
  float scale, cap;
  CapArgs c;
  int* err;
};

// One sequence's lengths, checked against the call's bounds.
struct Seq {
  int t0, nq, kv;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const PagedArgs& a, int s) {
  Seq q;
  q.t0 = __ldg(a.q_start + s);
  const int t1 = __ldg(a.q_start + s + 1);
  q.kv = __ldg(a.kv_len + s);
  q.ok = q.t0 >= 0 && t1 >= q.t0 && t1 <= a.tokens && t1 - q.t0 <= a.max_q && q.kv >= t1 - q.t0 && q.kv <= a.max_kv &&
         static_cast<int64_t>(q.kv) <= a.table_stride * a.page16 * 16;
  q.nq = q.ok ? t1 - q.t0 : 0;
  return q;
}

// Keys that tile `qt` of a sequence reaches (up to its last token).
__device__ __forceinline__ int tile_keys(const PagedArgs& a, const Seq& s, int qt) {
  const int last = min(s.nq - 1, (qt * kRows + kRows - 1) / a.group);
  return s.kv - s.nq + last + 1;
}

// Scores that a row does not see (columns from `vis` on) to zero before the cap: slots
// behind the cache's end and columns of an earlier step may hold anything.
__device__ __forceinline__ void clear_hidden(uint32_t (&s)[32], bool live, int vis) {
  if (__builtin_expect(live && vis < 32, 0)) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= vis) s[i] = 0u;
  }
}

// Load n 16-slot pages (lane j: page pid of step page j) into a stage, one box per
// run of consecutive pages and power of two.  All 32 lanes call this.
template <int NCH>
__device__ __forceinline__ void load_cache_runs(uint8_t* dst, const CachePages& maps, int pid, int n, int head,
                                                uint64_t* bar) {
  const int lane = lane_id();
  const int nxt = __shfl_down_sync(0xffffffffu, pid, 1);
  const unsigned cont = __ballot_sync(0xffffffffu, lane + 1 < n && nxt == pid + 1);  // bit j: page j + 1 follows page j
  if (lane >= n || (lane > 0 && ((cont >> (lane - 1)) & 1u))) return;
  int rem = __ffs(~(cont >> lane)), j = 0;  // the run: at most kStep16 pages; j of them are on their way
  auto box = [&](const CUtensorMap* m, int pages) {
    tma_load_5d(dst + (lane + j) * NCH * 2048, m, 0, 0, 0, 2 * (pid + j), head, bar);
    j += pages;
    rem -= pages;
  };
  if (rem >= 4) box(&maps.m64, 4);
  if (rem >= 2) box(&maps.m32, 2);
  if (rem == 1) box(&maps.m16, 1);
}

template <int D, int FORM, bool SMALL>
__global__ void __launch_bounds__(PagedCfg<D, FORM, SMALL>::kThreads, 2)
    paged_kernel(const __grid_constant__ CachePages tm_k, const __grid_constant__ CachePages tm_v, const PagedArgs a) {
  using C = PagedCfg<D, FORM, SMALL>;
  constexpr bool kFixed = FORM == kScoreFixed, kCap = kFixed || FORM == kScoreCap;
  constexpr int KS = C::kKStages, VS = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kTile;
  uint8_t* sV = sK + KS * C::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + VS * C::kStage);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + VS;
  uint64_t* s_full = v_empty + VS;  // [2]
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* o_done = p_full + 2;
  uint64_t* drain = o_done + 1;
  uint64_t* o_last = drain + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(o_last + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  const Abort ab{abort_flag, a.err};
  float* ramp = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + C::kRamp);  // 0, 1, .. 63
  float* xrow = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + C::kBars);
  uint64_t* pair_bar = reinterpret_cast<uint64_t*>(xrow + 4 * 128);  // [4]

  // the join may be launched while this kernel runs; it waits for its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // tiles and then K/V heads vary fastest: CTAs that run together read the same
  // range, and the heads of its pages side by side
  const int split = blockIdx.x / (a.q_tiles * a.kv_heads), tile_hk = blockIdx.x - split * a.q_tiles * a.kv_heads;
  const int hk = tile_hk / a.q_tiles, qt = tile_hk - hk * a.q_tiles, sq = blockIdx.y;
  const Seq seq = load_seq(a, sq);
  if (!seq.ok && threadIdx.x == 0 && blockIdx.x == 0) atomicCAS(a.err, 0, kErrBadWork);
  const int rows = min(kRows, seq.nq * a.group - qt * kRows);
  if (rows <= 0) return;  // uniform over the CTA
  const int keys = tile_keys(a, seq, qt);
  const int k0 = split * a.chunk, k1 = min(keys, k0 + a.chunk);
  if (k0 >= k1) return;
  const bool whole = keys <= a.chunk;  // the only split of this tile
  const int n16 = (k1 - k0 + 15) / 16;
  const int n_steps = (n16 + kStep16 - 1) / kStep16;
  const int row_warps = (rows + C::kWarpRows - 1) / C::kWarpRows;
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    mbar_init(q_full, SMALL ? C::kRowThreads : 32 * row_warps);  // group 0 of the row threads loads Q
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], (kFixed ? 64 : 32) * row_warps);
    }
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    mbar_init(o_last, 1);
    if constexpr (kFixed)
      for (int i = 0; i < 4; ++i) mbar_init(&pair_bar[i], 64);
    fence_barrier_init();
  }
  if (threadIdx.x < kStepKeys) ramp[threadIdx.x] = static_cast<float>(threadIdx.x);
  if (warp == 1) tmem_alloc(tslot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tO = tmem + 128;

  if constexpr (SMALL) {
    // every row thread: zeros wherever Q has no live row
    if (warp >= 2) {
      for (int i = threadIdx.x - 64; i < C::kTile / 16; i += C::kRowThreads)
        if (((i >> 3) & 31) >= rows || i >= C::kNch * C::kQChunk / 16)
          reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      if (warp >= 6 || (warp & 3) >= row_warps) mbar_arrive(q_full);  // (the others when they have loaded their rows)
    }
  }
  if (warp == 0) {
    // ---------------- producer: lane j < 4 owns 16-slot page j of a step ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tm_k.m64);
      tma_prefetch_desc(&tm_v.m64);
    }
    __syncwarp();
    const int32_t* table = a.table + static_cast<int64_t>(sq) * a.table_stride;
    const int first16 = k0 / 16;
    // 16-slot page of the pool; an entry outside the pool is reported and read as page 0
    auto page_of = [&](int st) {
      const int j = st * kStep16 + lane;
      if (lane >= kStep16 || j >= n16) return 0;
      const int i = (first16 + j) / a.page16;
      int p = __ldg(table + i);
      if (p < 0 || p >= a.n_pages) {
        atomicCAS(a.err, 0, kErrBadWork);
        p = 0;
      }
      return p * a.page16 + (first16 + j) - i * a.page16;
    };
    int pid_next = page_of(0);
    int k_issued = 0, v_issued = 0;
    for (int st = 0; st < n_steps; ++st) {
      const int n = min(kStep16, n16 - st * kStep16);
      const int pid = pid_next;
      if (st + 1 < n_steps) pid_next = page_of(st + 1);
      const int ks = st % KS, vs = st % VS;
      if (st >= KS && !__all_sync(0xffffffffu, mbar_wait(&k_empty[ks], ((st / KS) - 1) & 1, ab))) break;
      if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], n * C::kNch * 2048);
      __syncwarp();
      load_cache_runs<C::kNch>(sK + ks * C::kStage, tm_k, pid, n, hk, &k_full[ks]);
      k_issued = st + 1;
      if (st >= VS && !__all_sync(0xffffffffu, mbar_wait(&v_empty[vs], ((st / VS) - 1) & 1, ab))) break;
      if (lane == 0) mbar_arrive_expect_tx(&v_full[vs], n * C::kNch * 2048);
      __syncwarp();
      load_cache_runs<C::kNch>(sV + vs * C::kStage, tm_v, pid, n, hk, &v_full[vs]);
      v_issued = st + 1;
    }
    // no copy may still be landing in shared memory when the CTA exits
    if (lane == 0) {
      for (int st = max(0, k_issued - KS); st < k_issued; ++st) mbar_wait_drain(&k_full[st % KS], (st / KS) & 1);
      for (int st = max(0, v_issued - VS); st < v_issued; ++st) mbar_wait_drain(&v_full[st % VS], (st / VS) & 1);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const uint64_t dq0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, C::kGroup);
    const uint64_t dv0 = sdesc_sw128(smem_u32(sV), 1024, C::kGroup);
    const uint32_t idesc_pv = idesc_bf16(C::kM, D, false, true);
    bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, ab));
    tc_fence_after();
    auto issue_pv = [&](int st) -> bool {
      const int b = st & 1, vs = st % VS;
      const bool w = mbar_wait(&p_full[b], (st >> 1) & 1, ab) && mbar_wait(&v_full[vs], (st / VS) & 1, ab);
      if (!__all_sync(0xffffffffu, w)) return false;
      const int n = min(kStep16, n16 - st * kStep16);
      // slots behind the range may never have been written: their V rows, which
      // meet weights of zero, become zero (a NaN there would not vanish)
      const int live = k1 - k0 - st * kStepKeys;
      if (live < 16 * n) {
        for (int i = lane; i < (16 * n - live) * 8 * C::kNch; i += 32) {
          const int r = live + i / (8 * C::kNch), c = i % (8 * C::kNch);
          *reinterpret_cast<uint4*>(sV + vs * C::kStage + (r >> 3) * C::kGroup + (c >> 3) * 1024 + (r & 7) * 128 +
                                    (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      const uint64_t dv = sdesc_add(dv0, vs * C::kStage);
#pragma unroll
      for (int j = 0; j < kStep16; ++j)
        if (j < n)
          umma_ts_w(tO, tmem + 64 * b + 8 * j + (kFixed && j >= 2 ? 16 : 0), sdesc_add(dv, j * 2 * C::kGroup), idesc_pv,
                    (st > 0 || j > 0) ? 1u : 0u);
      umma_commit_w(&v_empty[vs]);
      umma_commit_w(o_done);
      return true;
    };
    for (int st = 0; ok && st < n_steps; ++st) {
      const int ks = st % KS, b = st & 1;
      // buffer b holds P(st-2) until PV(st-2) has finished
      const bool w = mbar_wait(&k_full[ks], (st / KS) & 1, ab) && (st < 2 || mbar_wait(o_done, (st - 2) & 1, ab));
      if (!__all_sync(0xffffffffu, w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int n = min(kStep16, n16 - st * kStep16);
      const uint64_t dk = sdesc_add(dk0, ks * C::kStage);
      const uint32_t idesc_s = idesc_bf16(C::kM, 16 * n, false, false);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_ss_w(tmem + 64 * b, sdesc_add(dq0, (kk >> 2) * C::kQChunk + (kk & 3) * 32),
                  sdesc_add(dk, (kk >> 2) * 1024 + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
      umma_commit_w(&s_full[b]);
      umma_commit_w(&k_empty[ks]);
      if (st >= 1 && !issue_pv(st - 1)) ok = false;
    }
    if (ok && issue_pv(n_steps - 1)) umma_commit_w(o_last);
    umma_commit_w(drain);
    mbar_wait_drain(drain, 0);
  } else if ((warp & 3) < row_warps) {
    // ---------------- softmax + epilogue (row warps without rows stay out) ----------------
    const int grp = kFixed ? (warp - 2) >> 2 : 0;  // fixed form: column half of a step, and of O
    const int q4 = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const int row = C::kWarpRows * q4 + lane;
    const bool live = lane < C::kWarpRows && row < rows;  // the others are zeros, attend nothing and are not stored
    const int rr = qt * kRows + (live ? row : 0);
    const int tok = rr / a.group, head = hk * a.group + rr % a.group;
    const int last = live ? seq.kv - seq.nq + tok : -1;  // this row's position
    if (grp == 0) {
      // the row's 16-byte pieces go to their places in the 128-byte swizzle
      const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(seq.t0 + tok) * a.q_token +
                                                        static_cast<int64_t>(head) * a.q_head);
      uint4 v[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        if (live || !SMALL)
          *reinterpret_cast<uint4*>(sQ + (i >> 3) * C::kQChunk + row * 128 + (((i & 7) ^ (row & 7)) << 4)) = v[i];
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    }
    const float sl2 = a.scale * kLog2e;
    const float slope2 = a.slopes ? __ldg(a.slopes + head) * kLog2e : 0.f;
    bool ok = true;
    // results of the loops below: reference of the weights (log2), their sum, divisor of O
    float ref = -INFINITY, l_true = 0.f, l = 0.f;
    if constexpr (kFixed) {
      // The cap bounds the capped scores, and the bias is largest at the range's
      // nearest key (farthest for a negative slope), a distance known here: with it
      // as reference no weight passes 2^cap2, and that key's is at least 2^-cap2.
      const int d_ref = slope2 >= 0.f ? max(0, last - (k1 - 1)) : last - k0;
      ref = a.slopes ? -slope2 * static_cast<float>(d_ref) : 0.f;
      SoftRow r;
      for (int st = 0; st < n_steps; ++st) {
        const int b = st & 1;
        const bool active = 2 * grp < n16 - st * kStep16;
        const int base = k0 + st * kStepKeys + 32 * grp;  // position of this thread's first column
        const int vis = last - base + 1;                   // its columns 0 .. vis - 1 are allowed
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[b], (st >> 1) & 1, ab));
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_addr = tmem + 64 * b + lane_off + 32 * grp;
        if (active) {
          uint32_t x[32];
          tmem_ld32(s_addr, x);
          tmem_wait_ld();
          clear_hidden(x, live, vis);
          cap_scores<false>(x, x, a.c, live);
          if (a.slopes) {
            // - slope (distance - d_ref) = slope (column - (last - base - d_ref))
            const float b0 = -slope2 * static_cast<float>(last - base - d_ref);
            const uint64_t b2 = f2_pack(b0, b0), s2 = f2_pack(slope2, slope2);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 c = *reinterpret_cast<const float4*>(ramp + i);
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                float x0, x1;
                f2_unpack(f2_add(f2_pack(__uint_as_float(x[i + j]), __uint_as_float(x[i + j + 1])),
                                 f2_fma(j ? f2_pack(c.z, c.w) : f2_pack(c.x, c.y), s2, b2)),
                          x0, x1);
                x[i + j] = __float_as_uint(x0);
                x[i + j + 1] = __float_as_uint(x1);
              }
            }
          }
          // a step with fewer than 64 keys ends the range, so vis stays below them there
          if (__builtin_expect(vis < 32, 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= vis) x[i] = 0xFF800000u;  // -inf
          }
          soft_weights(x, 1.0f, 0.f, r, s_addr);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(o_last, 0, ab));
      tc_fence_after();
      ok = ok && soft_total(r, xrow + 32 * q4 + lane, grp, &pair_bar[q4], 0, ab, l, l_true);
    } else {
      const float mul = kCap ? 1.0f : sl2;  // after the cap the scores are in log2 units
      const uint64_t mul2 = f2_pack(mul, mul);
      const float slope = slope2 / mul;
      for (int st = 0; st < n_steps; ++st) {
        const int b = st & 1;
        const int N = 16 * min(kStep16, n16 - st * kStep16);
        const int base = k0 + st * kStepKeys;  // position of column 0
        const int vis = last - base + 1;       // columns 0 .. vis - 1 are allowed
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[b], (st >> 1) & 1, ab));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[2][32];
#pragma unroll
        for (int pc = 0; pc < 2; ++pc)
          if (pc * 32 < N) tmem_ld32(tmem + 64 * b + lane_off + pc * 32, sr[pc]);
        tmem_wait_ld();
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
          if (pc * 32 < N) {
            if constexpr (kCap) {
              clear_hidden(sr[pc], live, vis - 32 * pc);
              cap_scores<false>(sr[pc], sr[pc], a.c, live);
            }
            if (a.slopes) {
              const float b0 = -slope * static_cast<float>(last - base);
              const uint64_t b2 = f2_pack(b0, b0), s2 = f2_pack(slope, slope);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 c = *reinterpret_cast<const float4*>(ramp + 32 * pc + i);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                  float x0, x1;
                  f2_unpack(f2_add(f2_pack(__uint_as_float(sr[pc][i + j]), __uint_as_float(sr[pc][i + j + 1])),
                                   f2_fma(j ? f2_pack(c.z, c.w) : f2_pack(c.x, c.y), s2, b2)),
                            x0, x1);
                  sr[pc][i + j] = __float_as_uint(x0);
                  sr[pc][i + j + 1] = __float_as_uint(x1);
                }
              }
            }
            // a step whose N is not a multiple of 32 ends the range, so vis <= N there
            if (vis < pc * 32 + 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (pc * 32 + i >= vis) sr[pc][i] = 0xFF800000u;  // -inf
            }
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              mx[0] = fmax3(mx[0], __uint_as_float(sr[pc][i]), __uint_as_float(sr[pc][i + 1]));
              mx[1] = fmax3(mx[1], __uint_as_float(sr[pc][i + 2]), __uint_as_float(sr[pc][i + 3]));
              mx[2] = fmax3(mx[2], __uint_as_float(sr[pc][i + 4]), __uint_as_float(sr[pc][i + 5]));
              mx[3] = fmax3(mx[3], __uint_as_float(sr[pc][i + 6]), __uint_as_float(sr[pc][i + 7]));
            }
          }
        }
        const float mx2 = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * mul;
        const bool resc = mx2 > ref + kRescale;
        const float m_new = resc ? mx2 : ref;
        const float alpha = resc ? ex2(ref - m_new) : 1.0f;
        l *= alpha;
        ref = m_new;
        const float neg_mu = (ref == -INFINITY) ? 0.f : -ref;
        const uint64_t nmu2 = f2_pack(neg_mu, neg_mu);
        uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
          if (pc * 32 < N) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[pc][2 * i]), __uint_as_float(sr[pc][2 * i + 1])), mul2, nmu2),
                        x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              ls2[i & 1] = f2_add(ls2[i & 1], f2_pack(p0, p1));
              pk[i] = pack_bf16(p0, p1);
            }
            tmem_st16(tmem + 64 * b + lane_off + pc * 16, pk);
          }
        }
        {
          float a0, a1, b0, b1;
          f2_unpack(ls2[0], a0, a1);
          f2_unpack(ls2[1], b0, b1);
          l += (a0 + a1) + (b0 + b1);
        }
        if (st > 0 && __any_sync(0xffffffffu, resc)) {
          // O must hold the steps before this one; o_done has completed st - 1 or st
          // phases here (S(st) was issued after PV(st-2), PV(st) waits for this arrival)
          ok = __all_sync(0xffffffffu, mbar_wait(o_done, (st - 1) & 1, ab));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int pc = 0; pc < D / 32; ++pc) {
            uint32_t r[32];
            tmem_ld32(tO + lane_off + pc * 32, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st32(tO + lane_off + pc * 32, r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(o_last, 0, ab));
      tc_fence_after();
      l_true = l;
    }
    if (ok) {
      const int64_t out = static_cast<int64_t>(seq.t0 + tok) * a.heads + head;
      const int64_t tile = (static_cast<int64_t>(sq) * a.kv_heads + hk) * a.q_tiles + qt;
      const int64_t n_part = static_cast<int64_t>(gridDim.y) * a.kv_heads * a.q_tiles * a.splits * a.tile_rows;
      const int64_t part = (tile * a.splits + split) * a.tile_rows + row;
      const bool empty = l == 0.f;  // (a NaN score is no empty row: its O and LSE are NaN)
      const float inv = empty ? 0.f : 1.0f / l;
      constexpr int kOut = kFixed ? D / 2 : D;  // columns of O that this thread writes
      const int col = grp * kOut;
#pragma unroll
      for (int pc = 0; pc < kOut / 32; ++pc) {
        uint32_t r[32];
        tmem_ld32(tO + lane_off + col + pc * 32, r);
        tmem_wait_ld();
        if (live && whole) {
          store_row32(a.o + out * D + col + pc * 32, r, inv, empty);
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.part + part * D + col + pc * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
      }
      if (live && grp == 0) {
        if (whole) {
          if (a.lse) a.lse[out] = empty ? -INFINITY : (ref + lg2(l_true)) * kLn2;
        } else {
          *reinterpret_cast<float4*>(a.part + n_part * D + 4 * part) = make_float4(empty ? -INFINITY : ref, l_true, l, 0.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Join of split rows, W warps per (token, head): O = sum_s 2^(m_s - M) O_s /
// sum_s 2^(m_s - M) l_s (m_s, l_s: a split's reference and divisor; LSE has the sum
// t_s of its unrounded weights).  M is the largest m_s + log2 t_s, not the largest
// reference: a sum relative to a fixed reference may be 2^80 away from 1, so the
// references alone do not tell which split counts.  No 2^(m_s - M) t_s passes 1.
//
// Bound: the latency of the partial rows' loads, four in flight per warp.  Where one
// warp per row would leave the SMs short of warps, a block's warps share a row (one
// token of 16 heads over 8000 keys, 63 splits: 14.4 us for the call, not 26.7; 15
// splits: 12.3, not 16.4).  With many rows that costs more than it gives (2048 tokens
// over 131072 keys: 2275 us, not 2193).
constexpr int kJoinWarps = 8;
constexpr int kJoinShare = 4;        // splits from which warps may share a row,
constexpr int kJoinRowsPerSm = 8;    // up to as many rows per SM

template <int D, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const PagedArgs a, int n_seqs) {
  static_assert(W == 1 || W == kJoinWarps, "a warp's row or a block's");
  __shared__ float4 part_o[W > 1 ? W : 1][D / 4];
  __shared__ float2 part_l[W > 1 ? W : 1];
  const int lane = threadIdx.x & 31, sub = W > 1 ? threadIdx.x >> 5 : 0;
  const int64_t item = W > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  // the partial rows are there when the kernel before has ended; block 0 waits in any
  // case, so that this kernel does not end (and let the stream go on) before that one
  auto wait_parts = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (blockIdx.x == 0) wait_parts();
  if (item >= a.tokens * a.heads) return;
  const int at = static_cast<int>(item / a.heads), head = static_cast<int>(item % a.heads);
  // the sequence of row `at`: the last one that starts at or before it, 32 ways per pass
  int sq = 0;
  for (int span = n_seqs; span > 1;) {
    const int step = (span + 31) / 32, i = sq + lane * step;
    const bool before = lane * step < span && __ldg(a.q_start + i) <= at;
    const int last = max(0, 31 - __clz(__ballot_sync(0xffffffffu, before)));
    span = min(step, span - last * step);
    sq += last * step;
  }
  const Seq seq = load_seq(a, sq);
  const int tok = at - seq.t0;
  if (tok < 0 || tok >= seq.nq) return;
  const int hk = head / a.group, rr = tok * a.group + head % a.group;
  const int qt = rr / kRows, row = rr % kRows;
  const int n = (tile_keys(a, seq, qt) + a.chunk - 1) / a.chunk;
  if (n <= 1) return;  // written by the tile itself
  wait_parts();
  const int64_t tile = (static_cast<int64_t>(sq) * a.kv_heads + hk) * a.q_tiles + qt;
  const int64_t n_part = static_cast<int64_t>(n_seqs) * a.kv_heads * a.q_tiles * a.splits * a.tile_rows;
  const int64_t part0 = tile * a.splits * a.tile_rows + row;
  const float4* ml = reinterpret_cast<const float4*>(a.part + n_part * D);
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) {
    const float4 x = ml[part0 + static_cast<int64_t>(s) * a.tile_rows];
    if (x.z != 0.f) m = fmaxf(m, x.x + lg2(x.y));  // (a NaN drops out here and comes back with its weight below)
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  constexpr int E = D / 32;  // elements per lane
  float acc[E] = {}, l = 0.f, l_true = 0.f;
#pragma unroll 4
  for (int s = sub; s < n; s += W) {
    const int64_t p = part0 + static_cast<int64_t>(s) * a.tile_rows;
    const float4 x = ml[p];
    const float w = x.z == 0.f ? 0.f : ex2(x.x - m);
    l_true = fmaf(w, x.y, l_true);
    l = fmaf(w, x.z, l);
    const float* src = a.part + p * D + lane * E;
    if constexpr (E == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(w, v.x, acc[0]);
      acc[1] = fmaf(w, v.y, acc[1]);
      acc[2] = fmaf(w, v.z, acc[2]);
      acc[3] = fmaf(w, v.w, acc[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(w, v.x, acc[0]);
      acc[1] = fmaf(w, v.y, acc[1]);
    }
  }
  if constexpr (W > 1) {  // (a block's threads have the same row and come here together)
    float* mine = reinterpret_cast<float*>(part_o[sub]);
#pragma unroll
    for (int i = 0; i < E; ++i) mine[lane * E + i] = acc[i];
    if (lane == 0) part_l[sub] = make_float2(l, l_true);
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float* other = reinterpret_cast<const float*>(part_o[w]);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += other[lane * E + i];
      l += part_l[w].x;
      l_true += part_l[w].y;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int64_t out = static_cast<int64_t>(seq.t0 + tok) * a.heads + head;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + out * D + lane * E);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dst[i] = pack_bf16(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (a.lse && lane == 0) a.lse[out] = l == 0.f ? -INFINITY : (m + lg2(l_true)) * kLn2;
}

template <int D, int FORM, bool SMALL>
cudaError_t launch_paged_t(const CachePages& tk, const CachePages& tv, const PagedArgs& a, int n_seqs, cudaStream_t st) {
  using C = PagedCfg<D, FORM, SMALL>;
  cudaError_t e =
      cudaFuncSetAttribute(paged_kernel<D, FORM, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.q_tiles * a.kv_heads * a.splits), static_cast<unsigned>(n_seqs));
  paged_kernel<D, FORM, SMALL><<<grid, C::kThreads, C::kSmem, st>>>(tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  const bool share = a.splits >= kJoinShare && a.tokens * a.heads <= kJoinRowsPerSm * a.sms;
  const int64_t blocks = share ? a.tokens * a.heads : (a.tokens * a.heads + kJoinWarps - 1) / kJoinWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute behind = {};
  behind.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &behind;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, share ? paged_join_kernel<D, kJoinWarps> : paged_join_kernel<D, 1>, a, n_seqs);
}

template <int D, int FORM>
cudaError_t launch_paged_f(const CachePages& tk, const CachePages& tv, const PagedArgs& a, int n_seqs, cudaStream_t st) {
  return a.tile_rows <= 32 ? launch_paged_t<D, FORM, true>(tk, tv, a, n_seqs, st)
                           : launch_paged_t<D, FORM, false>(tk, tv, a, n_seqs, st);
}

template <int D>
cudaError_t launch_paged(const CachePages& tk, const CachePages& tv, const PagedArgs& a, int n_seqs, cudaStream_t st) {
  if (!(a.cap > 0.f)) return launch_paged_f<D, kScoreMask>(tk, tv, a, n_seqs, st);
  return a.c.cap2 <= kCapFixedMax ? launch_paged_f<D, kScoreFixed>(tk, tv, a, n_seqs, st)
                                  : launch_paged_f<D, kScoreCap>(tk, tv, a, n_seqs, st);
}

}  // namespace
}  // namespace spattn

using namespace spattn;

namespace {
struct Split {
  int q_tiles = 0, tile_rows = 0, splits = 0, chunk = 0;
};
}  // namespace

struct spattn_paged_s {
  spattn_paged_layout lay;
  Split one;  // the split of calls with one sequence
  int device = -1;
  int sms = 148;
  int* d_err = nullptr;
};

namespace {

// Split of a call over n sequences: q tiles per (sequence, K/V head), splits and
// their length in keys.  Two CTAs run on an SM.  A CTA costs its keys, about 320
// keys' time for its start and end and, with a full tile, about 550 for writing
// its rows in fp32 and reading them back.  One sequence fills whole rounds of CTAs, so
// the split count with the fewest rounds x cost wins.  Of several, the host knows
// only the bounds: with half of them as the mean length, ranges of about
// sqrt(work x overhead / slots) keys balance that overhead against the last
// CTA's tail.  1.5 times that measured best over both kinds of call: with factors
// 1, 1.5, 2 and 2.7, 64 decoding sequences of 500 .. 9000 keys took 243, 235, 230
// and 240 us, eight of 4000 .. 60000 keys 232, 201, 201 and 219, and five
// sequences of chunks up to 700 tokens 375, 384, 427 and 475.
Split choose_split(const spattn_paged_s* p, int64_t n_seqs) {
  if (n_seqs == 1 && p->one.splits) return p->one;
  const auto& L = p->lay;
  const int64_t group = L.heads / L.kv_heads;
  Split s;
  const int64_t rows = L.max_q * group;
  s.q_tiles = static_cast<int>((rows + 127) / 128);
  s.tile_rows = static_cast<int>(rows < 128 ? rows : 128);
  const int64_t tiles = n_seqs * L.kv_heads * s.q_tiles, slots = 2 * p->sms;
  const double overhead = 320 + 550.0 * s.tile_rows / 128;
  // at most sixteen rounds of CTAs, which bounds the workspace (320 MB of full tiles)
  const int64_t most = std::max<int64_t>(1, std::min({(L.max_kv + 127) / int64_t{128}, int64_t{1024}, 16 * slots / tiles}));
  int64_t n = 1;
  if (n_seqs == 1) {
    double best = -1;
    for (int64_t k = 1; k <= most; ++k) {
      const int64_t chunk = ((L.max_kv + k - 1) / k + 63) / 64 * 64;
      const double cost = static_cast<double>((tiles * k + slots - 1) / slots) * (chunk + (k > 1 ? overhead : 320));
      if (best < 0 || cost < best) {
        best = cost;
        n = k;
      }
    }
  } else {
    const double chunk = 1.5 * std::sqrt(0.5 * tiles * L.max_kv * overhead / slots);
    n = std::min<int64_t>(most, std::max<int64_t>(1, static_cast<int64_t>(L.max_kv / chunk + 0.5)));
  }
  s.chunk = static_cast<int>(((L.max_kv + n - 1) / n + 63) / 64 * 64);
  s.splits = (L.max_kv + s.chunk - 1) / s.chunk;
  return s;
}

int64_t split_bytes(const spattn_paged_s* p, const Split& s, int64_t n_seqs) {
  if (s.splits == 1) return 0;
  return n_seqs * p->lay.kv_heads * s.q_tiles * s.splits * s.tile_rows * (p->lay.head_dim + 4) * 4;
}

bool aligned(const void* p, uintptr_t al) { return p && reinterpret_cast<uintptr_t>(p) % al == 0; }

}  // namespace

extern "C" {

int spattn_paged_create(const spattn_paged_layout* L, spattn_paged_t* out) {
  if (!out) return SPATTN_ERR_INVALID_ARG;
  *out = nullptr;
  if (!L || L->heads < 1 || L->kv_heads < 1 || L->heads % L->kv_heads || L->page_slots < 16 || L->page_slots % 16 ||
      L->max_seqs < 1 || L->max_q < 1 || L->max_kv < 1 || !std::isfinite(L->scale) || L->scale < 0.f ||
      !std::isfinite(L->softcap) || L->softcap < 0.f)
    return SPATTN_ERR_INVALID_ARG;
  if ((L->head_dim != 64 && L->head_dim != 128) || L->heads > 32768 || L->max_seqs > 65535 || L->max_kv > (1 << 30) ||
      static_cast<int64_t>(L->max_q) * L->heads > (1 << 30) || L->page_slots > (1 << 20))
    return SPATTN_ERR_UNSUPPORTED;
  auto* p = new (std::nothrow) spattn_paged_s();
  if (!p) return SPATTN_ERR_OOM;
  p->lay = *L;
  if (p->lay.scale == 0.f) p->lay.scale = 1.0f / std::sqrt(static_cast<float>(L->head_dim));
  int n = 0;
  if (cudaGetDeviceCount(&n) == cudaSuccess && n > 0) {
    if (cudaGetDevice(&p->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess) {
      delete p;
      return SPATTN_ERR_CUDA;
    }
    if (cudaMalloc(&p->d_err, sizeof(int)) != cudaSuccess) {
      delete p;
      return SPATTN_ERR_OOM;
    }
    if (cudaMemset(p->d_err, 0, sizeof(int)) != cudaSuccess) {
      cudaFree(p->d_err);
      delete p;
      return SPATTN_ERR_CUDA;
    }
  } else {
    cudaGetLastError();  // no device: checks and workspace sizes only
  }
  p->one = choose_split(p, 1);
  *out = p;
  return SPATTN_OK;
}

void spattn_paged_destroy(spattn_paged_t p) {
  if (!p) return;
  if (p->d_err) cudaFree(p->d_err);
  delete p;
}

int spattn_paged_workspace(spattn_paged_t p, int64_t n_seqs, int64_t* bytes) {
  if (!p || !bytes || n_seqs < 0 || n_seqs > p->lay.max_seqs) return SPATTN_ERR_INVALID_ARG;
  *bytes = n_seqs ? split_bytes(p, choose_split(p, n_seqs), n_seqs) : 0;
  return SPATTN_OK;
}

int spattn_paged_fwd(spattn_paged_t p, const spattn_paged_call* c, void* stream) {
  if (!p || !c) return SPATTN_ERR_INVALID_ARG;
  const auto& L = p->lay;
  if (c->n_seqs < 0 || c->n_seqs > L.max_seqs || c->tokens < 0 || c->n_pages < 0 || c->table_stride < 0)
    return SPATTN_ERR_INVALID_ARG;
  if (c->n_seqs == 0 || c->tokens == 0) return SPATTN_OK;
  if (c->tokens > 0x7FFFFFFFll || c->tokens * L.heads > 0x7FFFFFFFll || c->n_pages > 0x7FFFFFFFll / L.page_slots || c->table_stride > 0x7FFFFFFFll)
    return SPATTN_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->table_stride < 1) return SPATTN_ERR_INVALID_ARG;
  if (!aligned(c->q, 16) || !aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->o, 16) ||
      !aligned(c->page_table, 4) || !aligned(c->q_start, 4) || !aligned(c->kv_len, 4) ||
      (c->lse && !aligned(c->lse, 4)) || (c->slopes && !aligned(c->slopes, 4)))
    return SPATTN_ERR_INVALID_ARG;
  // rows are read in 16-byte pieces and mapped with 16-byte strides
  for (int64_t s : {c->q_token_stride, c->q_head_stride, c->k_slot_stride, c->k_head_stride, c->v_slot_stride,
                    c->v_head_stride})
    if (s < 0 || s % 8) return SPATTN_ERR_INVALID_ARG;
  if (c->k_slot_stride < L.head_dim || c->v_slot_stride < L.head_dim ||
      (L.kv_heads > 1 && (c->k_head_stride < L.head_dim || c->v_head_stride < L.head_dim)))
    return SPATTN_ERR_INVALID_ARG;
  if (p->device < 0) return SPATTN_ERR_CUDA;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPATTN_ERR_CUDA;
  if (dev != p->device) return SPATTN_ERR_INVALID_ARG;
  const Split sp = choose_split(p, c->n_seqs);
  const int64_t need = split_bytes(p, sp, c->n_seqs);
  if (c->workspace_bytes < need || (need > 0 && !aligned(c->workspace, 16))) return SPATTN_ERR_INVALID_ARG;
  const int64_t slots = c->n_pages * L.page_slots;
  CachePages tk, tv;
  if (!make_cache_pages(&tk, c->k_cache, L.head_dim, slots, c->k_slot_stride, L.kv_heads, c->k_head_stride) ||
      !make_cache_pages(&tv, c->v_cache, L.head_dim, slots, c->v_slot_stride, L.kv_heads, c->v_head_stride))
    return SPATTN_ERR_CUDA;
  PagedArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(c->q);
  a.q_token = c->q_token_stride;
  a.q_head = c->q_head_stride;
  a.tokens = c->tokens;
  a.table = c->page_table;
  a.table_stride = c->table_stride;
  a.q_start = c->q_start;
  a.kv_len = c->kv_len;
  a.o = static_cast<__nv_bfloat16*>(c->o);
  a.lse = c->lse;
  a.slopes = c->slopes;
  a.part = static_cast<float*>(c->workspace);
  a.n_pages = c->n_pages;
  a.heads = L.heads;
  a.kv_heads = L.kv_heads;
  a.group = L.heads / L.kv_heads;
  a.page16 = L.page_slots / 16;
  a.max_q = L.max_q;
  a.max_kv = L.max_kv;
  a.q_tiles = sp.q_tiles;
  a.tile_rows = sp.tile_rows;
  a.splits = sp.splits;
  a.chunk = sp.chunk;
  a.sms = p->sms;
  a.scale = L.scale;
  a.cap = L.softcap;
  a.c = cap_args(L.softcap, L.scale);
  a.err = p->d_err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(c->n_seqs);
  const cudaError_t e = L.head_dim == 128 ? launch_paged<128>(tk, tv, a, n, s) : launch_paged<64>(tk, tv, a, n, s);
  return e == cudaSuccess ? SPATTN_OK : SPATTN_ERR_CUDA;
}

int spattn_paged_check(spattn_paged_t p, void* stream) {
  if (!p) return SPATTN_ERR_INVALID_ARG;
  if (p->device < 0) return SPATTN_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SPATTN_ERR_CUDA;
  int h = 0;
  if (cudaMemcpy(&h, p->d_err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SPATTN_ERR_CUDA;
  if (h == 0) return SPATTN_OK;
  if (cudaMemset(p->d_err, 0, sizeof(int)) != cudaSuccess) return SPATTN_ERR_CUDA;
  return h == 1 ? SPATTN_ERR_TIMEOUT : SPATTN_ERR_DEVICE;
}

}  // extern "C"
