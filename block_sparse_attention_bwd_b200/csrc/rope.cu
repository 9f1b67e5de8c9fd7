// Rotary positions of Q and K, forward and backward.
//
// Pair p of a row (elements 2p, 2p + 1 when interleaved, p and p + rot/2
// otherwise) is turned by the angle t = pos[axis(p)] * freq[p] and scaled:
//   a' = m (a cos t - b sin t),   b' = m (a sin t + b cos t);
// the gradient is the same with -t.  Elements from rot on are copied.
//
// The angle is formed in fp64 as a fraction of a turn (pos * freq / 2 pi,
// less its nearest integer): off by 2^-52 or so of the turns, at worst 3.2e-7 rad at
// position 2^31 with freq 1, and 1e-7 more by the fraction's rounding to fp32.
// Rotation is fp32, rounded once on the store.
//
// Bound: memory (each element read and written once, 3 flops per element): 75600
// slots of 40 + 40 heads, D = 128, bf16, three axes take 490 us (6.3 TB/s); a row
// whose alignment leaves single 16-bit elements runs at 2.4 TB/s.  64 slots of
// 32 + 8 heads take 4.2 us, a launch and one round of loads.
// A thread computes the sines of its pairs once and walks over the heads of
// its slot, Q's heads and then K's, so that the fp64 angle costs little per
// byte; two to four heads are in flight per thread to cover DRAM latency.  Input and
// output have their own strides, so the change from a projection's
// [B, S, H, D] (or a slice of a packed QKV) to [B, H, S, D] costs no pass.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "kernels.cuh"
#include "spattn.h"

namespace spattn {
namespace {

constexpr int kRopeThreads = 128;
struct RopeArgs {
  const void* x[2];  // Q, K
  void* y[2];
  int64_t xs[2][3], ys[2][3];  // batch, head, slot strides (elements)
  int heads, heads_all;        // Q heads; Q and K heads
  int head_group;              // heads per thread
  int64_t slots, tiles;        // tiles: slot tiles per batch entry
  int head_dim, rot, cut1, cut2;  // pairs from cut1 / cut2 on use axis 1 / 2
  bool inverse;
  float mscale;
  const int32_t* pos;
  int64_t pos_batch;
  const double* freqs;
};

// V elements of a row in registers: 32-bit words that hold two 16-bit elements or
// one fp32 (kept packed until they are used: separate 16-bit elements would
// take a register each), or a single 16-bit element.
template <typename T, int V>
struct Vec {
  static constexpr int kWords = V * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords > 0 ? kWords : 1];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (kWords == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 4)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kWords == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kWords == 1)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint32_t x = w[i >> 1];
      if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return __uint_as_float((i & 1) ? x & 0xFFFF0000u : x << 16);
      else
        return __half2float(__ushort_as_half(static_cast<unsigned short>((i & 1) ? x >> 16 : x)));
    }
  }
  // elements i, i + 1 of a pair of words (16-bit types) or i alone
  __device__ __forceinline__ void put2(int i, float lo, float hi) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(lo);
      w[i + 1] = __float_as_uint(hi);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
      w[i >> 1] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __half2 v = __floats2half2_rn(lo, hi);
      w[i >> 1] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  __device__ __forceinline__ void put1(float x) {
    if constexpr (sizeof(T) == 4)
      w[0] = __float_as_uint(x);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else
      w[0] = __half_as_ushort(__float2half_rn(x));
  }
};

// A row is cut into units.  Pairs p, p + rot / 2: unit u < rot / 2 / V holds the
// V-element vectors at u V and u V + rot / 2, and later units are V copied
// elements.  Interleaved pairs lie inside a vector: unit u is the vector at u V,
// turned or copied pair by pair (single elements, for odd alignments: 2u and
// 2u + 1, then copied ones).
template <int V, bool INTER>
__host__ __device__ constexpr int rope_turned(int rot, int head_dim) {
  return INTER && V > 1 ? head_dim / V : rot / 2 / V;
}
template <int V, bool INTER>
__host__ __device__ constexpr int rope_units(int rot, int head_dim) {
  return INTER && V > 1 ? head_dim / V : rot / 2 / V + (head_dim - rot) / V;
}

// Heads in flight per thread.  64 bytes of loads in eight CTAs per SM (64
// registers) is 64 KB per SM; four heads of two vectors took 80 registers, six
// CTAs, and 526 us where this takes 497 (75600 slots x 80 heads, bf16).
template <typename T, int V, bool INTER>
constexpr int kRopeUnroll = V * sizeof(T) * (INTER && V > 1 ? 1 : 2) >= 32 ? 2 : 4;

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const RopeArgs a) {
  using VT = Vec<T, V>;
  constexpr bool kWithin = INTER && V > 1;  // pairs lie inside a vector
  constexpr int U = kRopeUnroll<T, V, INTER>;
  constexpr int P = kWithin ? V / 2 : V;  // pairs of a unit
  const int n_rot = rope_turned<V, INTER>(a.rot, a.head_dim);
  const int units = rope_units<V, INTER>(a.rot, a.head_dim);
  const int64_t b = blockIdx.x / a.tiles;
  const int64_t tile = blockIdx.x - b * a.tiles;
  const int per_tile = kRopeThreads / units > 0 ? kRopeThreads / units : 1;  // slots per tile
  const int h0 = blockIdx.y * a.head_group;
  const int h1 = min(a.heads_all, h0 + a.head_group);

  for (int w = threadIdx.x; w < per_tile * units; w += kRopeThreads) {
    const int u = w % units;
    const int64_t s = tile * per_tile + w / units;
    if (s >= a.slots) continue;
    const bool turn = u < n_rot;
    const int off0 = !turn ? a.rot + (u - n_rot) * V : (INTER && V == 1) ? 2 * u : u * V;
    const int off1 = (INTER && V == 1) ? off0 + 1 : off0 + a.rot / 2;
    float c[P], sn[P];
    if (turn) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int p = u * P + i;
        if (kWithin && p >= a.rot / 2) {  // copied below
          c[i] = sn[i] = 0.f;
          continue;
        }
        const int axis = (p >= a.cut1) + (p >= a.cut2);
        const int64_t pos = __ldg(a.pos + b * a.pos_batch + axis * a.slots + s);
        double t = static_cast<double>(pos) * (__ldg(a.freqs + p) * 0.15915494309189533577);
        t -= rint(t);
        float si, co;
        sincospif(2.0f * static_cast<float>(t), &si, &co);
        c[i] = co * a.mscale;
        sn[i] = (a.inverse ? -si : si) * a.mscale;
      }
    }
    // Q's heads of the range, then K's
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int first = max(h0, k * a.heads), end = k ? h1 : min(h1, a.heads);
      if (first >= end) continue;
      const T* x = static_cast<const T*>(a.x[k]) + b * a.xs[k][0] + (first - k * a.heads) * a.xs[k][1] + s * a.xs[k][2];
      T* y = static_cast<T*>(a.y[k]) + b * a.ys[k][0] + (first - k * a.heads) * a.ys[k][1] + s * a.ys[k][2];
      const int64_t xh = a.xs[k][1], yh = a.ys[k][1];
      for (int h = first; h < end; h += U, x += U * xh, y += U * yh) {
        VT va[U], vb[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (h + j < end) {
            va[j].load(x + j * xh + off0);
            if (!kWithin && turn) vb[j].load(x + j * xh + off1);
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (h + j < end) {
            if (turn) {
              if constexpr (kWithin) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                  const float p0 = va[j].get(2 * i), p1 = va[j].get(2 * i + 1);
                  if (u * P + i < a.rot / 2) va[j].put2(2 * i, p0 * c[i] - p1 * sn[i], p0 * sn[i] + p1 * c[i]);
                }
              } else if constexpr (V > 1) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                  const float p0 = va[j].get(i), q0 = vb[j].get(i), p1 = va[j].get(i + 1), q1 = vb[j].get(i + 1);
                  va[j].put2(i, p0 * c[i] - q0 * sn[i], p1 * c[i + 1] - q1 * sn[i + 1]);
                  vb[j].put2(i, p0 * sn[i] + q0 * c[i], p1 * sn[i + 1] + q1 * c[i + 1]);
                }
              } else {
                const float p0 = va[j].get(0), q0 = vb[j].get(0);
                va[j].put1(p0 * c[0] - q0 * sn[0]);
                vb[j].put1(p0 * sn[0] + q0 * c[0]);
              }
              if constexpr (!kWithin) vb[j].store(y + j * yh + off1);
            }
            va[j].store(y + j * yh + off0);
          }
        }
      }
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_rope_v(RopeArgs& a, int64_t batch, cudaStream_t st) {
  constexpr int U = kRopeUnroll<T, V, INTER>;
  const int units = rope_units<V, INTER>(a.rot, a.head_dim);
  const int per_tile = kRopeThreads / units > 0 ? kRopeThreads / units : 1;
  a.tiles = (a.slots + per_tile - 1) / per_tile;
  const int64_t blocks = a.tiles * batch;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  // All heads in one thread while that leaves four CTAs per SM; fewer heads per
  // thread below that, down to one unrolled group.
  const int64_t want = (4 * 148 + blocks - 1) / blocks;
  const int groups_max = (a.heads_all + U - 1) / U;
  const int64_t groups = want > groups_max ? groups_max : want;
  a.head_group = static_cast<int>((a.heads_all + groups - 1) / groups);
  a.head_group = (a.head_group + U - 1) / U * U;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((a.heads_all + a.head_group - 1) / a.head_group));
  rope_kernel<T, V, INTER><<<grid, kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t launch_rope_t(RopeArgs& a, int64_t batch, cudaStream_t st) {
  // Widest vector (up to 16 bytes) that divides the halves of the turned part and
  // the copied tail (the row, when pairs lie inside a vector), every stride and
  // every address.
  constexpr int kMax = 16 / sizeof(T);
  int v = kMax;
  auto fits = [&](int w) {
    if (INTER ? a.head_dim % w : (a.rot / 2) % w || (a.head_dim - a.rot) % w) return false;
    for (int k = 0; k < (a.heads_all > a.heads ? 2 : 1); ++k) {
      if (reinterpret_cast<uintptr_t>(a.x[k]) % (w * sizeof(T)) || reinterpret_cast<uintptr_t>(a.y[k]) % (w * sizeof(T)))
        return false;
      for (int i = 0; i < 3; ++i)
        if (a.xs[k][i] % w || a.ys[k][i] % w) return false;
    }
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  if constexpr (kMax == 8)
    if (v == 8) return launch_rope_v<T, 8, INTER>(a, batch, st);
  if (v == 4) return launch_rope_v<T, 4, INTER>(a, batch, st);
  if (v == 2) return launch_rope_v<T, 2, INTER>(a, batch, st);
  return launch_rope_v<T, 1, INTER>(a, batch, st);
}

template <typename T>
cudaError_t launch_rope(RopeArgs& a, int64_t batch, bool interleaved, cudaStream_t st) {
  return interleaved ? launch_rope_t<T, true>(a, batch, st) : launch_rope_t<T, false>(a, batch, st);
}

}  // namespace
}  // namespace spattn

using namespace spattn;

extern "C" int spattn_rope(const spattn_rope_layout* L, const void* q, const void* k, const int32_t* pos,
                           const double* freqs, void* q_out, void* k_out, void* stream) {
  if (!L || L->dtype < 0 || L->dtype > 2 || L->batch < 0 || L->slots < 0 || L->heads < 1 || L->kv_heads < 0 ||
      L->head_dim < 1 || L->rot_dim < 0 || L->rot_dim > L->head_dim || L->rot_dim % 2 || !std::isfinite(L->mscale) ||
      L->n_axes < 1 || L->n_axes > 3)
    return SPATTN_ERR_INVALID_ARG;
  if (L->head_dim > 1024 || L->heads > 32767 || L->kv_heads > 32767) return SPATTN_ERR_UNSUPPORTED;
  int64_t pairs = 0;
  for (int i = 0; i < L->n_axes; ++i) {
    if (L->sections[i] < 0) return SPATTN_ERR_INVALID_ARG;
    pairs += L->sections[i];
  }
  if (pairs != L->rot_dim / 2) return SPATTN_ERR_INVALID_ARG;
  if (L->batch == 0 || L->slots == 0) return SPATTN_OK;
  const uintptr_t es = L->dtype == 2 ? 4 : 2;
  auto good = [](const void* p, uintptr_t al) { return p && reinterpret_cast<uintptr_t>(p) % al == 0; };
  if (!good(q, es) || !good(q_out, es) || (L->kv_heads > 0 && (!good(k, es) || !good(k_out, es))) || !good(pos, 4) ||
      (pairs > 0 && !good(freqs, 8)))
    return SPATTN_ERR_INVALID_ARG;
  RopeArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k_out;
  for (int i = 0; i < 3; ++i) {
    a.xs[0][i] = L->q_stride[i];
    a.ys[0][i] = L->q_out_stride[i];
    a.xs[1][i] = L->kv_heads ? L->k_stride[i] : 0;
    a.ys[1][i] = L->kv_heads ? L->k_out_stride[i] : 0;
  }
  a.heads = L->heads;
  a.heads_all = L->heads + L->kv_heads;
  a.slots = L->slots;
  a.head_dim = L->head_dim;
  a.rot = L->rot_dim;
  a.cut1 = L->n_axes > 1 ? L->sections[0] : 0x7FFFFFFF;
  a.cut2 = L->n_axes > 2 ? L->sections[0] + L->sections[1] : 0x7FFFFFFF;
  a.inverse = L->inverse != 0;
  a.mscale = L->mscale;
  a.pos = pos;
  a.pos_batch = L->pos_batch_stride;
  a.freqs = freqs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = L->interleaved != 0;
  const cudaError_t e = L->dtype == 0   ? launch_rope<__nv_bfloat16>(a, L->batch, inter, s)
                        : L->dtype == 1 ? launch_rope<__half>(a, L->batch, inter, s)
                                        : launch_rope<float>(a, L->batch, inter, s);
  return e == cudaSuccess ? SPATTN_OK : e == cudaErrorInvalidValue ? SPATTN_ERR_UNSUPPORTED : SPATTN_ERR_CUDA;
}
