// Rotary positions of Q and K, forward and backward.
//
// Pair p of a row (elements 2p, 2p + 1 when interleaved, p and p + rot/2
// otherwise) is turned by the angle t = pos[axis(p)] * freq[p] and scaled:
//   a' = m (a cos t - b sin t),   b' = m (a sin t + b cos t);
// the gradient is the same with -t.  Elements from rot on are copied.
//
// The angle is formed in fp64 as a fraction of a turn (pos * freq / 2 pi,
// less its nearest integer), which keeps 1e-7 rad at position 2^31; only the
// fraction is rounded to fp32.  Rotation is fp32, rounded once on the store.
//
// Bound: memory (each element read and written once, 3 flops per element).
// A thread computes the sines of its pairs once and walks over the heads of
// its slot, Q's heads and then K's, so that the fp64 angle costs little per
// byte; four heads are in flight per thread to cover DRAM latency.  Input and
// output have their own strides, so the change from a projection's
// [B, S, H, D] (or a slice of a packed QKV) to [B, H, S, D] costs no pass.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "kernels.cuh"
#include "spattn.h"

namespace spattn {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;  // heads in flight per thread

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

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half& y) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// A row is cut into units: unit u < rot / 2 / V holds the two V-element vectors
// at u V and u V + rot / 2 (for interleaved single elements, 2u and 2u + 1),
// which are whole pairs in either layout; later units are V copied elements.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  using VT = Vec<T, V>;
  constexpr bool kWithin = INTER && V > 1;  // pairs lie inside a vector
  const int n_rot = a.rot / 2 / V;
  const int units = n_rot + (a.head_dim - a.rot) / V;
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
    float c[V], sn[V];
    if (turn) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // pairs of the first vector, then of the second, when they lie inside
        const int p = !kWithin ? u * V + i : (i < V / 2 ? off0 / 2 + i : off1 / 2 + i - V / 2);
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
    for (int h = h0; h < h1; h += kRopeUnroll) {
      VT va[kRopeUnroll], vb[kRopeUnroll];
#pragma unroll
      for (int j = 0; j < kRopeUnroll; ++j) {
        if (h + j < h1) {
          const int k = h + j >= a.heads;
          const T* x = static_cast<const T*>(a.x[k]) + b * a.xs[k][0] + (h + j - k * a.heads) * a.xs[k][1] + s * a.xs[k][2];
          va[j] = *reinterpret_cast<const VT*>(x + off0);
          if (turn) vb[j] = *reinterpret_cast<const VT*>(x + off1);
        }
      }
#pragma unroll
      for (int j = 0; j < kRopeUnroll; ++j) {
        if (h + j < h1) {
          const int k = h + j >= a.heads;
          T* y = static_cast<T*>(a.y[k]) + b * a.ys[k][0] + (h + j - k * a.heads) * a.ys[k][1] + s * a.ys[k][2];
          if (turn) {
            if constexpr (kWithin) {
#pragma unroll
              for (int i = 0; i < V / 2; ++i) {
                const float p0 = to_f(va[j].e[2 * i]), p1 = to_f(va[j].e[2 * i + 1]);
                from_f(p0 * c[i] - p1 * sn[i], va[j].e[2 * i]);
                from_f(p0 * sn[i] + p1 * c[i], va[j].e[2 * i + 1]);
                const float r0 = to_f(vb[j].e[2 * i]), r1 = to_f(vb[j].e[2 * i + 1]);
                from_f(r0 * c[V / 2 + i] - r1 * sn[V / 2 + i], vb[j].e[2 * i]);
                from_f(r0 * sn[V / 2 + i] + r1 * c[V / 2 + i], vb[j].e[2 * i + 1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float p0 = to_f(va[j].e[i]), p1 = to_f(vb[j].e[i]);
                from_f(p0 * c[i] - p1 * sn[i], va[j].e[i]);
                from_f(p0 * sn[i] + p1 * c[i], vb[j].e[i]);
              }
            }
            *reinterpret_cast<VT*>(y + off1) = vb[j];
          }
          *reinterpret_cast<VT*>(y + off0) = va[j];
        }
      }
    }
  }
}

template <typename T, int V>
cudaError_t launch_rope_v(RopeArgs& a, int64_t batch, bool interleaved, cudaStream_t st) {
  const int units = a.rot / 2 / V + (a.head_dim - a.rot) / V;
  const int per_tile = kRopeThreads / units > 0 ? kRopeThreads / units : 1;
  a.tiles = (a.slots + per_tile - 1) / per_tile;
  const int64_t blocks = a.tiles * batch;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  // All heads in one thread while that leaves four CTAs per SM; fewer heads per
  // thread below that, down to one unrolled group.
  const int64_t want = (4 * 148 + blocks - 1) / blocks;
  const int groups_max = (a.heads_all + kRopeUnroll - 1) / kRopeUnroll;
  const int64_t groups = want < 1 ? 1 : want > groups_max ? groups_max : want;
  a.head_group = static_cast<int>((a.heads_all + groups - 1) / groups);
  a.head_group = (a.head_group + kRopeUnroll - 1) / kRopeUnroll * kRopeUnroll;
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((a.heads_all + a.head_group - 1) / a.head_group));
  if (interleaved)
    rope_kernel<T, V, true><<<grid, kRopeThreads, 0, st>>>(a);
  else
    rope_kernel<T, V, false><<<grid, kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope_t(RopeArgs& a, int64_t batch, bool interleaved, cudaStream_t st) {
  // Widest vector (up to 16 bytes) that divides the pair halves, the copied
  // tail, every stride and every address.
  constexpr int kMax = 16 / sizeof(T);
  int v = kMax;
  auto fits = [&](int w) {
    if ((a.rot / 2) % w || (a.head_dim - a.rot) % w) return false;
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
    if (v == 8) return launch_rope_v<T, 8>(a, batch, interleaved, st);
  if (v == 4) return launch_rope_v<T, 4>(a, batch, interleaved, st);
  if (v == 2) return launch_rope_v<T, 2>(a, batch, interleaved, st);
  return launch_rope_v<T, 1>(a, batch, interleaved, st);
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
  const cudaError_t e = L->dtype == 0   ? launch_rope_t<__nv_bfloat16>(a, L->batch, inter, s)
                        : L->dtype == 1 ? launch_rope_t<__half>(a, L->batch, inter, s)
                                        : launch_rope_t<float>(a, L->batch, inter, s);
  return e == cudaSuccess ? SPATTN_OK : e == cudaErrorInvalidValue ? SPATTN_ERR_UNSUPPORTED : SPATTN_ERR_CUDA;
}
