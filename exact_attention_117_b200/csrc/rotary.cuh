// rotary.cuh -- rotary positions of queries and keys, and their gradient.
//
// Channels (x1, x2) of pair i at position p turn by the angle t = p * f_i:
//   y1 = A (x1 cos t - x2 sin t),  y2 = A (x2 cos t + x1 sin t).
// The pairs are (i, i + rot/2) or (2i, 2i + 1); channels from rot on pass
// through.  The map is A times a rotation, so the gradient is the same map
// with -t.
//
// The angle: p * f_i is reduced in 64 bits (t / 2 pi minus its nearest whole
// number; at p = 2^31 a 64-bit product is still exact to 1e-7 turns, a 32-bit
// one would be off by many turns), and sin and cos of the remainder are taken
// in 32 bits.  The products are 32-bit; the result is rounded once.
//
// Bound: every channel is read once and written once.  A thread owns one
// 16-byte vector of pairs at one position and walks `heads_per_thread` heads
// of the queries and then of the keys with it, so the sines are computed once
// for those heads.  Loads of four heads are in flight before the first is
// turned.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace fa {

struct RotaryParams {
  const void* x[2];      // queries, keys
  void* y[2];
  long long xs[2][3];    // strides of x in elements: batch, head, position
  long long ys[2][3];
  int heads[2];
  const void* positions;  // [B, N], or [N] when pos_stride is 0
  const double* inv_freq;
  long long pos_stride;
  long long n_threads;    // B * N * chunks * groups
  int n, rot, d, chunks, heads_per_thread, groups;
  float amplitude;        // the gradient turns by -t: sin_sign = -1
  float sin_sign;
  int pos64;
};

template <typename T>
__device__ __forceinline__ float rot_float(T x);
template <>
__device__ __forceinline__ float rot_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float rot_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float rot_float(float x) { return x; }
template <typename T>
__device__ __forceinline__ T rot_round(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 rot_round(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rot_round(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float rot_round(float x) { return x; }

template <typename T, int V>
struct alignas(V * sizeof(T)) RotVec {
  T v[V];
};

// V: elements of a vector.  Half layout: a rotated chunk is two vectors, at
// c V and rot/2 + c V (V pairs).  Interleaved: one vector of V/2 pairs.
// Chunks behind the rotated ones copy one vector each of [rot, d).
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using Vec = RotVec<T, V>;
  constexpr int kPairs = kInterleaved ? V / 2 : V;
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (id >= p.n_threads) return;
  const int c = static_cast<int>(id % p.chunks);
  const long long rest = id / p.chunks;
  const int group = static_cast<int>(rest % p.groups);
  const long long bn = rest / p.groups;
  const int b = static_cast<int>(bn / p.n);
  const int n = static_cast<int>(bn - static_cast<long long>(b) * p.n);

  const int rot_chunks = kInterleaved ? p.rot / V : p.rot / 2 / V;
  const bool turned = c < rot_chunks;
  const int e1 = turned ? c * V : p.rot + (c - rot_chunks) * V;
  const int e2 = kInterleaved ? e1 : e1 + (turned ? p.rot / 2 : 0);

  float cs[kPairs], sn[kPairs];
  if (turned) {
    const long long at = b * p.pos_stride + n;
    const double pos = p.pos64 ? static_cast<double>(static_cast<const long long*>(p.positions)[at])
                               : static_cast<double>(static_cast<const int*>(p.positions)[at]);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const double turns = pos * p.inv_freq[c * kPairs + i] * 0.15915494309189535;
      const float r = static_cast<float>(turns - rint(turns));
      float s, co;
      sincospif(2.f * r, &s, &co);
      cs[i] = co * p.amplitude;
      sn[i] = s * p.amplitude * p.sin_sign;
    }
  }

  const int h0 = group * p.heads_per_thread;
  const int h_end = min(h0 + p.heads_per_thread, p.heads[0] + p.heads[1]);
  for (int h4 = h0; h4 < h_end; h4 += 4) {
    Vec a[4], z[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int hh = h4 + u;
      if (hh < h_end) {
        const int w = hh >= p.heads[0];
        const int h = w ? hh - p.heads[0] : hh;
        const T* x = static_cast<const T*>(p.x[w]) + b * p.xs[w][0] + h * p.xs[w][1] + n * p.xs[w][2];
        a[u] = *reinterpret_cast<const Vec*>(x + e1);
        if (!kInterleaved && turned) z[u] = *reinterpret_cast<const Vec*>(x + e2);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int hh = h4 + u;
      if (hh < h_end) {
        const int w = hh >= p.heads[0];
        const int h = w ? hh - p.heads[0] : hh;
        T* y = static_cast<T*>(p.y[w]) + b * p.ys[w][0] + h * p.ys[w][1] + n * p.ys[w][2];
        if (turned) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            T& r1 = kInterleaved ? a[u].v[(2 * i) % V] : a[u].v[i];
            T& r2 = kInterleaved ? a[u].v[(2 * i + 1) % V] : z[u].v[i];
            const float x1 = rot_float<T>(r1), x2 = rot_float<T>(r2);
            r1 = rot_round<T>(x1 * cs[i] - x2 * sn[i]);
            r2 = rot_round<T>(x2 * cs[i] + x1 * sn[i]);
          }
          if (!kInterleaved) *reinterpret_cast<Vec*>(y + e2) = z[u];
        }
        *reinterpret_cast<Vec*>(y + e1) = a[u];
      }
    }
  }
}

}  // namespace fa
