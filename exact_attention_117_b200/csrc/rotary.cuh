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
// Bound: every channel is read once and written once; the issue slots are half
// taken.  B=2 H=16 N=4096 d=128, queries and keys (134 MB): 24.1 us, 5.6 TB/s; a
// decode step of 8 tokens 2.8 us, a launch.
//
// A block takes a few positions and a range of heads.  Its threads first compute
// each (position, pair)'s sine and cosine once, into shared memory, with their
// first rows' loads already in flight; then each keeps the sines of one position
// and one 16-byte vector of pairs in registers and walks the heads.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"

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
  int n, rot, d;
  int chunks;             // vectors (or pairs of them) of a row
  int block_pos, block_heads, pos_blocks, head_groups;
  int block_rows;         // chunks * block_pos: threads that share a head
  float amplitude;
  float sin_sign;         // the gradient turns by -t: -1
  int pos64;
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryPairs = 512;  // (position, pair)s of a block

// V elements of type T (2 to 16 bytes) as they lie in memory.  16-bit types are
// taken apart and put together two at a time.
template <typename T, int V>
struct alignas(V * sizeof(T)) RotVec {
  static constexpr int kWords = (V * sizeof(T) + 3) / 4;
  using Word = std::conditional_t<V * sizeof(T) == 2, uint16_t, uint32_t>;
  Word w[kWords];
};
template <typename T>
__device__ __forceinline__ float2 rot_split(uint32_t w);
template <>
__device__ __forceinline__ float2 rot_split<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 rot_split<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t rot_join(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t rot_join<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t rot_join<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void rot_unpack(const RotVec<T, V>& x, float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(x.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
      const float2 v = rot_split<T>(x.w[i]);
      f[2 * i] = v.x;
      if (2 * i + 1 < V) f[(2 * i + 1) % V] = v.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void rot_pack(const float (&f)[V], RotVec<T, V>& x) {
  using Word = typename RotVec<T, V>::Word;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) x.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i)
      x.w[i] = static_cast<Word>(rot_join<T>(f[2 * i], f[(2 * i + 1) % V]));
  }
}

// V: elements of a vector.  Half layout: a rotated chunk is two vectors, at
// c V and rot/2 + c V (V pairs).  Interleaved: one vector of V/2 pairs.
// Chunks behind the rotated ones copy one vector each of [rot, d).
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using Vec = RotVec<T, V>;
  constexpr int kPairs = kInterleaved ? V / 2 : V;
  constexpr int kBatch = 4;  // heads whose loads are in flight together
  // the sines of a position: four pairs of a chunk together, chunks beside
  // each other, so that a warp's 16-byte reads meet no bank twice
  constexpr int kRun = kPairs < 4 ? kPairs : 4;
  __shared__ __align__(16) float s_cos[kRotaryPairs], s_sin[kRotaryPairs];

  // blocks: head groups fastest, then positions, then the batch
  const int group = blockIdx.x % p.head_groups;
  const int rest = blockIdx.x / p.head_groups;
  const int b = rest / p.pos_blocks;
  const int n0 = (rest - b * p.pos_blocks) * p.block_pos;
  const int rot_chunks = (kInterleaved ? p.rot : p.rot / 2) / V;
  const int pairs = p.rot / 2;

  const int tid = threadIdx.x, head_lane = tid / p.block_rows;
  const int in_head = tid - head_lane * p.block_rows;
  const int pos = in_head / p.chunks, c = in_head - pos * p.chunks;
  const int n = n0 + pos, head_lanes = kRotaryThreads / p.block_rows;
  const bool live = head_lane < head_lanes && n < p.n, turned = c < rot_chunks;
  const int e = turned ? c * V : p.rot + (c - rot_chunks) * V;

  // The thread's heads: every head_lanes-th of the block's range, which is cut
  // into the queries' heads and the keys'.
  const int first = group * p.block_heads;
  int end = live ? min(first + p.block_heads, p.heads[0] + p.heads[1]) : 0;
  if (!dbg_access(!live || (n >= 0 && e >= 0 && e + V <= (turned ? (kInterleaved ? p.rot : p.rot / 2) : p.d) &&
                            (pos + 1) * pairs <= kRotaryPairs && first >= 0),
                  kErrRotary))
    end = 0;
  const T* x[2];
  T* y[2];
  int count[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int from = w ? p.heads[0] : 0;
    const int stop = min(end, w ? end : p.heads[0]);
    int h = first + head_lane;
    if (h < from) h += (from - h + head_lanes - 1) / head_lanes * head_lanes;
    count[w] = h < stop ? (stop - h + head_lanes - 1) / head_lanes : 0;
    const long long hw = h - from;
    x[w] = static_cast<const T*>(p.x[w]) + b * p.xs[w][0] + hw * p.xs[w][1] + n * p.xs[w][2] + e;
    y[w] = static_cast<T*>(p.y[w]) + b * p.ys[w][0] + hw * p.ys[w][1] + n * p.ys[w][2] + e;
  }
  Vec a[kBatch], z[kBatch];
  auto load = [&](int w) {
    const long long step = p.xs[w][1] * head_lanes;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= count[w]) continue;
      const T* from = x[w] + u * step;
      a[u] = *reinterpret_cast<const Vec*>(from);
      if (!kInterleaved && turned) z[u] = *reinterpret_cast<const Vec*>(from + p.rot / 2);
    }
    x[w] += kBatch * step;
  };
  if (count[0] > 0) load(0);
  else if (count[1] > 0) load(1);

  for (int i = tid; i < p.block_pos * pairs; i += kRotaryThreads) {
    const int ps = i / pairs, pair = i - ps * pairs;
    if (n0 + ps >= p.n) break;
    const long long at = b * p.pos_stride + n0 + ps;
    const double where = p.pos64 ? static_cast<double>(static_cast<const long long*>(p.positions)[at])
                                 : static_cast<double>(static_cast<const int*>(p.positions)[at]);
    const double turns = where * p.inv_freq[pair] * 0.15915494309189535;
    const float r = static_cast<float>(turns - rint(turns));
    float s, co;
    if (sizeof(T) == 2)  // within 2^-21 on [-pi, pi], a thousandth of fp16's half step
      __sincosf(6.283185307179586f * r, &s, &co);
    else
      sincospif(2.f * r, &s, &co);
    const int in = pair % kPairs;
    const int to = ps * pairs + (in / kRun * rot_chunks + pair / kPairs) * kRun + in % kRun;
    s_cos[to] = co * p.amplitude;
    s_sin[to] = s * p.amplitude * p.sin_sign;
  }
  __syncthreads();

  float cs[kPairs], sn[kPairs];
  if (live && turned) {
    struct alignas(4 * kRun) Run { float v[kRun]; };
#pragma unroll
    for (int k = 0; k < kPairs; k += kRun) {
      const int at = pos * pairs + (k / kRun * rot_chunks + c) * kRun;
      const Run rc = *reinterpret_cast<const Run*>(s_cos + at), rs = *reinterpret_cast<const Run*>(s_sin + at);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        cs[k + i] = rc.v[i];
        sn[k + i] = rs.v[i];
      }
    }
  }
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const long long step = p.ys[w][1] * head_lanes;
    if (w == 1 && count[1] > 0 && count[0] > 0) load(1);  // else loaded above
    for (int left = count[w]; left > 0; left -= kBatch) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (u >= left) continue;
        T* to = y[w] + u * step;
        if (turned) {
          float f[V], g[V];
          rot_unpack<T, V>(a[u], f);
          if (!kInterleaved) rot_unpack<T, V>(z[u], g);
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            float& r1 = kInterleaved ? f[(2 * k) % V] : f[k];
            float& r2 = kInterleaved ? f[(2 * k + 1) % V] : g[k];
            const float x1 = r1, x2 = r2;
            r1 = x1 * cs[k] - x2 * sn[k];
            r2 = x2 * cs[k] + x1 * sn[k];
          }
          rot_pack<T, V>(f, a[u]);
          if (!kInterleaved) {
            rot_pack<T, V>(g, z[u]);
            *reinterpret_cast<Vec*>(to + p.rot / 2) = z[u];
          }
        }
        *reinterpret_cast<Vec*>(to) = a[u];
      }
      y[w] += kBatch * step;
      if (left > kBatch) {
        count[w] = left - kBatch;
        load(w);
      }
    }
  }
}

}  // namespace fa
