// kv4_attend.cuh -- attention of packed queries over the paged 4-bit cache.
//
//   O_i = sum_j softmax_j(scale q_i . K_j) V_j over the keys row i sees,
//   LSE_i = ln sum_j exp(scale q_i . K_j),
// where K_j and V_j are the values the cache's codes stand for.  With K_j =
// mid + s (n - 8) per group of 64 channels (mid = lowest + 8 s),
//   q . K_j = sum_groups s (q . (n - 8)) + mid (sum of q),
// so the matrix instructions multiply the codes themselves and scale and mid
// act on the 64-channel sums; for V, P s goes into the matrix instructions and
// P mid is summed beside them.
//
// Codes are small whole numbers, exact in fp16.  q enters as fp16 after an
// exact scaling of each row by a power of two (largest element in [1, 2)), so
// a bf16 q keeps all its bits down to 2^-24 of the row's largest.  P s enters
// as fp16 relative to a power of two above the largest s seen: 11 bits,
// against the 8 of a bf16 P.  Scores, softmax statistics and O are fp32.
//
// Rows: the queries of a request times the heads that share a kv head, in
// tiles of 8 NT.  Transposed products (S^T = K q^T, O^T = V^T P^T) put tokens
// and channels on the 16-row side of m16n8k16, so a single token of a group of
// up to 8 heads wastes little.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv4.cuh"

namespace fa {

struct Kv4AttendParams {
  const void* q;
  void* o;
  float* lse;             // [tokens, heads]
  const uint8_t* cache;
  const int* table;
  const int* lengths;
  const int* cu_tokens;
  float* part;            // partial results: 2 per CTA
  long long q_st, q_sh, o_st, o_sh;  // strides in elements
  long long table_stride;
  int requests, heads, kv_heads, group, tokens, pages, page_size, width;
  float scale_log2;
  int causal, is_half;
};

constexpr int kKv4Warps = 4;
constexpr int kKv4Chunk = 16 * kKv4Warps;  // keys of a work unit

// ------------------------------------------------------------ the work's order
// Units: (request, row tile, kv head, chunk of keys), chunks innermost.  CTA c
// of n takes units [c U / n, (c + 1) U / n): every CTA reads the same share of
// the cache whatever the lengths are.  A (request, row tile, head) that a
// CTA's range cuts is left as partial results, which the combine kernel joins.
struct Kv4Req {
  int first, n, len, row_tiles, chunks;
};
template <int ROWS>
__device__ __forceinline__ Kv4Req kv4_request(const Kv4AttendParams& p, int b) {
  Kv4Req r;
  r.first = min(max(p.cu_tokens[b], 0), p.tokens);
  r.n = max(min(p.cu_tokens[b + 1], p.tokens) - r.first, 0);
  r.len = max(0, static_cast<int>(min(static_cast<long long>(p.lengths[b]),
                                      static_cast<long long>(p.width) * p.page_size)));
  r.row_tiles = static_cast<int>((static_cast<long long>(r.n) * p.group + ROWS - 1) / ROWS);
  r.chunks = max(1, (r.len + kKv4Chunk - 1) / kKv4Chunk);
  return r;
}
__device__ __forceinline__ long long kv4_units(const Kv4AttendParams& p, const Kv4Req& r) {
  return static_cast<long long>(r.row_tiles) * p.kv_heads * r.chunks;
}

struct Kv4Shared {
  long long warp_sum[kKv4Warps];
  long long total, found_excl;
  int found_b;
};

// Block-wide: the total number of units, and the request that holds unit
// share_of(total) together with the units before it (-1 if there is none).
template <int ROWS, typename F>
__device__ __forceinline__ void kv4_locate(const Kv4AttendParams& p, Kv4Shared& sh, F share_of) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kThreads = kKv4Warps * 32;
  const int chunks = (p.requests + kThreads - 1) / kThreads;
  long long total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * kThreads + tid;
      const long long mine = b < p.requests ? kv4_units(p, kv4_request<ROWS>(p, b)) : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) sh.warp_sum[warp] = incl;
      __syncthreads();
      long long all = 0;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        if (w < warp) incl += sh.warp_sum[w];
        all += sh.warp_sum[w];
      }
      if (pass == 1) {
        const long long u = share_of(total), e = base + incl - mine;
        if (u >= e && u < e + mine) {
          sh.found_b = b;
          sh.found_excl = e;
        }
      }
      base += all;
    }
    if (pass == 0) {
      total = base;
      if (tid == 0) {
        sh.total = total;
        sh.found_b = -1;
      }
    }
  }
  __syncthreads();
}

// Range start of CTA c of n.
__device__ __forceinline__ long long kv4_start(long long total, int c, int n) {
  return total / n * c + total % n * c / n;
}

// ------------------------------------------------------------ matrix pieces
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes 0..7 of a word as four fp16 pairs n - 8: (0, 4), (1, 5), (2, 6), (3, 7).
// A code under the bits of 1024.0 reads 1024 + n, one four bits higher 1024 +
// 16 n; one addition or fused multiply-add takes the offset off, exactly.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t w8 = w >> 8;
  uint32_t a, b, c, d;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(a) : "r"(w));
  asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(b) : "r"(w));
  asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(c) : "r"(w8));
  asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(d) : "r"(w8));
  const uint32_t off1 = 0xe408e408u, sixteenth = 0x2c002c00u, off16 = 0xd480d480u;  // -1032, 1/16, -72
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h[0]) : "r"(a), "r"(off1));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[1]) : "r"(b), "r"(sixteenth), "r"(off16));
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h[2]) : "r"(c), "r"(off1));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[3]) : "r"(d), "r"(sixteenth), "r"(off16));
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[W]) {
  if (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x, w[1 % W] = x.y, w[2 % W] = x.z, w[3 % W] = x.w;
  } else if (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    w[0] = x.x, w[1 % W] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

// Row r of a 16-token tile's fragments is token tau(r): a lane's V tokens for
// one load are then four adjacent rows.
__device__ __forceinline__ int kv4_tau(int r) { return (r >> 1) + 4 * (r & 1); }

template <int D, int NT>
struct Kv4AttendLayout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;  // floats of a row in the merge buffer
  static constexpr int kOffMl = kKv4Warps * kRows * kPitch * 4;
  static constexpr int kBytes = kOffMl + 2 * kKv4Warps * kRows * 4;
  static constexpr int kPartFloats = kRows * (D + 2);  // O, then m and l
};

// One partial or final result from the per-warp results in shared memory.
template <int D, int NT>
__device__ __forceinline__ void kv4_store_row(const Kv4AttendParams& p, const Kv4Req& rq, int h,
                                              int row, int ch, float o, float m, float l) {
  // `row` of the request: query row / group, head h group + row % group
  const int tok = rq.first + row / p.group, head = h * p.group + row % p.group;
  const float out = l == 0.f ? 0.f : o / l;
  const long long at = tok * p.o_st + head * p.o_sh + ch;
  if (p.is_half)
    static_cast<__half*>(p.o)[at] = __float2half_rn(out);
  else
    static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(out);
  if (ch == 0)
    p.lse[static_cast<long long>(tok) * p.heads + head] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32)
    kv4_attend_kernel(const __grid_constant__ Kv4AttendParams p) {
  using T = Kv4Tile<D>;
  using L = Kv4AttendLayout<D, NT>;
  constexpr int kGroups = D / 64, kKW = D / 32, kVW = D / 64;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Kv4Shared sh;
  float* merge = reinterpret_cast<float*>(smem);
  float* s_m = reinterpret_cast<float*>(smem + L::kOffMl);
  float* s_l = s_m + kKv4Warps * L::kRows;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int ctas = gridDim.x, cta = blockIdx.x;
  kv4_locate<L::kRows>(p, sh, [&](long long total) { return kv4_start(total, cta, ctas); });
  const long long u_begin = kv4_start(sh.total, cta, ctas), u_end = kv4_start(sh.total, cta + 1, ctas);
  if (u_begin >= u_end) return;
  int b = sh.found_b;
  long long excl = sh.found_excl;
  Kv4Req rq = kv4_request<L::kRows>(p, b);

  for (long long u = u_begin; u < u_end;) {
    while (u - excl >= kv4_units(p, rq)) {
      excl += kv4_units(p, rq);
      rq = kv4_request<L::kRows>(p, ++b);
    }
    const long long job = (u - excl) / rq.chunks;
    const int c0 = static_cast<int>(u - excl - job * rq.chunks);
    const int c1 = static_cast<int>(min(static_cast<long long>(rq.chunks), c0 + (u_end - u)));
    const int h = static_cast<int>(job % p.kv_heads);
    const int row0 = static_cast<int>(job / p.kv_heads) * L::kRows;
    const int rows = min(L::kRows, rq.n * p.group - row0);

    // ---- the rows: q as B fragments, sums over groups, factor, visible keys
    uint32_t qf[NT][kKW][4];
    float qs[NT][kGroups][2], rs[NT][2];
    int lim[NT][2];
    int all_see = 0x7fffffff, any_sees = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;  // this lane's row of the B fragments
      float x[kKW][8], top = 0.f;
      const bool real = r < rows;
      const int row = row0 + r;
      const long long at = real ? (rq.first + row / p.group) * p.q_st +
                                      (h * p.group + row % p.group) * p.q_sh
                                : 0;
#pragma unroll
      for (int j = 0; j < kKW; ++j) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (real)
          raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + 32 * j + 8 * t);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.is_half) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[j][2 * i] = f.x;
            x[j][2 * i + 1] = f.y;
          } else {
            x[j][2 * i] = bf16_lo(w[i]);
            x[j][2 * i + 1] = bf16_hi(w[i]);
          }
          top = fmaxf(top, fmaxf(fabsf(x[j][2 * i]), fabsf(x[j][2 * i + 1])));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e with top / 2^e in [1, 2); kept within 2^+-100
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 227);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
      float sum[kGroups] = {};
#pragma unroll
      for (int j = 0; j < kKW; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qf[nt][j][i] = pack_f16x2(x[j][i] * down, x[j][i + 4] * down);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[nt][j][i]));
          sum[j / 2] += f.x + f.y;
        }
      }
#pragma unroll
      for (int gp = 0; gp < kGroups; ++gp) {
        sum[gp] += __shfl_xor_sync(0xffffffffu, sum[gp], 1);
        sum[gp] += __shfl_xor_sync(0xffffffffu, sum[gp], 2);
      }
      // from the lane of a row (g = row) to the lanes of its column (t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int src = (2 * t + i) * 4;
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp)
          qs[nt][gp][i] = __shfl_sync(0xffffffffu, sum[gp], src);
        rs[nt][i] = __shfl_sync(0xffffffffu, up, src) * p.scale_log2;
        const int rr = 8 * nt + 2 * t + i;
        int see = rq.len;
        if (p.causal) see = min(max(rq.len - rq.n + (row0 + rr) / p.group + 1, 0), rq.len);
        lim[nt][i] = rr < rows ? see : 0;
        if (rr < rows) {
          all_see = min(all_see, see);
          any_sees = max(any_sees, see);
        }
      }
    }
    all_see = __reduce_min_sync(0xffffffffu, all_see);
    any_sees = __reduce_max_sync(0xffffffffu, any_sees);

    float acc[kVW][4][NT][4] = {};
    float lo_sum[NT][kGroups][2] = {}, l[NT][2] = {}, m[NT][2], thr[NT][2];
    float vref = 0.f, vinv = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = 0.f;
        thr[nt][i] = -INFINITY;
      }

    const int kt_end = min(c1 * kKv4Warps, (any_sees + 15) / 16);
    for (int kt = c0 * kKv4Warps + warp; kt < kt_end; kt += kKv4Warps) {
      const int key0 = kt * 16;
      const int page = p.table[b * p.table_stride + key0 / p.page_size];
      if (page < 0 || page >= p.pages) {  // reported, and read as absent keys
        if (lane == 0) atomicOr(&g_error_word, kErrBadPage);
        continue;
      }
      const uint8_t* tile =
          p.cache + ((static_cast<long long>(page) * p.kv_heads + h) * (p.page_size / 16) +
                     key0 % p.page_size / 16) * T::kBytes;
      uint32_t k0[kKW], k1[kKW], kp0[kGroups], kp1[kGroups], vp0[kGroups], vp1[kGroups], vw[4][kVW];
      const int tau = kv4_tau(g);
      load_words<kKW>(tile + tau * T::kRow + t * kKW * 4, k0);
      load_words<kKW>(tile + (tau + 8) * T::kRow + t * kKW * 4, k1);
      load_words<kGroups>(tile + T::kOffKPar + tau * T::kPar, kp0);
      load_words<kGroups>(tile + T::kOffKPar + (tau + 8) * T::kPar, kp1);
      load_words<kGroups>(tile + T::kOffVPar + tau * T::kPar, vp0);
      load_words<kGroups>(tile + T::kOffVPar + (tau + 8) * T::kPar, vp1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_words<kVW>(tile + T::kOffV + (t + 4 * i) * T::kRow + g * kVW * 4, vw[i]);

      // ---- S^T = K q^T, by groups
      float s[NT][kGroups][4] = {};
#pragma unroll
      for (int j = 0; j < kKW; ++j) {
        uint32_t a[4], c[4];
        codes_f16(k0[j], a);
        codes_f16(k1[j], c);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(s[nt][j / 2], a[0], c[0], a[1], c[1], qf[nt][j][0], qf[nt][j][1]);
          mma_f16(s[nt][j / 2], a[2], c[2], a[3], c[3], qf[nt][j][2], qf[nt][j][3]);
        }
      }
      const bool masked = key0 + 16 > all_see;
      const int key[2] = {key0 + tau, key0 + tau + 8};
      float ks[2][kGroups], km[2][kGroups], vs[2][kGroups], vm[2][kGroups];
      bool again = false;
#pragma unroll
      for (int gp = 0; gp < kGroups; ++gp) {
        ks[0][gp] = bf16_lo(kp0[gp]);
        ks[1][gp] = bf16_lo(kp1[gp]);
        km[0][gp] = fmaf(8.f, ks[0][gp], bf16_hi(kp0[gp]));
        km[1][gp] = fmaf(8.f, ks[1][gp], bf16_hi(kp1[gp]));
        vs[0][gp] = bf16_lo(vp0[gp]);
        vs[1][gp] = bf16_lo(vp1[gp]);
        vm[0][gp] = fmaf(8.f, vs[0][gp], bf16_hi(vp0[gp]));
        vm[1][gp] = fmaf(8.f, vs[1][gp], bf16_hi(vp1[gp]));
        // keys no row sees may hold anything
        if (masked) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (key[i] >= any_sees) vs[i][gp] = vm[i][gp] = 0.f;
        }
        again |= vs[0][gp] > vref || vs[1][gp] > vref;
      }
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = c >> 1, r = c & 1;
          float v = 0.f;
#pragma unroll
          for (int gp = 0; gp < kGroups; ++gp)
            v += ks[i][gp] * s[nt][gp][c] + km[i][gp] * qs[nt][gp][r];
          v *= rs[nt][r];
          if (masked && key[i] >= lim[nt][r]) v = -INFINITY;
          x[nt][c] = v;
          again |= v > thr[nt][r];
        }
      // ---- the running reference moves only when a score passes it by 2^8
      // (or a scale of V passes its own): P stays below 2^8, far from fp16's
      // largest, and most tiles need no reduction over lanes
      if (__any_sync(0xffffffffu, again)) {
        float top = vref;
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) top = fmaxf(top, fmaxf(vs[0][gp], vs[1][gp]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float vf = 1.f;
        if (top > vref) {
          const uint32_t bits = min((__float_as_uint(top) & 0x7f800000u) + 0x800000u, 0x7f000000u);
          const float next = __uint_as_float(bits);
          vf = vref / next;
          vref = next;
          vinv = 1.f / next;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float hi = fmaxf(x[nt][r], x[nt][r + 2]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            const bool none = thr[nt][r] == -INFINITY;
            float f = 1.f;
            if (hi > -INFINITY && (none || hi > m[nt][r])) {
              f = none ? 0.f : ex2_approx(m[nt][r] - hi);
              m[nt][r] = hi;
              thr[nt][r] = hi + 8.f;
            }
            l[nt][r] *= f;
#pragma unroll
            for (int gp = 0; gp < kGroups; ++gp) lo_sum[nt][gp][r] *= f;
#pragma unroll
            for (int j = 0; j < kVW; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc[j][i][nt][r] *= f * vf;
                acc[j][i][nt][r + 2] *= f * vf;
              }
          }
      }
      // ---- P, P s as B fragments, P mid
      uint32_t pb[NT][kGroups][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          e[c] = ex2_approx(x[nt][c] - m[nt][c & 1]);
          l[nt][c & 1] += e[c];
        }
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) {
          float pv[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = c >> 1, r = c & 1;
            pv[c] = e[c] * (vs[i][gp] * vinv);
            float pm = e[c] * vm[i][gp];
            if (masked && key[i] >= lim[nt][r]) pv[c] = pm = 0.f;
            lo_sum[nt][gp][r] += pm;
          }
          pb[nt][gp][0] = transpose8(pack_f16x2(pv[0], pv[1]));
          pb[nt][gp][1] = transpose8(pack_f16x2(pv[2], pv[3]));
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < kVW; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          uint32_t a[4], c[4];
          codes_f16(__byte_perm(vw[0][j], vw[1][j], sel), a);
          codes_f16(__byte_perm(vw[2][j], vw[3][j], sel), c);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(acc[j][2 * half][nt], a[0], a[1], c[0], c[1], pb[nt][j][0], pb[nt][j][1]);
            mma_f16(acc[j][2 * half + 1][nt], a[2], a[3], c[2], c[3], pb[nt][j][0], pb[nt][j][1]);
          }
        }
    }

    // ---- this warp's results to shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[nt][r];
        float lo[kGroups];
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) lo[gp] = lo_sum[nt][gp][r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
          for (int gp = 0; gp < kGroups; ++gp) lo[gp] += __shfl_xor_sync(0xffffffffu, lo[gp], o);
        }
        const int row = 8 * nt + 2 * t + r;
        float* to = merge + (warp * L::kRows + row) * L::kPitch;
#pragma unroll
        for (int j = 0; j < kVW; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            to[64 * j + 8 * g + 2 * i] = fmaf(acc[j][i][nt][r], vref, lo[j]);
            to[64 * j + 8 * g + 2 * i + 1] = fmaf(acc[j][i][nt][r + 2], vref, lo[j]);
          }
        if (g == 0) {
          // no key seen (a row of NaN scores has a NaN sum instead)
          s_m[warp * L::kRows + row] = thr[nt][r] == -INFINITY && sum == 0.f ? -INFINITY : m[nt][r];
          s_l[warp * L::kRows + row] = sum;
        }
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == rq.chunks;
    float* part = p.part + (2LL * cta + (u == u_begin && c0 > 0 ? 0 : 1)) * L::kPartFloats;
    for (int idx = tid; idx < rows * D; idx += kKv4Warps * 32) {
      const int r = idx / D, ch = idx % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) top = fmaxf(top, s_m[w * L::kRows + r]);
      float o = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        const float mw = s_m[w * L::kRows + r];
        if (mw == -INFINITY) continue;
        const float f = ex2_approx(mw - top);
        o = fmaf(merge[(w * L::kRows + r) * L::kPitch + ch], f, o);
        sum = fmaf(s_l[w * L::kRows + r], f, sum);
      }
      if (whole) {
        kv4_store_row<D, NT>(p, rq, h, row0 + r, ch, o, top, sum);
      } else {
        part[r * D + ch] = o;
        if (ch == 0) {
          part[L::kRows * D + r] = top;
          part[L::kRows * (D + 1) + r] = sum;
        }
      }
    }
    __syncthreads();
    u += c1 - c0;
  }
}

// Joins the partial results.  Block c looks at the start of CTA c + 1's range:
// if it cuts a (request, row tile, head), and no earlier range start does, the
// block owns that cut one and sums its pieces, left by the CTAs in order.
template <int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32)
    kv4_combine_kernel(const __grid_constant__ Kv4AttendParams p, int ctas) {
  using L = Kv4AttendLayout<D, NT>;
  __shared__ Kv4Shared sh;
  const int cta = blockIdx.x + 1;
  kv4_locate<L::kRows>(p, sh, [&](long long total) { return kv4_start(total, cta, ctas); });
  if (sh.found_b < 0) return;
  const long long total = sh.total, cut = kv4_start(total, cta, ctas);
  const Kv4Req rq = kv4_request<L::kRows>(p, sh.found_b);
  const long long job = (cut - sh.found_excl) / rq.chunks;
  const long long u0 = sh.found_excl + job * rq.chunks, u1 = u0 + rq.chunks;
  if (cut == u0 || kv4_start(total, cta - 1, ctas) > u0) return;
  int last = cta;  // the CTA that holds the last unit
  while (kv4_start(total, last + 1, ctas) < u1) ++last;
  const int h = static_cast<int>(job % p.kv_heads);
  const int row0 = static_cast<int>(job / p.kv_heads) * L::kRows;
  const int rows = min(L::kRows, rq.n * p.group - row0);
  for (int idx = threadIdx.x; idx < rows * D; idx += kKv4Warps * 32) {
    const int r = idx / D, ch = idx % D;
    float o = 0.f, sum = 0.f, top = -INFINITY;
    for (int c = cta - 1; c <= last; ++c) {
      // empty ranges (fewer units than CTAs) left nothing
      if (kv4_start(total, c, ctas) == kv4_start(total, c + 1, ctas)) continue;
      const float* part = p.part + (2LL * c + (kv4_start(total, c, ctas) > u0 ? 0 : 1)) * L::kPartFloats;
      const float m = part[L::kRows * D + r];
      if (m == -INFINITY) continue;
      const float next = fmaxf(top, m);
      const float fo = ex2_approx(top - next), fn = ex2_approx(m - next);
      o = o * fo + part[r * D + ch] * fn;
      sum = sum * fo + part[L::kRows * (D + 1) + r] * fn;
      top = next;
    }
    kv4_store_row<D, NT>(p, rq, h, row0 + r, ch, o, top, sum);
  }
}

}  // namespace fa
