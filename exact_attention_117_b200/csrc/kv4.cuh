// kv4.cuh -- the paged 4-bit key/value cache: its layout, the kernels that
// write and read it, and the kernel that plans its pages.
//
// The cache is uint8 [pages, kv_heads, page / 16, 18 d].  A tile of 18 d bytes
// holds 16 tokens of one kv head, contiguous, so that attention fetches a tile
// with one copy:
//   K codes  16 rows of d/2 bytes      K parameters  16 rows of d/64 pairs
//   V codes  16 rows of d/2 bytes      V parameters  16 rows of d/64 pairs
// A group of 64 channels of one token and head shares a pair (scale, lowest
// value) in bf16; a code n in 0..15 stands for lowest + scale n.  32-bit word w
// of a row holds channels 8w .. 8w + 7, the first in the lowest four bits.
// The words stand in the order in which attention's matrix fragments take
// them: word 4j + t of a K row at place t d/32 + j (a lane of its fragments
// reads d/32 adjacent words), word 8j + g of a V row at place g d/64 + j.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"

namespace fa {

constexpr int kKv4TileTokens = 16;
constexpr int kKv4Group = 64;

template <int D>
struct Kv4Tile {
  static constexpr int kRow = D / 2;                // code bytes of a token
  static constexpr int kPar = D / kKv4Group * 4;    // parameter bytes of a token
  static constexpr int kOffK = 0;
  static constexpr int kOffKPar = 16 * kRow;
  static constexpr int kOffV = kOffKPar + 16 * kPar;
  static constexpr int kOffVPar = kOffV + 16 * kRow;
  static constexpr int kBytes = kOffVPar + 16 * kPar;
  static_assert(kBytes == 18 * D, "tile size");
  __host__ __device__ static constexpr int place(int word, bool value) {
    return value ? (word & 7) * (D / 64) + (word >> 3) : (word & 3) * (D / 32) + (word >> 2);
  }
};

// Division of 0 <= n < 2^31 by a divisor known at launch: one high product, an
// addition and a shift (m = floor(2^32 (2^s - d) / d) + 1, 2^s >= d).
struct FastDiv {
  uint32_t mul, shift, by;
  static FastDiv of(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1), s, d};
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
};

struct Kv4StoreParams {
  const __nv_bfloat16* x[2];  // keys, values
  __nv_bfloat16* y[2];        // of a gather
  long long st[2], sh[2];     // strides in elements: token, head
  uint8_t* cache;
  const long long* slots;     // page * page_size + offset in the page
  long long n_slots;          // slots of the cache
  long long n_items;          // tokens * heads * 2 * (d / 8)
  int heads, page_size;
};

// Byte offset of the row parts of a (slot, head): tile base and row.
template <int D>
__device__ __forceinline__ long long kv4_tile_at(const Kv4StoreParams& p, long long slot, int h) {
  const long long page = slot / p.page_size;
  const int off = static_cast<int>(slot - page * p.page_size);
  return ((page * p.heads + h) * (p.page_size / 16) + off / 16) * Kv4Tile<D>::kBytes;
}

__device__ __forceinline__ float group8_min(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v = fminf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float group8_max(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Smallest bf16 s with 15 s >= span (span > 0, finite): the product by 1/15
// cut to bf16 is that value or one step below it, and 15 s is exact in 32 bits.
__device__ __forceinline__ float kv4_scale(float span) {
  uint32_t bits = __float_as_uint(span * (1.f / 15.f)) & 0xffff0000u;
  if (15.f * __uint_as_float(bits) < span) bits += 0x10000u;
  if (15.f * __uint_as_float(bits) < span) bits += 0x10000u;
  return __uint_as_float(bits);
}

// Quantises keys and values into the cache.  One thread takes the 8 channels
// of one code word; 8 neighbouring lanes hold a group of 64 channels and find
// its lowest and highest value by shuffles.
//
// lowest = the minimum (a bf16 already), scale = the smallest bf16 with 15
// scale >= span, n = floor((x - lowest) / scale + 1/2).  The comparisons are
// exact: x - lowest is rounded down and the span up, and both are compared
// with (n + 1/2) scale and 15 scale, which 32 bits hold exactly; the quotient
// by the reciprocal only proposes n.  A group with an infinity, a NaN or a
// span beyond the largest float reads back as NaN.
template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const __grid_constant__ Kv4StoreParams p) {
  using L = Kv4Tile<D>;
  constexpr int kWords = D / 8;
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const bool live = id < p.n_items;
  const int word = static_cast<int>(id % kWords);
  const long long rest = live ? id / kWords : 0;
  const int h = static_cast<int>(rest % p.heads);
  const long long tk = rest / p.heads;
  const int value = static_cast<int>(tk & 1);
  const long long token = tk >> 1;
  const long long slot = live ? p.slots[token] : -1;
  const bool in = slot >= 0 && slot < p.n_slots;

  float x[8] = {};
  if (in) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p.x[value] + token * p.st[value] +
                                                      h * p.sh[value] + word * 8);
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(r[i]);
      x[2 * i + 1] = bf16_hi(r[i]);
    }
  }
  float lo = x[0], hi = x[0], odd = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    odd = fmaxf(odd, isfinite(x[i]) ? 0.f : 1.f);
  }
  lo = group8_min(lo);
  hi = group8_max(hi);
  odd = group8_max(odd);
  const float span = __fsub_ru(hi, lo);
  const bool bad = odd != 0.f || !isfinite(span);
  const float scale = bad || span == 0.f ? 0.f : kv4_scale(span);

  uint32_t code = 0;
  if (scale > 0.f) {
    // groups of tiny values are lifted (exactly) so that 1 / scale is finite
    const float lift = scale < 0x1p-60f ? 0x1p100f : 1.f;
    const float s = scale * lift, inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float dist = __fsub_rd(x[i], lo) * lift;
      float n = fminf(floorf(dist * inv + 0.5f), 15.f);
      if (dist < (n - 0.5f) * s) n -= 1.f;
      if (dist >= (n + 0.5f) * s) n += 1.f;
      code |= static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f)) << (4 * i);
    }
  }
  if (!in) return;
  uint8_t* tile = p.cache + kv4_tile_at<D>(p, slot, h);
  const int row = static_cast<int>(slot & 15);
  *reinterpret_cast<uint32_t*>(tile + (value ? L::kOffV : L::kOffK) + row * L::kRow +
                               4 * L::place(word, value != 0)) = code;
  if ((word & 7) == 0) {
    const uint32_t lo_bits = bad ? 0x7fc00000u : __float_as_uint(lo);
    *reinterpret_cast<uint32_t*>(tile + (value ? L::kOffVPar : L::kOffKPar) + row * L::kPar +
                                 (word >> 3) * 4) =
        (__float_as_uint(scale) >> 16) | (lo_bits & 0xffff0000u);
  }
}

// Reads slots back: lowest + scale n, one fused multiply-add (scale n has 12
// bits, so only its sum is rounded) and one rounding to bf16.  Slots outside
// the cache give zeros.
template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const __grid_constant__ Kv4StoreParams p) {
  using L = Kv4Tile<D>;
  constexpr int kWords = D / 8;
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (id >= p.n_items) return;
  const int word = static_cast<int>(id % kWords);
  const long long rest = id / kWords;
  const int h = static_cast<int>(rest % p.heads);
  const long long tk = rest / p.heads;
  const int value = static_cast<int>(tk & 1);
  const long long token = tk >> 1;
  const long long slot = p.slots[token];
  uint4 out = make_uint4(0, 0, 0, 0);
  if (slot >= 0 && slot < p.n_slots) {
    const uint8_t* tile = p.cache + kv4_tile_at<D>(p, slot, h);
    const int row = static_cast<int>(slot & 15);
    const uint32_t code = *reinterpret_cast<const uint32_t*>(
        tile + (value ? L::kOffV : L::kOffK) + row * L::kRow + 4 * L::place(word, value != 0));
    const uint32_t par = *reinterpret_cast<const uint32_t*>(
        tile + (value ? L::kOffVPar : L::kOffKPar) + row * L::kPar + (word >> 3) * 4);
    const float scale = bf16_lo(par), lo = bf16_hi(par);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = fmaf(static_cast<float>((code >> (4 * i)) & 15u), scale, lo);
    out = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
  }
  *reinterpret_cast<uint4*>(p.y[value] + token * p.st[value] + h * p.sh[value] + word * 8) = out;
}

// ---------------------------------------------------------------- the plan
// From each request's cached length and the length wanted: the pages it needs
// more (popped from a ring of free pages) or gives back (pushed onto it), the
// new tokens' positions and slots, and the prefix sums of their counts.
enum : int {
  kPlanPages = 1,    // not enough free pages
  kPlanTokens = 2,   // more new tokens than max_tokens
  kPlanLength = 4,   // a length below zero or above the table's width
  kPlanRing = 8,     // the ring's range is inconsistent
};

struct Kv4PlanParams {
  const int* old_len;
  const int* new_len;
  int* table;             // [requests, table stride]
  int* ring;              // free pages
  const long long* range; // head, tail: ring[head % P .. tail % P) are free
  int* out_len;
  long long* out_range;
  int* cu_tokens;
  long long* slots;
  int* positions;
  int* status;
  long long table_stride;
  int requests, width, page_size, ring_size, max_tokens;
};

struct PlanRow {
  int need, back;  // pages popped, pushed
  long long grow;  // new tokens
};

__device__ __forceinline__ PlanRow plan_row(int old_len, int new_len, int page_size,
                                            long long limit, bool* bad) {
  PlanRow r = {0, 0, 0};
  if (old_len < 0 || new_len < 0 || old_len > limit || new_len > limit) {
    *bad = true;
    return r;
  }
  const int held = static_cast<int>((static_cast<long long>(old_len) + page_size - 1) / page_size);
  const int want = static_cast<int>((static_cast<long long>(new_len) + page_size - 1) / page_size);
  r.need = max(0, want - held);
  r.back = max(0, held - want);
  r.grow = max(0, new_len - old_len);
  return r;
}

constexpr int kPlanThreads = 1024;

// Largest i in [0, n) with cu[i] <= x (cu[0] <= x, cu not decreasing).
__device__ __forceinline__ int plan_find(const int* cu, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One cluster; every CTA scans all requests (a block-wide scan of 1024 at a
// time, held in shared memory), and the CTAs share out the tokens and pages of
// the chunk, each located by a binary search.  Nothing is written that another
// CTA may still read: a popped or released page's ring and table places are
// disjoint, and lengths and range (which may be updated in place) are written
// after a cluster barrier.
__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const __grid_constant__ Kv4PlanParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int s_cu[kPlanThreads + 1], s_need[kPlanThreads + 1], s_back[kPlanThreads + 1];
  __shared__ int s_old[kPlanThreads], s_held[kPlanThreads];
  __shared__ long long w_grow[32];
  __shared__ int w_need[32], w_back[32];
  __shared__ long long t_grow, t_need, t_back;
  __shared__ int s_bad;

  const long long limit = static_cast<long long>(p.width) * p.page_size;
  const int chunks = (p.requests + kPlanThreads - 1) / kPlanThreads;
  const long long head = p.range[0], tail = p.range[1];
  if (tid == 0) {
    s_bad = 0;
    t_grow = t_need = t_back = 0;
  }
  __syncthreads();
  // totals
  {
    long long need = 0, back = 0, grow = 0;
    bool bad = false;
    for (int b = tid; b < p.requests; b += kPlanThreads) {
      const PlanRow r = plan_row(p.old_len[b], p.new_len[b], p.page_size, limit, &bad);
      need += r.need;
      back += r.back;
      grow += r.grow;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      need += __shfl_xor_sync(0xffffffffu, need, o);
      back += __shfl_xor_sync(0xffffffffu, back, o);
      grow += __shfl_xor_sync(0xffffffffu, grow, o);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      atomicAdd(reinterpret_cast<unsigned long long*>(&t_need), static_cast<unsigned long long>(need));
      atomicAdd(reinterpret_cast<unsigned long long*>(&t_back), static_cast<unsigned long long>(back));
      atomicAdd(reinterpret_cast<unsigned long long*>(&t_grow), static_cast<unsigned long long>(grow));
      if (bad) s_bad = 1;
    }
  }
  __syncthreads();
  const long long avail = tail - head;
  int status = s_bad ? kPlanLength : 0;
  if (t_need > avail) status |= kPlanPages;
  if (t_grow > p.max_tokens) status |= kPlanTokens;
  if (head < 0 || avail < 0 || avail > p.ring_size || avail + t_back > p.ring_size)
    status |= kPlanRing;
  const bool ok = status == 0;
  const int total = ok ? static_cast<int>(t_grow) : 0;

  int base_cu = 0, base_need = 0, base_back = 0;
  for (int c = 0; c < chunks; ++c) {
    const int b0 = c * kPlanThreads, cnt = min(kPlanThreads, p.requests - b0);
    int old_len = 0, new_len = 0;
    PlanRow r = {0, 0, 0};
    if (tid < cnt) {
      old_len = p.old_len[b0 + tid];
      new_len = p.new_len[b0 + tid];
      bool bad = false;
      if (ok) r = plan_row(old_len, new_len, p.page_size, limit, &bad);
    }
    // block-wide inclusive scan of the three counts
    int grow = static_cast<int>(r.grow), need = r.need, back = r.back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int g = __shfl_up_sync(0xffffffffu, grow, o), n = __shfl_up_sync(0xffffffffu, need, o),
                k = __shfl_up_sync(0xffffffffu, back, o);
      if (lane >= o) {
        grow += g;
        need += n;
        back += k;
      }
    }
    if (lane == 31) {
      w_grow[warp] = grow;
      w_need[warp] = need;
      w_back[warp] = back;
    }
    __syncthreads();
    if (warp == 0) {
      int g = static_cast<int>(w_grow[lane]), n = w_need[lane], k = w_back[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int g1 = __shfl_up_sync(0xffffffffu, g, o), n1 = __shfl_up_sync(0xffffffffu, n, o),
                  k1 = __shfl_up_sync(0xffffffffu, k, o);
        if (lane >= o) {
          g += g1;
          n += n1;
          k += k1;
        }
      }
      w_grow[lane] = g;
      w_need[lane] = n;
      w_back[lane] = k;
    }
    __syncthreads();
    if (warp > 0) {
      grow += static_cast<int>(w_grow[warp - 1]);
      need += w_need[warp - 1];
      back += w_back[warp - 1];
    }
    s_cu[tid + 1] = base_cu + grow;
    s_need[tid + 1] = base_need + need;
    s_back[tid + 1] = base_back + back;
    if (tid == 0) {
      s_cu[0] = base_cu;
      s_need[0] = base_need;
      s_back[0] = base_back;
    }
    const int held = static_cast<int>((static_cast<long long>(old_len) + p.page_size - 1) / p.page_size);
    s_old[tid] = old_len;
    s_held[tid] = held;
    __syncthreads();
    const int cu_end = s_cu[cnt], need_end = s_need[cnt], back_end = s_back[cnt];
    const int step = ranks * kPlanThreads, me = rank * kPlanThreads + tid;
    if (rank == 0 && tid < cnt) p.cu_tokens[b0 + tid] = s_cu[tid];
    for (int t = base_cu + me; t < cu_end; t += step) {
      const int i = plan_find(s_cu, cnt, t);
      const int pos = s_old[i] + (t - s_cu[i]);
      const int page_i = pos / p.page_size;
      const int page = page_i < s_held[i]
                           ? p.table[(b0 + i) * p.table_stride + page_i]
                           : p.ring[(head + s_need[i] + (page_i - s_held[i])) % p.ring_size];
      p.positions[t] = pos;
      p.slots[t] = static_cast<long long>(page) * p.page_size + (pos - page_i * p.page_size);
    }
    for (int k = base_need + me; k < need_end; k += step) {
      const int i = plan_find(s_need, cnt, k);
      p.table[(b0 + i) * p.table_stride + s_held[i] + (k - s_need[i])] =
          p.ring[(head + k) % p.ring_size];
    }
    for (int k = base_back + me; k < back_end; k += step) {
      const int i = plan_find(s_back, cnt, k);
      const int rows = s_back[i + 1] - s_back[i];
      p.ring[(tail + k) % p.ring_size] =
          p.table[(b0 + i) * p.table_stride + s_held[i] - rows + (k - s_back[i])];
    }
    base_cu = cu_end;
    base_need = need_end;
    base_back = back_end;
    __syncthreads();
  }
  for (int t = total + rank * kPlanThreads + tid; t < p.max_tokens; t += ranks * kPlanThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  cluster.sync();  // every CTA has read lengths and range
  if (rank == 0) {
    for (int b = tid; b < p.requests; b += kPlanThreads)
      p.out_len[b] = ok ? p.new_len[b] : p.old_len[b];
    if (tid == 0) {
      p.cu_tokens[p.requests] = total;
      p.out_range[0] = head + (ok ? t_need : 0);
      p.out_range[1] = tail + (ok ? t_back : 0);
      *p.status = status;
    }
  }
}

}  // namespace fa
