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
  long long tokens;
  int heads, page_tiles, block_tokens;
  FastDiv by_page_tiles, by_lanes;  // tiles of a page, `lanes`
  int lanes, side_by_side;  // threads that share a token, tokens walked side by side
};

// A block of append or gather takes up to kStoreTokens tokens.  A thread keeps
// two adjacent code words (16 channels of a K or V head) and walks the block's
// tokens with them, two at a time so that their loads are in flight together;
// where a token has fewer words than the block threads, several tokens are
// walked side by side.  The slots' places in the cache are worked out once, in shared memory.
constexpr int kStoreThreads = 256;
constexpr int kStoreTokens = 16;
constexpr int kStoreBatch = 2;

struct StorePlaces {
  long long tile[kStoreTokens];  // byte offset of head 0's tile, -1: outside
  int row[kStoreTokens];
};
template <int D>
__device__ __forceinline__ int store_places(const Kv4StoreParams& p, long long token0,
                                            StorePlaces& sp) {
  const int n = static_cast<int>(min(static_cast<long long>(p.block_tokens), p.tokens - token0));
  if (static_cast<int>(threadIdx.x) < n) {
    const long long slot = p.slots[token0 + threadIdx.x];
    long long at = -1;
    if (slot >= 0 && slot < p.n_slots) {
      const uint32_t tile = static_cast<uint32_t>(slot >> 4);  // below 2^31
      const uint32_t page = p.by_page_tiles(tile);
      at = (static_cast<long long>(tile) + static_cast<long long>(page) * (p.heads - 1) * p.page_tiles) *
           Kv4Tile<D>::kBytes;
    }
    sp.tile[threadIdx.x] = at;
    sp.row[threadIdx.x] = static_cast<int>(slot & 15);
  }
  __syncthreads();
  return n;
}
// The cache's bytes; all that a thread of append or gather touches of row `row`
// at `first` lies inside.
template <int D>
__device__ __forceinline__ bool store_inside(const Kv4StoreParams& p, long long first, int next, int par) {
  const long long bytes = (p.n_slots >> 4) * p.heads * Kv4Tile<D>::kBytes;
  return dbg_access(first >= 0 && first + next + 4 <= bytes && first + par >= 0 && first + par + 4 <= bytes,
                    kErrKv4);
}

// The pair of words a thread keeps: where it lies in x and in a tile.
template <int D>
struct StoreWords {
  int value, h, word, next;  // next: bytes from the first word to the second
  long long in_cache;        // of row 0
  __device__ __forceinline__ StoreWords(const Kv4StoreParams& p, int i) {
    using L = Kv4Tile<D>;
    const int half = p.heads * (D / 16);
    value = i >= half;
    const int of_kind = i - (value ? half : 0);
    h = of_kind / (D / 16);
    word = of_kind % (D / 16) * 2;
    next = value ? D / 16 : D / 8;
    in_cache = static_cast<long long>(h) * p.page_tiles * L::kBytes +
               (value ? L::kOffV : L::kOffK) + 4 * L::place(word, value != 0);
  }
  // of a row's parameters, from the row's first word
  __device__ __forceinline__ int par(int row) const {
    using L = Kv4Tile<D>;
    return 16 * L::kRow - 4 * L::place(word, value != 0) - row * (L::kRow - L::kPar) + (word >> 3) * 4;
  }
};

// Lower and higher of two pairs of bf16; a NaN wins.
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Smallest bf16 s with 15 s >= span (span > 0, finite): the product by 1/15
// cut to bf16 is that value or one step below it, and 15 s is exact in 32 bits.
__device__ __forceinline__ float kv4_scale(float span) {
  uint32_t bits = __float_as_uint(span * (1.f / 15.f)) & 0xffff0000u;
  if (15.f * __uint_as_float(bits) < span) bits += 0x10000u;
  if (15.f * __uint_as_float(bits) < span) bits += 0x10000u;
  return __uint_as_float(bits);
}

// Quantises keys and values into the cache: 4 neighbouring lanes hold a group
// of 64 channels and find its lowest and highest value by shuffles.
//
// lowest = the minimum (a bf16 already), scale = the smallest bf16 with 15
// scale >= span, n = floor((x - lowest) / scale + 1/2).  The comparisons are
// exact.  With dist = x - lowest rounded down and a reciprocal a little too
// large, n0 = dist * reciprocal to the nearest is n or, once in 10^5, n + 1; it is
// n + 1 just where dist - n0 scale, rounded down, is below -scale / 2: every
// border (n0 - 1/2) scale is a 32-bit number, and rounding down moves no number
// across it.  Only the least of these differences is looked at, and a thread that
// finds one too low corrects its codes.  Four codes are packed as one exact
// 32-bit float.
// A group with an infinity, a NaN or a span beyond the largest float reads back
// as NaN.
//
// Bound by instructions as much as by memory: 17 an element with the reduction and
// the walk.  16384 tokens of 8 heads, d = 128 (86 MB): 28.1 us with cold caches,
// 3.1 TB/s, issue slots 68 % taken; 32 tokens and their gather 4.7 us.
template <int D>
__device__ __forceinline__ void append_words(const Kv4StoreParams& p, const StoreWords<D>& w,
                                             long long tile, int row, const uint32_t (&r)[8]) {
  using L = Kv4Tile<D>;
  // (lowest, -highest) of the group as a pair: one shuffle serves both
  uint32_t least = r[0], most = r[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    least = min_nan_bf16x2(least, r[i]);
    most = max_nan_bf16x2(most, r[i]);
  }
  least = min_nan_bf16x2(least, __byte_perm(least, 0, 0x1032));
  most = max_nan_bf16x2(most, __byte_perm(most, 0, 0x1032)) ^ 0x80008000u;
  uint32_t ends = __byte_perm(least, most, 0x5410);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1)
    ends = min_nan_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  float lo = bf16_lo(ends);
  const float span = __fsub_ru(-bf16_hi(ends), lo);
  const bool bad = !isfinite(span);
  float scale = bad || span == 0.f ? 0.f : kv4_scale(span);
  const uint32_t par = (__float_as_uint(scale) >> 16) |
                       ((bad ? 0x7fc00000u : __float_as_uint(lo)) & 0xffff0000u);

  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(r[i]);
    x[2 * i + 1] = bf16_hi(r[i]);
  }
  if (scale < 0x1p-60f && scale > 0.f) {
    // a group of tiny values is lifted (exactly) so that 1 / scale is finite
    scale *= 0x1p100f;
    lo *= 0x1p100f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= 0x1p100f;
  }
  // (scale 0: the products by a zero reciprocal leave every code 0)
  const float inv = scale > 0.f ? __fdividef(1.f + 0x1p-20f, scale) : 0.f;
  const float half = 0.5f * scale;
  float four[4] = {0.f, 0.f, 0.f, 0.f}, least_left = 0.f;
#pragma unroll
  for (int i = 15; i >= 0; --i) {
    const float dist = __fsub_rd(x[i], lo);
    const float n = fmaf(dist, inv, 0x1p23f) - 0x1p23f;  // to the nearest whole number
    least_left = fminf(least_left, __fmaf_rd(-n, scale, dist));
    four[i >> 2] = fmaf(four[i >> 2], 16.f, n);
  }
  if (least_left < -half) {
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      const float dist = __fsub_rd(x[i], lo);
      const float n = fmaf(dist, inv, 0x1p23f) - 0x1p23f;
      if (__fmaf_rd(-n, scale, dist) < -half)
        four[i >> 2] -= static_cast<float>(1 << (4 * (i & 3)));
    }
  }
  // 2^23 + a whole number below 2^16: its bits are the number's
  uint32_t code[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    code[i] = bad ? 0u
                  : __byte_perm(__float_as_uint(four[2 * i] + 0x1p23f),
                                __float_as_uint(four[2 * i + 1] + 0x1p23f), 0x5410);
  if (tile < 0) return;
  const long long first = tile + w.in_cache + row * L::kRow;
  if (!store_inside<D>(p, first, w.next, w.par(row))) return;
  uint8_t* at = p.cache + first;
  *reinterpret_cast<uint32_t*>(at) = code[0];
  *reinterpret_cast<uint32_t*>(at + w.next) = code[1];
  if ((w.word & 7) == 0) *reinterpret_cast<uint32_t*>(at + w.par(row)) = par;
}

template <int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const __grid_constant__ Kv4StoreParams p) {
  __shared__ StorePlaces sp;
  const long long token0 = static_cast<long long>(blockIdx.x) * p.block_tokens;
  const int n = store_places<D>(p, token0, sp);
  // every lane runs every loop (the shuffles need the whole warp)
  const int total = 2 * p.heads * (D / 16), side = p.by_lanes(threadIdx.x);
  for (int i0 = 0; i0 < total; i0 += p.lanes) {
    const int i = i0 + static_cast<int>(threadIdx.x) - side * p.lanes;
    const bool live = side < p.side_by_side && i < total;
    const StoreWords<D> w(p, live ? i : 0);
    const __nv_bfloat16* x = p.x[w.value] + w.h * p.sh[w.value] + w.word * 8;
    for (int t = 0; t < n; t += kStoreBatch * p.side_by_side) {
      uint32_t raw[kStoreBatch][8];
      long long tile[kStoreBatch];
#pragma unroll
      for (int u = 0; u < kStoreBatch; ++u) {
        const int tk = t + side + u * p.side_by_side;
        tile[u] = live && tk < n ? sp.tile[tk] : -1;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (tile[u] >= 0) {
          const uint4* from = reinterpret_cast<const uint4*>(x + (token0 + tk) * p.st[w.value]);
          a = __ldg(from);
          b = __ldg(from + 1);
        }
        raw[u][0] = a.x, raw[u][1] = a.y, raw[u][2] = a.z, raw[u][3] = a.w;
        raw[u][4] = b.x, raw[u][5] = b.y, raw[u][6] = b.z, raw[u][7] = b.w;
      }
#pragma unroll
      for (int u = 0; u < kStoreBatch; ++u) {
        if (t + u * p.side_by_side >= n) break;
        append_words<D>(p, w, tile[u], tile[u] >= 0 ? sp.row[t + side + u * p.side_by_side] : 0, raw[u]);
      }
    }
  }
}

// Reads slots back: lowest + scale n, one fused multiply-add (scale n has 12
// bits, so only its sum is rounded) and one rounding to bf16.  Slots outside
// the cache give zeros.
// Two tokens of three loads in flight a thread, 10 instructions an element (issue
// slots 55 % taken): the same 16384 tokens (86 MB) 21.4 us with cold caches,
// 4.0 TB/s; both together 47.4 us.
template <int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_gather_kernel(const __grid_constant__ Kv4StoreParams p) {
  using L = Kv4Tile<D>;
  __shared__ StorePlaces sp;
  const long long token0 = static_cast<long long>(blockIdx.x) * p.block_tokens;
  const int n = store_places<D>(p, token0, sp);
  const int side = p.by_lanes(threadIdx.x);
  if (side >= p.side_by_side) return;
  for (int i = threadIdx.x - side * p.lanes; i < 2 * p.heads * (D / 16); i += p.lanes) {
    const StoreWords<D> w(p, i);
    __nv_bfloat16* y = p.y[w.value] + w.h * p.sh[w.value] + w.word * 8;
    for (int t = side; t < n; t += kStoreBatch * p.side_by_side) {
      uint32_t code[kStoreBatch][2] = {}, par[kStoreBatch] = {};
#pragma unroll
      for (int u = 0; u < kStoreBatch; ++u) {
        const int tk = t + u * p.side_by_side;
        if (tk >= n || sp.tile[tk] < 0) continue;
        const long long first = sp.tile[tk] + w.in_cache + sp.row[tk] * L::kRow;
        if (!store_inside<D>(p, first, w.next, w.par(sp.row[tk]))) continue;
        const uint8_t* at = p.cache + first;
        code[u][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
        code[u][1] = __ldg(reinterpret_cast<const uint32_t*>(at + w.next));
        par[u] = __ldg(reinterpret_cast<const uint32_t*>(at + w.par(sp.row[tk])));
      }
#pragma unroll
      for (int u = 0; u < kStoreBatch; ++u) {
        const int tk = t + u * p.side_by_side;
        if (tk >= n) continue;
        const float scale = bf16_lo(par[u]), lo = bf16_hi(par[u]);
        uint32_t out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // 2^23 + n, from n's bits
            const uint32_t n_bits = (code[u][k >> 2] >> (8 * (k & 3) + 4 * e)) & 15u;
            x[e] = fmaf(__uint_as_float(n_bits | 0x4b000000u) - 0x1p23f, scale, lo);
          }
          out[k] = pack_bf16x2(x[0], x[1]);
        }
        uint4* to = reinterpret_cast<uint4*>(y + (token0 + tk) * p.st[w.value]);
        to[0] = make_uint4(out[0], out[1], out[2], out[3]);
        to[1] = make_uint4(out[4], out[5], out[6], out[7]);
      }
    }
  }
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
  FastDiv by_page;
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
constexpr int kPlanBatch = 4;  // tokens a thread looks up together

// Largest i in [0, n) with cu[i] <= x (cu[0] <= x, cu not decreasing, n at most
// 1024); without branches, so that several searches interleave.
__device__ __forceinline__ int plan_find(const int* cu, int n, int x) {
  int i = 0;
#pragma unroll
  for (int step = kPlanThreads / 2; step > 0; step >>= 1)
    if (i + step < n && cu[i + step] <= x) i += step;
  return i;
}

// One cluster; every CTA scans all requests (1024 at a time, their prefix sums
// in shared memory), and the CTAs share out the tokens and pages, each located
// by a binary search.  Nothing is written that another CTA may still read: a
// popped or released page's ring and table places are disjoint, and lengths and
// range (which may be updated in place) are written after a cluster barrier.
//
// Bound by latency: the loads of lengths, the scan, and the loads of pages.
// 8 requests 5.0 us, 1023 requests with 64 prompts (0.46 MB) 11.9 us.
__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const __grid_constant__ Kv4PlanParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int s_cu[kPlanThreads + 1], s_need[kPlanThreads + 1], s_back[kPlanThreads + 1];
  __shared__ int s_old[kPlanThreads], s_held[kPlanThreads];
  __shared__ int w_sum[3][32];
  __shared__ unsigned long long t_grow, t_need, t_back;
  __shared__ int s_bad, s_head, s_tail;

  const long long limit = static_cast<long long>(p.width) * p.page_size;
  const int chunks = (p.requests + kPlanThreads - 1) / kPlanThreads;
  const long long head = p.range[0], tail = p.range[1];
  if (tid == 0) {
    s_bad = 0;
    t_grow = t_need = t_back = 0;
  }
  __syncthreads();
  // totals; the first 1024 requests stay in registers
  int old_len = 0, new_len = 0;
  PlanRow row = {0, 0, 0};
  {
    long long grow = 0;
    int need = 0, back = 0;
    bool bad = false;
    for (int c = chunks - 1; c >= 0; --c) {
      const int b = c * kPlanThreads + tid;
      row = {0, 0, 0};
      if (b < p.requests) {
        old_len = p.old_len[b];
        new_len = p.new_len[b];
        row = plan_row(old_len, new_len, p.page_size, limit, &bad);
      }
      need += row.need;
      back += row.back;
      grow += row.grow;
    }
    need = __reduce_add_sync(0xffffffffu, need);
    back = __reduce_add_sync(0xffffffffu, back);
#pragma unroll
    for (int o = 16; o; o >>= 1) grow += __shfl_xor_sync(0xffffffffu, grow, o);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (need) atomicAdd(&t_need, static_cast<unsigned long long>(need));
      if (back) atomicAdd(&t_back, static_cast<unsigned long long>(back));
      if (grow) atomicAdd(&t_grow, static_cast<unsigned long long>(grow));
      if (bad) s_bad = 1;
    }
    if (tid == kPlanThreads - 1) {  // (a warp with little to add)
      s_head = head >= 0 ? static_cast<int>(head % p.ring_size) : 0;
      s_tail = tail >= 0 ? static_cast<int>(tail % p.ring_size) : 0;
    }
  }
  __syncthreads();
  const long long avail = tail - head, all_need = static_cast<long long>(t_need),
                  all_back = static_cast<long long>(t_back), all_grow = static_cast<long long>(t_grow);
  int status = s_bad ? kPlanLength : 0;
  if (all_need > avail) status |= kPlanPages;
  if (all_grow > p.max_tokens) status |= kPlanTokens;
  if (head < 0 || avail < 0 || avail > p.ring_size || avail + all_back > p.ring_size)
    status |= kPlanRing;
  const bool ok = status == 0;
  const int total = ok ? static_cast<int>(all_grow) : 0;
  // place i <= ring_size behind a start
  auto ring_at = [&](int start, int i) {
    const int at = start + i;
    return p.ring + (at >= p.ring_size ? at - p.ring_size : at);
  };

  int base_cu = 0, base_need = 0, base_back = 0;
  for (int c = 0; c < chunks; ++c) {
    const int b0 = c * kPlanThreads, cnt = min(kPlanThreads, p.requests - b0);
    if (c > 0) {
      row = {0, 0, 0};
      old_len = 0;
      if (tid < cnt) {
        bool bad = false;
        old_len = p.old_len[b0 + tid];
        row = plan_row(old_len, p.new_len[b0 + tid], p.page_size, limit, &bad);
      }
    }
    // block-wide inclusive scan of the three counts
    int v[3] = {ok ? static_cast<int>(row.grow) : 0, ok ? row.need : 0, ok ? row.back : 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int x = __shfl_up_sync(0xffffffffu, v[k], o);
        if (lane >= o) v[k] += x;
      }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 3; ++k) w_sum[k][warp] = v[k];
    }
    __syncthreads();
    const int base[3] = {base_cu, base_need, base_back};
#pragma unroll
    for (int k = 0; k < 3; ++k)  // the warps before this one
      v[k] += base[k] + __reduce_add_sync(0xffffffffu, lane < warp ? w_sum[k][lane] : 0);
    s_cu[tid + 1] = v[0];
    s_need[tid + 1] = v[1];
    s_back[tid + 1] = v[2];
    if (tid == 0) {
      s_cu[0] = base_cu;
      s_need[0] = base_need;
      s_back[0] = base_back;
    }
    s_old[tid] = old_len;
    s_held[tid] = static_cast<int>(p.by_page(static_cast<uint32_t>(max(old_len, 0)) + p.page_size - 1));
    __syncthreads();
    const int cu_end = s_cu[cnt], need_end = s_need[cnt], back_end = s_back[cnt];
    const int step = ranks * kPlanThreads, me = rank * kPlanThreads + tid;
    if (rank == 0 && tid < cnt) p.cu_tokens[b0 + tid] = s_cu[tid];
    for (int t0 = base_cu + me; t0 < cu_end; t0 += kPlanBatch * step) {
      int i[kPlanBatch], pos[kPlanBatch], in_page[kPlanBatch], page[kPlanBatch];
#pragma unroll
      for (int u = 0; u < kPlanBatch; ++u) i[u] = plan_find(s_cu, cnt, min(t0 + u * step, cu_end - 1));
#pragma unroll
      for (int u = 0; u < kPlanBatch; ++u) {
        if (t0 + u * step >= cu_end) continue;
        pos[u] = s_old[i[u]] + (t0 + u * step - s_cu[i[u]]);
        const int n = static_cast<int>(p.by_page(pos[u])), held = s_held[i[u]];
        in_page[u] = pos[u] - n * p.page_size;
        page[u] = 0;
        if (!dbg_access(n >= 0 && n < p.width && t0 + u * step < p.max_tokens &&
                            (n < held || (n - held >= 0 && s_need[i[u]] + n - held < p.ring_size)),
                        kErrKv4))
          continue;
        page[u] = n < held ? p.table[(b0 + i[u]) * p.table_stride + n]
                           : *ring_at(s_head, s_need[i[u]] + n - held);
      }
#pragma unroll
      for (int u = 0; u < kPlanBatch; ++u) {
        if (t0 + u * step >= cu_end) continue;
        p.positions[t0 + u * step] = pos[u];
        p.slots[t0 + u * step] = static_cast<long long>(page[u]) * p.page_size + in_page[u];
      }
    }
    for (int k = base_need + me; k < need_end; k += step) {
      const int i = plan_find(s_need, cnt, k);
      if (!dbg_access(k < p.ring_size && s_held[i] + (k - s_need[i]) < p.width, kErrKv4)) continue;
      p.table[(b0 + i) * p.table_stride + s_held[i] + (k - s_need[i])] = *ring_at(s_head, k);
    }
    for (int k = base_back + me; k < back_end; k += step) {
      const int i = plan_find(s_back, cnt, k);
      const int rows = s_back[i + 1] - s_back[i];
      if (!dbg_access(k < p.ring_size && s_held[i] - rows >= 0 && s_held[i] - rows + (k - s_back[i]) < p.width,
                      kErrKv4))
        continue;
      *ring_at(s_tail, k) = p.table[(b0 + i) * p.table_stride + s_held[i] - rows + (k - s_back[i])];
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
  if (ranks > 1) cluster.sync();  // every CTA has read lengths and range
  if (rank == 0) {
    for (int b = tid; b < p.requests; b += kPlanThreads)
      p.out_len[b] = ok ? p.new_len[b] : p.old_len[b];
    if (tid == 0) {
      p.cu_tokens[p.requests] = total;
      p.out_range[0] = head + (ok ? all_need : 0);
      p.out_range[1] = tail + (ok ? all_back : 0);
      *p.status = status;
    }
  }
}

}  // namespace fa
