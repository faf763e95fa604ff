// kv4_attend.cuh -- attention of packed queries over the paged 4-bit cache.
//
//   O_i = sum_j softmax_j(scale q_i . K_j) V_j over the keys row i sees,
//   LSE_i = ln sum_j exp(scale q_i . K_j),
// where K_j and V_j are the values the cache's codes stand for.  With K_j =
// lowest + s n per group of 64 channels,
//   q . K_j = sum_groups s (q . n) + lowest (sum of q),
// so the matrix instructions multiply the codes themselves, and scale and
// lowest act on the 64-channel sums; for V, P s goes into the matrix
// instructions and P lowest is summed beside them.
//
// Codes enter as fp16 subnormal numbers, exactly.  q enters as fp16 after an
// exact scaling of each row by a power of two (its largest element near fp16's
// largest), so a bf16 or fp16 q keeps all its bits down to 2^-24 of the row's
// largest.  P s enters as fp16 times a power of two of its row and 64-channel
// group, by the largest P s that the row has met: 11 bits, against the 8 of a
// bf16 P, and none lost to a large token without weight, to another group or to
// a token that the row does not see.  Scores, softmax statistics and O are fp32.
//
// Rows: the queries of a request times the heads that share a kv head, in
// tiles of 8 NT.  Transposed products (S^T = K q^T, O^T = V^T P^T) put tokens
// and channels on the 16-row side of m16n8k16, so a single token of a group of
// up to 8 heads wastes little.
//
// Bound: at long contexts the memory, as far as the instructions let it (261 a
// 16-key tile of d = 128, issue slots 56 % taken): 3 requests of 100000 to 131072
// keys, H=32/8 d=128, 88 us, 4.4 TB/s (more keys take longer by 5.6 TB/s);
// 64 requests of 200 to 8192 keys 76 us, 4.1 TB/s, the rest being what a job and
// the join of its pieces cost; with more row tiles the latency of a tile, as few
// warps fit: 32 requests of 4096 keys with 5 drafted tokens 80 us (151 MB), 24 of
// up to 4096 with 5, H=16/4 d=64, 23.6 us; one request of 1000 keys 9.1 us, two
// launches and the latency of one tile.  The units of P s a row and group cost
// nothing that shows with one row tile, 2 to 4 % with two and three, 13 % with four
// (spilled registers), against one unit a warp.
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
  long long part_floats;  // room for them
  struct Kv4Cut* cuts;    // of kv4_chunk.cuh: one per CTA
  long long q_st, q_sh, o_st, o_sh;  // strides in elements
  long long table_stride;
  int requests, heads, kv_heads, group, tokens, pages, page_size, width;
  int lead;               // units of a job before those of its keys
  FastDiv page_tiles, by_group;  // 16-key tiles of a page, heads of a group
  float scale_log2;
  int causal, is_half;
  uint64_t limit_ns;      // of a bounded wait
};

constexpr int kKv4Warps = 4;

// ------------------------------------------------------------ the work's order
// Jobs: (request, tile of ROWS rows, kv head).  A job's units are first p.lead
// that stand for what it costs to begin and end one (q, the first keys'
// latency, the output), then one for each UNIT keys that its last row sees (in
// all at least one, so that a row that sees none gets its zeros).  Each CTA takes
// an equal, contiguous range of the units, and so an equal share of the time
// whatever the lengths are.  A job that a CTA's range cuts is left as partial
// results, which the combine kernel joins.
struct Kv4Req {
  int first, n, len, rows;  // first query, queries, keys, rows (queries * group)
};
__device__ __forceinline__ Kv4Req kv4_request(const Kv4AttendParams& p, int b) {
  Kv4Req r;
  r.first = min(max(p.cu_tokens[b], 0), p.tokens);
  r.n = max(min(p.cu_tokens[b + 1], p.tokens) - r.first, 0);
  r.len = max(0, static_cast<int>(min(static_cast<long long>(p.lengths[b]),
                                      static_cast<long long>(p.width) * p.page_size)));
  r.rows = r.n * p.group;
  return r;
}
// Keys that row `row` of a request sees.
__device__ __forceinline__ int kv4_sees(const Kv4AttendParams& p, const Kv4Req& r, int row) {
  return p.causal ? min(max(r.len - r.n + static_cast<int>(p.by_group(row)) + 1, 0), r.len) : r.len;
}
// Units of a row tile for one head.
template <int ROWS, int UNIT>
__device__ __forceinline__ int kv4_tile_units(const Kv4AttendParams& p, const Kv4Req& r, int tile) {
  const int last = min((tile + 1) * ROWS, r.rows) - 1;
  return max(1, p.lead + (kv4_sees(p, r, last) + UNIT - 1) / UNIT);
}
template <int ROWS, int UNIT>
__device__ __forceinline__ long long kv4_units(const Kv4AttendParams& p, const Kv4Req& r) {
  long long sum = 0;
  for (int t = 0; t * ROWS < r.rows; ++t) sum += kv4_tile_units<ROWS, UNIT>(p, r, t);
  return sum * p.kv_heads;
}

// a / b for non-negative numbers, in 32 bits where they fit (nearly always).
__device__ __forceinline__ long long kv4_div(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

struct Kv4Share {  // of the units: CTA c of n starts at each * c + min(c, rest)
  long long each;
  int rest;
  __device__ __forceinline__ Kv4Share(long long total, int n) {
    each = kv4_div(total, n);
    rest = static_cast<int>(total - each * n);
  }
  __device__ __forceinline__ long long start(int c) const { return each * c + min(c, rest); }
};

struct Kv4Shared {
  long long warp_sum[32];
  long long total, found_excl;
  int found_b;
};

// Block-wide (kWarps warps): the total number of units, and the request that
// holds the first unit of CTA `cta` of `ctas` together with the units before it
// (-1 if there is none).  Requests up to the number of threads are summed once,
// more are walked twice.
template <int ROWS, int UNIT, int kWarps>
__device__ __forceinline__ void kv4_locate(const Kv4AttendParams& p, Kv4Shared& sh, int cta,
                                           int ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kThreads = kWarps * 32;
  const int chunks = (p.requests + kThreads - 1) / kThreads;
  long long total = 0, mine = 0, incl = 0;
  if (tid == 0) sh.found_b = -1;
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c * kThreads + tid;
      if (pass == 0 || chunks > 1) {
        mine = b < p.requests ? kv4_units<ROWS, UNIT>(p, kv4_request(p, b)) : 0;
        incl = mine;
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
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) incl += sh.warp_sum[w];
          all += sh.warp_sum[w];
        }
        if (pass == 0) total += all;
        else incl += base;
        base += all;
      }
      if (pass == 1) {
        const long long u = Kv4Share(total, ctas).start(cta);
        if (u >= incl - mine && u < incl) {
          sh.found_b = b;
          sh.found_excl = incl - mine;
        }
      }
    }
  }
  if (tid == 0) sh.total = total;
  __syncthreads();
}

// Where unit u lies, walked forwards from the start of a request.
template <int ROWS, int UNIT>
struct Kv4Walk {
  int b, tile, units;  // request, row tile, units of the tile for one head
  long long excl;      // units before the tile
  Kv4Req rq;
  int h, c0;           // of unit u: kv head, unit inside (tile, head)
  __device__ __forceinline__ Kv4Walk(const Kv4AttendParams& p, int b_, long long excl_)
      : b(b_), tile(0), excl(excl_), rq(kv4_request(p, b_)) {
    units = kv4_tile_units<ROWS, UNIT>(p, rq, 0);
  }
  // u at or behind the last one, and inside the work
  __device__ __forceinline__ void to(const Kv4AttendParams& p, long long u) {
    while (u - excl >= static_cast<long long>(units) * p.kv_heads) {
      excl += static_cast<long long>(units) * p.kv_heads;
      if (++tile * ROWS >= rq.rows) {
        do rq = kv4_request(p, ++b);
        while (rq.rows == 0);
        tile = 0;
      }
      units = kv4_tile_units<ROWS, UNIT>(p, rq, tile);
    }
    h = static_cast<int>(kv4_div(u - excl, units));
    c0 = static_cast<int>(u - excl - static_cast<long long>(h) * units);
  }
  __device__ __forceinline__ long long job_start() const {
    return excl + static_cast<long long>(h) * units;
  }
};

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

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Codes 0..7 of a word as four fp16 pairs: (0, 4), (1, 5), (2, 6), (3, 7).  Four
// bits at the bottom of an fp16 are the subnormal number n 2^-24, four bits
// higher 16 n 2^-24: exact operands of the matrix instructions without any
// conversion (adding 1024 under the bits and taking it off again costs another
// instruction a pair).  The factor 16 is taken out of q beforehand and of O
// afterwards, 2^24 out of the scores' factor and of O.
// flip: all ones for 15 - n in place of n (no further instruction), else 0.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4], uint32_t flip = 0) {
  const uint32_t w8 = w >> 8;
  h[0] = (w ^ flip) & 0x000f000fu;
  h[1] = (w ^ flip) & 0x00f000f0u;
  h[2] = (w8 ^ flip) & 0x000f000fu;
  h[3] = (w8 ^ flip) & 0x00f000f0u;
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
  static constexpr int kFast = NT <= 2 ? 2 : 1;  // tiles taken together where all rows see them
  // CTAs on an SM, by registers (d = 64, drafted tokens: 3 against 2 23.6 vs 26.3 us)
  static constexpr int kCtas = NT == 1 ? (D == 64 ? 4 : 3) : D == 64 ? 3 : 2;
  // tiles of a block, one stage of a warp's ring: 4, so that the waits, look-ups
  // and copies of a block weigh little (2: 258 -> 284 instructions a tile, 83 ->
  // 98 us for 64 requests of 200 to 8192 keys, H=32/8 d=128)
  static constexpr int kTiles = 4;
  static constexpr int kUnit = 16 * kTiles * kKv4Warps;  // keys of a work unit
  static constexpr int kBlock = kTiles * Kv4Tile<D>::kBytes;
  static constexpr int kStages = 2;
  static constexpr int kRing = kKv4Warps * kStages * kBlock;
  static constexpr int kPitch = D + 4;  // floats of a row in the merge buffer
  // the merge buffer lies over the ring, which is empty by then
  static constexpr int kOffMl = kKv4Warps * kRows * kPitch * 4;
  static constexpr int kMerge = kOffMl + 2 * kKv4Warps * kRows * 4;
  static constexpr int kOffQ = kRing > kMerge ? kRing : kMerge;
  // more than two row tiles share their q fragments through shared memory
  static constexpr int kOffQs = kOffQ + (NT > 2 ? NT * (D / 32) * 32 * 16 : 0);
  static constexpr int kOffRs = kOffQs + (NT > 2 ? NT * (D / 64) * 8 * 4 : 0);  // sums of q, factors
  static constexpr int kOffBar = kOffRs + (NT > 2 ? kRows * 4 : 0);
  static constexpr int kBytes = kOffBar + kKv4Warps * kStages * 8;
  static constexpr int kPartFloats = kRows * (D + 2);  // O, then m and l
  static_assert(kOffBar % 8 == 0 && kCtas * (kBytes + 256 + 1024) <= 233472, "shared memory");
};

template <int N>
__device__ __forceinline__ void load_floats(const float* at, float (&v)[N]) {
  if (N == 4) {
    const float4 x = *reinterpret_cast<const float4*>(at);
    v[0] = x.x, v[1] = x.y, v[2 % N] = x.z, v[3 % N] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(at);
    v[0] = x.x, v[1] = x.y;
  }
}
template <int N>
__device__ __forceinline__ void store_floats(float* at, const float (&v)[N]) {
  if (N == 4)
    *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2 % N], v[3 % N]);
  else
    *reinterpret_cast<float2*>(at) = make_float2(v[0], v[1]);
}

// A finished row of a request (query row / group, head h group + row % group)
// by a whole warp, lane's channels D / 32 lane and on; o is not yet over l.
template <int D>
__device__ __forceinline__ void kv4_store_row(const Kv4AttendParams& p, const Kv4Req& rq, int h,
                                              int row, int lane, const float (&o)[D / 32], float m,
                                              float l) {
  const int i = p.by_group(row), tok = rq.first + i, head = h * p.group + row - i * p.group;
  if (!dbg_access(row >= 0 && row < rq.rows && tok < p.tokens && head < p.heads, kErrKv4)) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long long at = tok * p.o_st + head * p.o_sh + lane * (D / 32);
  uint32_t w[D / 64];
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
    w[k] = p.is_half ? pack_f16x2(o[2 * k] * inv, o[2 * k + 1] * inv)
                     : pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv);
  uint16_t* to = static_cast<uint16_t*>(p.o) + at;
  if (D == 128)
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[D / 64 - 1]);
  else
    *reinterpret_cast<uint32_t*>(to) = w[0];
  if (lane == 0)
    p.lse[static_cast<long long>(tok) * p.heads + head] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Row r of a tile (of `rows` real ones) for the lane's fragments: q as fp16
// times a power of two that brings the row's largest element to [2^14, 2^15)
// (the power itself kept within 2^+-100), every other channel pair a sixteenth
// of that; the sums of q over the groups beside scores in units of 2^-24; the
// factor from those scores to base-2 exponents.
template <int D>
__device__ __forceinline__ void kv4_rows(const Kv4AttendParams& p, const Kv4Req& rq, int h,
                                         int row0, int r, int rows, uint32_t (&f)[D / 32][4],
                                         float (&sum)[D / 64], float& factor) {
  const int t = threadIdx.x & 3;
  float x[D / 32][8], top = 0.f;
  const int i = p.by_group(row0 + r);
  const long long at = (rq.first + i) * p.q_st + (h * p.group + row0 + r - i * p.group) * p.q_sh;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (r < rows && dbg_access(rq.first + i < p.tokens && h < p.kv_heads && row0 + r < rq.rows, kErrKv4))
      raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + 32 * j + 8 * t);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p.is_half) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[j][2 * k] = v.x;
        x[j][2 * k + 1] = v.y;
      } else {
        x[j][2 * k] = bf16_lo(w[k]);
        x[j][2 * k + 1] = bf16_hi(w[k]);
      }
      top = fmaxf(top, fmaxf(fabsf(x[j][2 * k]), fabsf(x[j][2 * k + 1])));
    }
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 227);
  const float down = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
#pragma unroll
  for (int gp = 0; gp < D / 64; ++gp) sum[gp] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float less = k & 1 ? down * 0.0625f : down;
      f[j][k] = pack_f16x2(x[j][k] * less, x[j][k + 4] * less);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[j][k]));
      sum[j / 2] = fmaf(v.x + v.y, k & 1 ? 16.f : 1.f, sum[j / 2]);
    }
#pragma unroll
  for (int gp = 0; gp < D / 64; ++gp) {
    sum[gp] += __shfl_xor_sync(0xffffffffu, sum[gp], 1);
    sum[gp] += __shfl_xor_sync(0xffffffffu, sum[gp], 2);
    sum[gp] *= 0x1p-24f;
  }
  factor = __uint_as_float(static_cast<uint32_t>(e + 10) << 23) * p.scale_log2;
}

// Running state of a warp's rows (columns 2t, 2t + 1 of each row tile).  A row's
// state follows from the keys that the row sees alone: what moves for one row
// moves for no other, so a row's bits do not depend on tokens hidden from it.
template <int D, int NT>
struct Kv4State {
  float acc[D / 64][4][NT][4];  // O^T 2^-34 w, odd channels times 16
  float lo_sum[NT][D / 64][2];  // sum of P times V's lowest values
  float l[NT][2], m[NT][2];
  uint32_t w[NT];  // byte 2 group + r: the unit w = 2^(2 byte - 127) of P s 2^-10; byte 0: w = 0
  float w_most[D / 64];  // the largest w of the lane's rows times 2^-4
};
__device__ __forceinline__ float kv4_unit(uint32_t w, int gp, int r) {
  return __uint_as_float(__byte_perm(w, 0, 0x444 | (2 * gp + r) << 12));
}
// The unit that brings `big` to [8, 32).
__device__ __forceinline__ uint32_t kv4_unit_byte(float big) {
  return min(max((258 - static_cast<int>(__float_as_uint(big) >> 23)) >> 1, 2), 126);
}
// One unit over another, 0 where that one is 0; at most 2^126.
__device__ __forceinline__ float kv4_unit_ratio(uint32_t to, uint32_t from) {
  const int steps = static_cast<int>(to) - static_cast<int>(from);
  return from == 0 || steps < -63 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + 2 * min(steps, 63)) << 23);
}
// The least of the row's largest P s for which a unit may stand.
__device__ __forceinline__ float kv4_unit_least(float unit) {
  return unit == 0.f ? 0.f : __uint_as_float(0x80800000u - __float_as_uint(unit));  // 8 / unit
}

// A lane's places in a tile: K code words of its two rows' first, their
// parameters, V code words of its four tokens' first.
template <int D>
struct Kv4Lane {
  uint32_t k, par, v;
  __device__ __forceinline__ Kv4Lane() {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, tau = kv4_tau(g);
    k = tau * Kv4Tile<D>::kRow + t * (D / 32) * 4;
    par = tau * Kv4Tile<D>::kPar;
    v = t * Kv4Tile<D>::kRow + g * (D / 64) * 4;
  }
};

// kTiles tiles of 16 adjacent keys from shared memory.  kMasked: some row does
// not see all of them (keys no row sees may hold anything).
//
// Every second tile takes V as highest - s (15 - n) in place of lowest + s n: the
// sums of P s n that the matrix instructions add up, all of one sign, then cancel
// from tile to tile.  Over a long context O is a small difference of those sums
// and of P lowest, and their own roundings would show in it (2 million keys of
// one head: O off by 2.4e-3 of itself without this, 1.7e-3 with it, 1.66e-3 of
// which is its rounding to bf16; 131072 keys 1.70e-3 either way).
template <int D, int NT, int kTiles, bool kMasked>
__device__ __forceinline__ void kv4_tiles(const uint8_t* tile, const Kv4Lane<D>& at,
                                          const uint8_t* q_smem,
                                          const uint32_t (&qf)[NT > 2 ? 1 : NT][D / 32][4],
                                          const float (&qs)[NT][D / 64][2],
                                          const float (&rs)[NT][2], const int (&lim)[NT][2],
                                          int key0, int any_sees, Kv4State<D, NT>& st) {
  using T = Kv4Tile<D>;
  constexpr int kGroups = D / 64, kKW = D / 32, kVW = D / 64, kTok = 2 * kTiles;
  const int lane = threadIdx.x & 31;
  // the lane's tokens in the score fragments: tau and tau + 8 of each tile
  uint32_t kp[kTok][kGroups], vp[kTok][kGroups];
  float s[kTiles][NT][kGroups][4] = {};
  // ---- S^T = K q^T, by groups
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
    const uint8_t* base = tile + u * T::kBytes;
    uint32_t k0[kKW], k1[kKW];
    load_words<kKW>(base + at.k, k0);
    load_words<kKW>(base + at.k + 8 * T::kRow, k1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_words<kGroups>(base + at.par + T::kOffKPar + 8 * i * T::kPar, kp[2 * u + i]);
      load_words<kGroups>(base + at.par + T::kOffVPar + 8 * i * T::kPar, vp[2 * u + i]);
    }
#pragma unroll
    for (int j = 0; j < kKW; ++j) {
      uint32_t a[4], c[4];
      codes_f16(k0[j], a);
      codes_f16(k1[j], c);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint4 f;
        if (NT > 2)
          f = *reinterpret_cast<const uint4*>(q_smem + ((nt * kKW + j) * 32 + lane) * 16);
        else
          f = make_uint4(qf[nt % (NT > 2 ? 1 : NT)][j][0], qf[nt % (NT > 2 ? 1 : NT)][j][1],
                         qf[nt % (NT > 2 ? 1 : NT)][j][2], qf[nt % (NT > 2 ? 1 : NT)][j][3]);
        mma_f16(s[u][nt][j / 2], a[0], c[0], a[1], c[1], f.x, f.y);
        mma_f16(s[u][nt][j / 2], a[2], c[2], a[3], c[3], f.z, f.w);
      }
    }
  }
  auto odd = [&](int u) { return kTiles == 2 ? u == 1 : ((key0 >> 4) & 1) != 0; };
  int key[kTok];
  float vs[kTok][kGroups], vl[kTok][kGroups], x[NT][2 * kTok], y[NT][2 * kTok];
  float most = 0.f, large = 0.f;
  // (s times 2^-10, so that its product with P is finite for every s; negative for
  // the tiles taken from above)
#pragma unroll
  for (int i = 0; i < kTok; ++i) {
    key[i] = key0 + kv4_tau(lane >> 2) + 8 * i;
    const bool gone = kMasked && key[i] >= any_sees;
#pragma unroll
    for (int gp = 0; gp < kGroups; ++gp) {
      const float s_v = bf16_lo(vp[i][gp]), lowest = bf16_hi(vp[i][gp]);
      vs[i][gp] = gone ? 0.f : s_v * (odd(i >> 1) ? -0x1p-10f : 0x1p-10f);
      vl[i][gp] = gone ? 0.f : odd(i >> 1) ? fmaf(15.f, s_v, lowest) : lowest;
    }
  }
#pragma unroll
  for (int gp = 0; gp < kGroups; ++gp) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; i += 2) top = fmax3(fabsf(vs[i][gp]), fabsf(vs[i + 1][gp]), top);
    large = fmaxf(large, top * st.w_most[gp]);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2 * kTok; ++c) {
      const int i = c >> 1, r = c & 1;
      float v = 0.f;
#pragma unroll
      for (int gp = 0; gp < kGroups; ++gp)
        v = fmaf(bf16_lo(kp[i][gp]), s[i >> 1][nt][gp][c & 3], fmaf(bf16_hi(kp[i][gp]), qs[nt][gp][r], v));
      // (a product and a difference, not one fused: the row's largest is then
      // exactly 0 away from its reference, whatever its size)
      x[nt][c] = __fmul_rn(v, rs[nt][r]);
      y[nt][c] = __fsub_rn(x[nt][c], st.m[nt][r]);
      if (kMasked && key[i] >= lim[nt][r]) y[nt][c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 2 * kTok; c += 2) most = fmax3(y[nt][c], y[nt][c + 1], most);
  }
  // ---- A row's reference moves only when one of its scores passes it by 2^8, its
  // groups' units with it, and where a P s would pass 2^15 (fp16 ends below 2^16):
  // most tiles need no reduction over lanes.  P is below 2^8, so only a tile with a
  // scale of V beyond 2^7 in some row's unit has its products looked at.  (What
  // follows is seldom run and long: fetched anew it costs some 30000 cycles, so that
  // 2^4 in place of 2^8 made 8 drafted tokens of 4 heads twice as slow.)
  bool over = most > 8.f;
  if (__any_sync(0xffffffffu, fmaxf(most, large) > 8.f)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int gp = 0; gp < kGroups; ++gp)
#pragma unroll
        for (int c = 0; c < 2 * kTok; ++c)
          over |= ex2_approx(y[nt][c]) * fabsf(vs[c >> 1][gp]) * kv4_unit(st.w[nt], gp, c & 1) > 32768.f;
    over = __any_sync(0xffffffffu, over);
  } else {
    over = false;
  }
  if (over) {
#pragma unroll
    for (int gp = 0; gp < kGroups; ++gp) st.w_most[gp] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float hi = -INFINITY;
#pragma unroll
        for (int c = r; c < 2 * kTok; c += 2)
          if (!kMasked || key[c >> 1] < lim[nt][r]) hi = fmaxf(hi, x[nt][c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        const bool moves = hi - st.m[nt][r] > 8.f;
        const float f = moves ? ex2_approx(st.m[nt][r] - hi) : 1.f;
        st.m[nt][r] = moves ? hi : st.m[nt][r];
        st.l[nt][r] *= f;
#pragma unroll
        for (int c = r; c < 2 * kTok; c += 2) {
          y[nt][c] = __fsub_rn(x[nt][c], st.m[nt][r]);
          if (kMasked && key[c >> 1] >= lim[nt][r]) y[nt][c] = -INFINITY;
        }
        float weight[kGroups] = {};  // the largest P s of the tile
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) {
#pragma unroll
          for (int c = r; c < 2 * kTok; c += 2)
            if (!kMasked || key[c >> 1] < lim[nt][r])
              weight[gp] = fmaxf(weight[gp], ex2_approx(y[nt][c]) * fabsf(vs[c >> 1][gp]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            weight[gp] = fmaxf(weight[gp], __shfl_xor_sync(0xffffffffu, weight[gp], o));
        }
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) {
          st.lo_sum[nt][gp][r] *= f;
          const int at = 8 * (2 * gp + r);
          const uint32_t from = st.w[nt] >> at & 0xffu;
          const float old = kv4_unit(st.w[nt], gp, r);
          uint32_t to = from;
          float fall = f;
          if (moves || weight[gp] * old > 32768.f) {
            to = kv4_unit_byte(fmaxf(kv4_unit_least(old) * f, weight[gp]));
            fall *= kv4_unit_ratio(to, from);
          }
          st.w[nt] = (st.w[nt] & ~(0xffu << at)) | to << at;
          st.w_most[gp] = fmaxf(st.w_most[gp], kv4_unit(st.w[nt], gp, r) * 0x1p-4f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            st.acc[gp][i][nt][r] *= fall;
            st.acc[gp][i][nt][r + 2] *= fall;
          }
        }
      }
  }
  // ---- P, P s as B fragments, P lowest
  uint32_t pb[kTiles][NT][kGroups][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float e[2 * kTok];
#pragma unroll
    for (int c = 0; c < 2 * kTok; ++c) {
      e[c] = ex2_approx(y[nt][c]);
      st.l[nt][c & 1] += e[c];
    }
#pragma unroll
    for (int gp = 0; gp < kGroups; ++gp) {
      const float2 unit = make_float2(kv4_unit(st.w[nt], gp, 0), kv4_unit(st.w[nt], gp, 1));
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        float2 v = mul_f32x2(make_float2(e[2 * i] * vs[i][gp], e[2 * i + 1] * vs[i][gp]), unit);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bool hidden = kMasked && key[i] >= lim[nt][r];
          if (hidden) (r ? v.y : v.x) = 0.f;
          st.lo_sum[nt][gp][r] = hidden ? st.lo_sum[nt][gp][r]
                                        : fmaf(e[2 * i + r], vl[i][gp], st.lo_sum[nt][gp][r]);
        }
        pb[i >> 1][nt][gp][i & 1] = transpose8(pack_f16x2(v.x, v.y));
      }
    }
  }
  // ---- O^T += V^T P^T
#pragma unroll
  for (int u = 0; u < kTiles; ++u) {
    uint32_t vw[4][kVW];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_words<kVW>(tile + u * T::kBytes + at.v + T::kOffV + 4 * i * T::kRow, vw[i]);
#pragma unroll
    for (int j = 0; j < kVW; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7632u : 0x5410u;
        uint32_t a[4], c[4];
        const uint32_t flip = odd(u) ? ~0u : 0u;
        codes_f16(__byte_perm(vw[0][j], vw[1][j], sel), a, flip);
        codes_f16(__byte_perm(vw[2][j], vw[3][j], sel), c, flip);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = pb[u][nt][j][0], b1 = pb[u][nt][j][1];
          mma_f16(st.acc[j][2 * half][nt], a[0], a[1], c[0], c[1], b0, b1);
          mma_f16(st.acc[j][2 * half + 1][nt], a[2], a[3], c[2], c[3], b0, b1);
        }
      }
  }
}

// The bounded wait, with everything but its first look out of line.
__device__ __noinline__ bool kv4_wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                           volatile int* abort_flag) {
  return wait_bounded_warp(bar, parity, limit_ns, abort_flag, kErrKv4 | kErrRoleLoad);
}
__device__ __forceinline__ bool kv4_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                         volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         kv4_wait_long(bar, parity, limit_ns, abort_flag);
}

// Each warp walks its own blocks of 64 keys (every fourth of the CTA's) through
// its own ring of stages, filled by bulk copies of whole tiles: no barrier
// between warps until their results are joined.
template <int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32, (Kv4AttendLayout<D, NT>::kCtas))
    kv4_attend_kernel(const __grid_constant__ Kv4AttendParams p) {
  using T = Kv4Tile<D>;
  using L = Kv4AttendLayout<D, NT>;
  constexpr int kGroups = D / 64, kKW = D / 32, kVW = D / 64, kS = L::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Kv4Shared sh;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  float* merge = reinterpret_cast<float*>(smem);
  float* s_m = reinterpret_cast<float*>(smem + L::kOffMl);
  float* s_l = s_m + kKv4Warps * L::kRows;
  float* s_qs = reinterpret_cast<float*>(smem + L::kOffQs);
  float* s_rs = reinterpret_cast<float*>(smem + L::kOffRs);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  constexpr int kFast = L::kFast, kBT = L::kTiles;
  constexpr uint32_t kAll = (1u << kBT) - 1u;
  const Kv4Lane<D> places;
  const int ctas = gridDim.x, cta = blockIdx.x;
  const uint8_t* ring = smem + warp * kS * L::kBlock;
  const uint32_t ring_at = smem_u32(ring);
  const uint32_t bars = smem_u32(smem + L::kOffBar) + warp * kS * 8;
  if (lane == 0)
    for (int i = 0; i < kS; ++i) mbar_init(bars + 8 * i, 1);
  if (tid == 0) abort_word = 0;
  fence_barrier_init();
  fence_proxy_async_smem();
  kv4_locate<L::kRows, L::kUnit, kKv4Warps>(p, sh, cta, ctas);
  const Kv4Share share(sh.total, ctas);
  const long long u_begin = share.start(cta), u_end = share.start(cta + 1);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (u_begin >= u_end) return;
  Kv4Walk<L::kRows, L::kUnit> walk(p, sh.found_b, sh.found_excl);
  const int tiles_per_page = p.page_size / 16;
  int it = 0;  // blocks this warp has taken from its ring

  for (long long u = u_begin; u < u_end;) {
    walk.to(p, u);
    const Kv4Req& rq = walk.rq;
    const int b = walk.b, h = walk.h, c0 = walk.c0;
    const int c1 = static_cast<int>(min(static_cast<long long>(walk.units), c0 + (u_end - u)));
    const int row0 = walk.tile * L::kRows;
    const int rows = min(L::kRows, rq.rows - row0);
    const int all_see = kv4_sees(p, rq, row0), any_sees = kv4_sees(p, rq, row0 + rows - 1);

    // ---- fill the ring; pages of the block after next are looked up an
    // iteration ahead of their copy
    const int tile_end = min(max(c1 - p.lead, 0) * (L::kUnit / 16), (any_sees + 15) / 16);
    const int blk0 = max(c0 - p.lead, 0) * kKv4Warps + warp;
    const int n_blk = max(0, ((tile_end + kBT - 1) / kBT - blk0 + kKv4Warps - 1) / kKv4Warps);
    const int* table = p.table + b * p.table_stride;
    const uint8_t* head_base = p.cache + static_cast<long long>(h) * tiles_per_page * T::kBytes;
    const long long page_bytes = static_cast<long long>(p.kv_heads) * tiles_per_page * T::kBytes;
    // Lane i looks up and copies a block's tile i, a block ahead with the look-up.
    uint32_t present = 0;  // a bit a tile of each stage: it is there
    int tile = kBT * blk0 + lane, fill = it % kS;
    long long from = -1;  // the lane's next tile in the cache, -1: none
    auto look_up = [&]() {
      from = -1;
      if (lane < kBT && tile < tile_end) {
        const int page = p.page_tiles(tile);
        const int id = dbg_access(tile >= 0 && page < p.width && tile - page * tiles_per_page < tiles_per_page &&
                                      b < p.requests && h < p.kv_heads,
                                  kErrKv4)
                           ? table[page]
                           : -1;
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.pages))
          from = id * page_bytes + static_cast<long long>(tile - page * tiles_per_page) * T::kBytes;
        else
          atomicOr(&g_error_word, kErrBadPage);
      }
      tile += kBT * kKv4Warps;
    };
    auto copy = [&]() {  // (a block past the end: nothing is expected)
      const uint32_t in = __ballot_sync(0xffffffffu, from >= 0);
      present = (present & ~(kAll << (kBT * fill))) | in << (kBT * fill);
      const uint32_t bar = bars + 8 * fill;
      if (lane < kBT) {
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(in) * T::kBytes);
        if (from >= 0)
          bulk_load(ring_at + fill * L::kBlock + lane * T::kBytes, head_base + from, T::kBytes, bar);
      }
      if (++fill == kS) fill = 0;
    };
    const int n_fill = min(kS - 1, n_blk);
    for (int i = 0; i < n_fill; ++i) {
      look_up();
      copy();
    }
    look_up();

    // ---- the rows: q as B fragments, its sums over groups, factors
    uint32_t qf[NT > 2 ? 1 : NT][kKW][4];
    float qs[NT][kGroups][2], rs[NT][2];
    int lim[NT][2];
    if (NT > 2) {  // warp nt lays out row tile nt for all
      if (warp < NT) {
        float sum[kGroups], factor;
        kv4_rows<D>(p, rq, h, row0, 8 * warp + g, rows, qf[0], sum, factor);
#pragma unroll
        for (int j = 0; j < kKW; ++j)
          *reinterpret_cast<uint4*>(smem + L::kOffQ + ((warp * kKW + j) * 32 + lane) * 16) =
              make_uint4(qf[0][j][0], qf[0][j][1], qf[0][j][2], qf[0][j][3]);
        if (t == 0) {
#pragma unroll
          for (int gp = 0; gp < kGroups; ++gp) s_qs[(warp * kGroups + gp) * 8 + g] = sum[gp];
          s_rs[8 * warp + g] = factor;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum[kGroups], factor = 0.f;
      if (NT <= 2)
        kv4_rows<D>(p, rq, h, row0, 8 * nt + g, rows, qf[nt % (NT > 2 ? 1 : NT)], sum, factor);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nt + 2 * t + i;
        // from a lane of the row (g = row) to the lanes of its column (t)
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp)
          qs[nt][gp][i] = NT > 2 ? s_qs[(nt * kGroups + gp) * 8 + 2 * t + i]
                                 : __shfl_sync(0xffffffffu, sum[gp], (2 * t + i) * 4);
        rs[nt][i] = NT > 2 ? s_rs[r] : __shfl_sync(0xffffffffu, factor, (2 * t + i) * 4);
        lim[nt][i] = r < rows ? kv4_sees(p, rq, row0 + r) : 0;
      }
    }

    Kv4State<D, NT> st = {};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) st.m[nt][0] = st.m[nt][1] = -3.402823466e38f;  // below every score

    bool ok = true;
    int i = 0, stage = it % kS, key0 = 16 * kBT * blk0;
    uint32_t parity = (it / kS) & 1;
    for (; i < n_blk; ++i) {
      if (i + kS - 1 < n_blk) {
        copy();
        look_up();
      }
      if (!kv4_wait(bars + 8 * stage, parity, p.limit_ns, abort_flag)) {
        ok = false;
        break;
      }
      const uint8_t* at = ring + stage * L::kBlock;
      const uint32_t there = (present >> (kBT * stage)) & kAll;
      if (there == kAll && key0 + 16 * kBT <= all_see) {
#pragma unroll 1
        for (int k = 0; k < kBT; k += kFast)
          kv4_tiles<D, NT, kFast, false>(at + k * T::kBytes, places, smem + L::kOffQ, qf, qs, rs, lim,
                                         key0 + 16 * k, any_sees, st);
      } else {
#pragma unroll 1
        for (int k = 0; k < kBT; ++k)
          if ((there >> k) & 1u)
            kv4_tiles<D, NT, 1, true>(at + k * T::kBytes, places, smem + L::kOffQ, qf, qs, rs, lim,
                                      key0 + 16 * k, any_sees, st);
      }
      __syncwarp();
      key0 += L::kUnit;
      if (++stage == kS) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (!ok && lane == 0)  // let the copies in flight land
      for (int j = i; j < min(i + kS, n_blk); ++j)
        drain_wait(bars + 8 * ((it + j) % kS), ((it + j) / kS) & 1, p.limit_ns);
    it += n_blk;
    __syncthreads();  // the ring is empty
    if (*abort_flag) return;

    // ---- this warp's results to shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = st.l[nt][r];
        float lo[kGroups];
#pragma unroll
        for (int gp = 0; gp < kGroups; ++gp) lo[gp] = st.lo_sum[nt][gp][r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
          for (int gp = 0; gp < kGroups; ++gp) lo[gp] += __shfl_xor_sync(0xffffffffu, lo[gp], o);
        }
        const int row = 8 * nt + 2 * t + r;
        float* to = merge + (warp * L::kRows + row) * L::kPitch;
#pragma unroll
        for (int j = 0; j < kVW; ++j) {
          float v[8];
          const float up = 0.125f * kv4_unit_least(kv4_unit(st.w[nt], j, r));  // 1 / unit
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = fmaf(st.acc[j][k][nt][r] * 0x1p34f, up, lo[j]);
            v[2 * k + 1] = fmaf(st.acc[j][k][nt][r + 2] * 0x1p30f, up, lo[j]);
          }
          *reinterpret_cast<float4*>(to + 64 * j + 8 * g) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(to + 64 * j + 8 * g + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
        if (g == 0) {
          // no key seen (a row of NaN scores has a NaN sum instead)
          s_m[warp * L::kRows + row] =
              st.m[nt][r] == -3.402823466e38f && sum == 0.f ? -INFINITY : st.m[nt][r];
          s_l[warp * L::kRows + row] = sum;
        }
      }
    __syncthreads();
    // a warp takes every fourth row: a lane D / 32 channels
    const bool whole = c0 == 0 && c1 == walk.units;
    float* part = p.part + (2LL * cta + (u == u_begin && c0 > 0 ? 0 : 1)) * L::kPartFloats;
    for (int r = warp; r < rows; r += kKv4Warps) {
      float top = -INFINITY, sum = 0.f, f[kKv4Warps], o[D / 32] = {};
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) top = fmaxf(top, s_m[w * L::kRows + r]);
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        const float mw = s_m[w * L::kRows + r];
        f[w] = mw == -INFINITY ? 0.f : ex2_approx(mw - top);
        const float lw = s_l[w * L::kRows + r];
        if (mw != -INFINITY) sum = fmaf(lw, f[w], sum);
        float v[D / 32];
        load_floats<D / 32>(merge + (w * L::kRows + r) * L::kPitch + lane * (D / 32), v);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          if (mw != -INFINITY) o[k] = fmaf(v[k], f[w], o[k]);
      }
      if (whole)
        kv4_store_row<D>(p, rq, h, row0 + r, lane, o, top, sum);
      else if (dbg_access(part + L::kPartFloats <= p.part + p.part_floats, kErrKv4)) {
        store_floats<D / 32>(part + r * D + lane * (D / 32), o);
        if (lane == 0) {
          part[L::kRows * D + r] = top;
          part[L::kRows * (D + 1) + r] = sum;
        }
      }
    }
    fence_proxy_async_smem();  // the next piece's copies follow these accesses
    __syncthreads();
    u += c1 - c0;
  }
}

// Joins the partial results.  Block (c, y) looks at the start of CTA c + 1's
// range: if it cuts a (request, row tile, head), and no earlier range start
// does, the blocks of c own that cut one and sum its pieces, left by the CTAs
// in order; each of their warps takes one row, its lanes first find the
// pieces' weights.  It is launched while the attention kernel still runs, finds
// its place meanwhile, and waits for that kernel's end before it reads.
template <int D, int NT>
__global__ void __launch_bounds__(kKv4Warps * 32)
    kv4_combine_kernel(const __grid_constant__ Kv4AttendParams p, int ctas) {
  using L = Kv4AttendLayout<D, NT>;
  __shared__ Kv4Shared sh;
  const int cta = blockIdx.x + 1, lane = threadIdx.x & 31;
  kv4_locate<L::kRows, L::kUnit, kKv4Warps>(p, sh, cta, ctas);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (sh.found_b < 0) return;
  const Kv4Share share(sh.total, ctas);
  const long long cut = share.start(cta);
  Kv4Walk<L::kRows, L::kUnit> walk(p, sh.found_b, sh.found_excl);
  walk.to(p, cut);
  const Kv4Req& rq = walk.rq;
  const long long u0 = walk.job_start(), u1 = u0 + walk.units;
  if (cut == u0 || share.start(cta - 1) > u0) return;
  const int h = walk.h, row0 = walk.tile * L::kRows;
  const int rows = min(L::kRows, rq.rows - row0);
  const int r = blockIdx.y * kKv4Warps + (threadIdx.x >> 5);
  if (r >= rows) return;
  // CTAs first .. last hold a piece each (none is empty: it starts below u1)
  const int first = cta - 1;
  int last = cta;
  while (share.start(last + 1) < u1) ++last;
  // piece k of the cut one: the first CTA left it in its second place if it
  // began there, all others in their first
  auto piece = [&](int k) {
    return p.part + (2LL * (first + k) + (k == 0 && share.start(first) <= u0 ? 1 : 0)) * L::kPartFloats;
  };
  const int n = last - first + 1;
  if (!dbg_access(first >= 0 && last < ctas && 2LL * ctas * L::kPartFloats <= p.part_floats, kErrKv4)) return;
  float top = -INFINITY;
  for (int k = lane; k < n; k += 32) top = fmaxf(top, piece(k)[L::kRows * D + r]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f, o[D / 32] = {};
  for (int k0 = 0; k0 < n; k0 += 32) {
    float w = 0.f;
    if (k0 + lane < n) {
      const float m = piece(k0 + lane)[L::kRows * D + r];
      if (m != -INFINITY) {
        w = ex2_approx(m - top);
        sum = fmaf(piece(k0 + lane)[L::kRows * (D + 1) + r], w, sum);
      }
    }
    const int here = min(32, n - k0);
#pragma unroll 4
    for (int k = 0; k < here; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      float v[D / 32];
      load_floats<D / 32>(piece(k0 + k) + r * D + lane * (D / 32), v);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] = fmaf(v[c], wk, o[c]);
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  kv4_store_row<D>(p, rq, h, row0 + r, lane, o, top, sum);
}

}  // namespace fa
