// kv4_chunk.cuh -- attention over the paged 4-bit cache for many query rows (a
// prompt's chunk, long drafts): the tcgen05 form of kv4_attend.cuh.
//
// Same operation, layouts and order of work; here a work item is 256 rows (two
// tiles of 128; row = query * group + head) of one request and kv head against
// 128-key tiles, with S = Q K^T and O += P V on tcgen05 (fp16 operands, fp32
// accumulators in TMEM).
//
// Operands.  Q rows enter as fp16 times a power of two that brings the row's
// largest element near fp16's largest (exact for bf16 and fp16 input down to
// 2^-24 of it).  K and V tiles are put together by four warps each from the codes:
// lowest, rounded to fp16, plus scale n in one fused multiply-add, in units of a
// power of two that bring the largest value to [2^8, 2^9).  So a key or value is
// off by at most 2^-11 of itself and of its group's lowest (a bf16 copy of the
// cache: 2^-8 of itself), and those below 2^-22 of the largest by 2^-33 of it.
// Whose largest: of the tile for K, of the keys so far for V (O is rescaled when
// it grows), where every row of the item sees the whole tile; in the last tiles,
// with keys that some rows do not see, each key has units of its own: the
// score's columns are multiplied by K's, and P by V's over a unit of the row that
// follows from the keys it sees.  So no bit of a row depends on a key hidden
// from it.  P is fp16, statistics and O are fp32.  The channels of a 64-bit chunk of codes stay in
// the order in which they come out of a word, (0, 4), (1, 5), (2, 6), (3, 7):
// Q is laid out alike, and O's columns are put back in order when they leave.
//
// Warps (640 threads, one CTA an SM): 0 issues the MMAs; 4-7 put K together,
// 8-11 V (one key a thread, the next tile's codes on their way); 12-15 and 16-19
// lay out the rows of Q tile 0 and 1, run their softmax (one row a thread,
// exponentials against a reference that moves only where a score passes it by
// 2^14) and write O.
//
// Bound: the tensor cores, the softmax and putting K and V together share the
// SM about evenly (issue slots 52 % taken, the tensor pipe 39 %), and a row's
// softmax with the two MMAs that follow it makes the chain that sets the pace (by
// clock stamps, in the form of 598 us below: 3.7 k and 1 k cycles, the MMA warp
// waiting for P 1.7 k of 5.6 k a 128-key tile).  The codes are read once an item, a
// quarter of the bytes of a bf16 cache.  Two requests of 1000 queries, on 16384
// and 3000 keys, H=32/8 d=128 (301 GFLOP): 398 us, 756 TFLOP/s; two of 1024 on
// 16384 (533 GFLOP) 637 us, 837.  Kept steps, whole calls of the first:
// probabilities of a whole row held in registers 929 us; 32 columns at a time
// 492; K and V by a group of four warps each 450 (as two copies of the code 597:
// the instruction cache); one copy of the column code 442; the join told what to
// do 435; a job's fixed cost counted as work 388; no spills in the MMA warp 368
// (the second 598); codes as normal numbers and own units, for the precision above,
// 405 (646), the latter out of the way of the ordinary tiles 398 (637).
#pragma once

#include "kv4_attend.cuh"

namespace fa {

constexpr int kChunkRows = 256;
constexpr int kChunkUnit = 256;  // keys of a work unit
constexpr int kChunkWarps = 20;

template <int D>
struct Kv4ChunkLayout {
  static constexpr int kTile = 128 * D * 2;  // bytes of a Q, K or V tile
  static constexpr int kStages = 2;
  static constexpr int kOffQ = 0;            // two tiles
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffBar = kOffV + kStages * kTile;
  static constexpr int kQFull = 0;                  // [2] row tile laid out
  static constexpr int kKFull = 2;                  // [stages]
  static constexpr int kKEmpty = kKFull + kStages;
  static constexpr int kVFull = kKEmpty + kStages;
  static constexpr int kVEmpty = kVFull + kStages;
  static constexpr int kSFull = kVEmpty + kStages;  // [2]
  static constexpr int kPFull = kSFull + 2;         // [2]
  static constexpr int kOFinal = kPFull + 2;        // [2]
  static constexpr int kSize = kOFinal + 2;         // [4] the tile's sizes are known
  static constexpr int kDrain = kSize + 4;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kNumBars;  // TMEM base address
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kBytes = kOffAbort + 8;
  static constexpr int kSmemAlloc = kBytes + 1024;  // slack to align the base to 1 KiB
  static_assert(kSmemAlloc + 6144 <= 232448, "shared memory budget");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256;  // S: 128 columns a tile, O: D
  static constexpr int kPartFloats = kChunkRows * (D + 2);
  // the block launches with 96 registers a thread; the MMA warp needs them all
  // (64 / 64 / 144: its spilled values hold it up, 368 -> 388 us; 96 / 72 / 120: 375)
  static constexpr uint32_t kRegsOther = 96, kRegsPut = 64, kRegsSoftmax = 128;
  static_assert(128 * (kRegsOther + 2 * kRegsPut + 2 * kRegsSoftmax) <= 640 * 96, "register split");
};

// fp16 A and B, fp32 D (see idesc_bf16_f32; format 0 is fp16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// What the join needs about a cut (request, row tile, head), written by the CTA
// whose range start is the first to cut it.  (kv4_combine_kernel finds its place
// itself, while the attention kernel still runs on other SMs; here that kernel
// fills every SM to its end.)
struct alignas(16) Kv4Cut {
  int first, pieces;    // CTAs first .. first + pieces - 1 hold a piece each
  int second;           // CTA `first` left its piece in its second place
  int rows;             // 0: this range start joins nothing
  int token0, row0, h;  // first query of the request, row tile's first row, head
  int unused;
};
// Where CTA `cta`'s range starts inside a job of units u0 .. u1 - 1.
__device__ __forceinline__ Kv4Cut kv4_cut(const Kv4Share& share, int cta, long long u0,
                                          long long u1, const Kv4Req& rq, int row0, int rows, int h) {
  Kv4Cut c = {};
  if (share.start(cta) == u0 || share.start(cta - 1) > u0) return c;  // an earlier start cuts it
  int last = cta;
  while (share.start(last + 1) < u1) ++last;
  c.first = cta - 1;
  c.pieces = last - cta + 2;
  c.second = share.start(cta - 1) <= u0;
  c.rows = rows;
  c.token0 = rq.first;
  c.row0 = row0;
  c.h = h;
  return c;
}

// One cut of the work: `tiles[t]` key tiles of row tile t from key tile k0 on.
struct ChunkPiece {
  int b, h, row0, rows, k0, tiles[2], most;
  bool whole, head_cut;  // all of the (tile, head); begun by an earlier CTA
};
__device__ __forceinline__ ChunkPiece chunk_piece(const Kv4AttendParams& p,
                                                  const Kv4Walk<kChunkRows, kChunkUnit>& w,
                                                  int units) {
  ChunkPiece c;
  c.b = w.b;
  c.h = w.h;
  c.row0 = w.tile * kChunkRows;
  c.rows = min(kChunkRows, w.rq.rows - c.row0);
  c.k0 = max(w.c0 - p.lead, 0) * (kChunkUnit / 128);
  c.whole = w.c0 == 0 && units == w.units;
  c.head_cut = w.c0 > 0;
  const int end = max(w.c0 + units - p.lead, 0) * (kChunkUnit / 128);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(128 * (t + 1), c.rows) - 1;
    const int see = last >= 128 * t ? kv4_sees(p, w.rq, c.row0 + last) : 0;
    c.tiles[t] = max(0, min(end, (see + 127) / 128) - c.k0);
  }
  c.most = max(c.tiles[0], c.tiles[1]);
  return c;
}

// 8 codes as fp16 lowest + scale n, pairs (0, 4), (1, 5), (2, 6), (3, 7).  The
// codes are subnormal numbers n 2^-24 or 16 n 2^-24; a multiplication makes them
// n 2^-9 (exactly), so that 2^9 scale is an fp16 number for values up to 2^9.
__device__ __forceinline__ uint4 put_word(uint32_t w, uint32_t s9, uint32_t lo) {
  uint32_t c[4], r[4];
  codes_f16(w, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c[i]) : "r"(c[i]), "r"(i & 1 ? 0x68006800u : 0x78007800u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(c[i]), "r"(s9), "r"(lo));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Shared memory of a CTA beside the tiles: what a key tile's factors are, by
// tile number mod 4.  The K warps write tile g's place after they have seen K of
// tile g - 3 multiplied (the wait in front of tile g - 1's words).  Those products
// are issued behind the arrivals that end the softmax of tile g - 4 and the V warps'
// work on it, the last that read the place: with four places there is none to spare.
struct ChunkShared {
  float k_up[4];          // K in the tile is K / k_up
  alignas(16) uint32_t absent[4][4];  // keys whose page lies outside the cache
  alignas(16) float own_up[4][2][128];  // a key's units of K and V, times 2^-32, in a tile of own units
  int size[4][4][2];      // per K warp: largest exponent of K and V
};

// Units.  Exponents (with float's bias) are kept where unit, its reciprocal and
// the unit times 2^-32 are normal numbers: values below 2^-86 count as small
// parts of 2^-86.
__device__ __forceinline__ int chunk_size(int exponent) { return min(max(exponent, 41), 254); }
__device__ __forceinline__ float chunk_up(int size) {
  return __uint_as_float(static_cast<uint32_t>(size - 8) << 23);
}
__device__ __forceinline__ float chunk_down(int size) {
  return __uint_as_float(static_cast<uint32_t>(262 - size) << 23);
}
// Whether key tile `tile` has own units: some row of the item does not see all
// of its keys (`sure`: what the first row sees).
__device__ __forceinline__ bool chunk_own(int tile, int len, int sure) { return min(128 * tile + 128, len) > sure; }

// The factors of a key's codes: 2^9 scale, lowest, in its unit.
struct PutFactors {
  uint32_t s9, lo;
  __device__ __forceinline__ PutFactors(uint32_t par, float down) {
    const float s = bf16_lo(par) * down * 512.f, l = bf16_hi(par) * down;
    s9 = pack_f16x2(s, s);
    lo = pack_f16x2(l, l);
  }
};

// The four warps that put K (`value`: V) tiles together from their codes, one
// key a thread.  One code for both: as two, it and the softmax did not stay in
// the instruction cache (450 -> 597 us).  A key's data comes in steps so that no latency shows: its page
// two tiles ahead, its parameters a tile ahead, its codes as soon as the last
// tile's are used.  The K warps read V's parameters too and say how large both
// tiles' values are.
template <int D>
__device__ __forceinline__ void chunk_put(bool value, const Kv4AttendParams& p, const Kv4Shared& sh,
                                          ChunkShared& cs, uint32_t sb, volatile int* abort_flag,
                                          long long u_begin, long long u_end) {
  using L = Kv4ChunkLayout<D>;
  using T = Kv4Tile<D>;
  constexpr int S = L::kStages;
  constexpr unsigned int err = kErrKv4 | kErrRoleLoad;
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  const int lane = threadIdx.x & 31, in_group = (threadIdx.x >> 5) & 3;
  const int row = threadIdx.x & 127;  // the thread's key of each tile
  const int tiles_per_page = p.page_size / 16;
  uint32_t code[D / 8], kp[D / 64], vp[D / 64];
  const uint8_t* at = nullptr;  // the key's tile in the cache, null: there is none
  bool gone = false;            // its page lies outside the cache
  auto page_of = [&](const ChunkPiece& c, int len, int j) {
    const int key = (c.k0 + j) * 128 + row;
    return j < c.most && key < len &&
                   dbg_check(key >= 0 && static_cast<int>(p.page_tiles(key >> 4)) < p.width && c.b < p.requests,
                             err, abort_flag)
               ? p.table[c.b * p.table_stride + p.page_tiles(key >> 4)]
               : -1;
  };
  auto locate = [&](const ChunkPiece& c, int len, int j, int id) {
    const int key = (c.k0 + j) * 128 + row, tile = key >> 4;
    const bool live = j < c.most && key < len;
    const bool in = live && static_cast<unsigned>(id) < static_cast<unsigned>(p.pages);
    gone = live && !in;
    if (!value && gone) atomicOr(&g_error_word, kErrBadPage);
    const int place = tile - static_cast<int>(p.page_tiles(tile)) * tiles_per_page;
    if (!dbg_check(!in || (place >= 0 && place < tiles_per_page && c.h < p.kv_heads), err, abort_flag)) {
      at = nullptr;
      return;
    }
    at = in ? p.cache + ((static_cast<long long>(id) * p.kv_heads + c.h) * tiles_per_page + place) * T::kBytes
            : nullptr;
  };
  // Keys from `sure` on are hidden from some rows: 0 times a value that is no
  // finite number would reach them, so there a key that has one gets values 0
  // and a score of NaN instead, for the rows that see it.  (The largest scale that
  // values of 32 bits have is below 2^125.)
  auto fetch_par = [&](const ChunkPiece& c, int sure, int j) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) kp[i] = vp[i] = 0;
    if (!at) return;
    if (!value) load_words<D / 64>(at + T::kOffKPar + (row & 15) * T::kPar, kp);
    load_words<D / 64>(at + T::kOffVPar + (row & 15) * T::kPar, vp);
    if ((c.k0 + j) * 128 + row < sure) return;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) odd |= !isfinite(bf16_hi(vp[i])) || !(fabsf(bf16_lo(vp[i])) < 0x1p125f);
    if (odd) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        vp[i] = 0;
        kp[i] = 0x7fc00000u;
      }
    }
  };
  auto fetch_codes = [&]() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if (at)
        load_words<4>(at + (value ? T::kOffV : T::kOffK) + (row & 15) * T::kRow + 16 * i,
                      *reinterpret_cast<uint32_t(*)[4]>(&code[4 * i]));
      else
        code[4 * i] = code[4 * i + 1] = code[4 * i + 2] = code[4 * i + 3] = 0;
    }
  };
  // exponent of the largest value a pair of parameters stands for
  auto size_of = [&](const uint32_t (&par)[D / 64]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float s = bf16_lo(par[i]), lo = bf16_hi(par[i]);
      top = fmaxf(top, fmaxf(fabsf(lo), fabsf(fmaf(15.f, s, lo))));
    }
    return min(static_cast<int>(__float_as_uint(top) >> 23), 254);
  };
  const uint32_t base = sb + (value ? L::kOffV : L::kOffK) + row * 128, turn = (row & 7) << 4;
  const int full = value ? L::kVFull : L::kKFull, empty = value ? L::kVEmpty : L::kKEmpty;

  Kv4Walk<kChunkRows, kChunkUnit> walk(p, sh.found_b, sh.found_excl);
  int g = 0;  // key tiles so far
  for (long long u = u_begin; u < u_end;) {
    walk.to(p, u);
    const int units = static_cast<int>(min(static_cast<long long>(walk.units - walk.c0), u_end - u));
    const ChunkPiece c = chunk_piece(p, walk, units);
    u += units;
    if (c.most == 0) continue;
    int size = 0;  // exponent of the common unit: K's of the tile, V's so far in this piece
    const int len = walk.rq.len, sure = kv4_sees(p, walk.rq, c.row0);
    locate(c, len, 0, page_of(c, len, 0));
    fetch_par(c, sure, 0);
    fetch_codes();
    int id = page_of(c, len, 1);  // of the next tile's key
    for (int j = 0; j < c.most; ++j, ++g) {
      const int s = g % S, slot = g & 3;
      const bool own = chunk_own(c.k0 + j, len, sure);
      int mine = 0;
      if (!value || own) mine = size_of(value ? vp : kp);
      if (!value) {
        const int v_size = size_of(vp);
        if (own) {
          cs.own_up[slot][0][row] = chunk_up(chunk_size(mine)) * 0x1p-32f;
          cs.own_up[slot][1][row] = chunk_up(chunk_size(v_size)) * 0x1p-32f;
        }
        const int ek = __reduce_max_sync(0xffffffffu, mine);
        const int ev = __reduce_max_sync(0xffffffffu, v_size);
        const uint32_t absent = __ballot_sync(0xffffffffu, gone);
        if (lane == 0) {
          cs.size[slot][in_group][0] = ek;
          cs.size[slot][in_group][1] = ev;
          cs.absent[slot][in_group] = absent;
          mbar_arrive(bar(L::kSize + slot));
        }
      }
      if (!wait_bounded_warp(bar(L::kSize + slot), (g >> 2) & 1, p.limit_ns, abort_flag, err)) return;
      if (!value) size = 0;
      if (!own) {
#pragma unroll
        for (int w = 0; w < 4; ++w) size = max(size, cs.size[slot][w][value ? 1 : 0]);
      }
      const int x = chunk_size(own ? mine : size);
      if (!value && row == 0) cs.k_up[slot] = chunk_up(x);
      const float down = chunk_down(x);
      const PutFactors f0(value ? vp[0] : kp[0], down);
      const PutFactors f1(value ? vp[D / 64 - 1] : kp[D / 64 - 1], down);
      // where K's word is of the first group and V's of the second, and conversely
      const PutFactors f01 = value ? f1 : f0, f10 = value ? f0 : f1;
      locate(c, len, j + 1, id);
      fetch_par(c, sure, j + 1);
      id = page_of(c, len, j + 2);
      if (!wait_bounded_warp(bar(empty + s), ((g / S) & 1) ^ 1, p.limit_ns, abort_flag, err)) return;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {  // place i of the row: chunk w of 8 channels is word w's
        const int wk = 4 * (i % (D / 32)) + i / (D / 32), wv = 8 * (i % (D / 64)) + i / (D / 64);
        const PutFactors& f = (wk >> 3) == 0 ? ((wv >> 3) == 0 ? f0 : f01) : ((wv >> 3) == 0 ? f10 : f1);
        const uint32_t to_k = (wk >> 3) * 16384 + (wk & 7) * 16, to_v = (wv >> 3) * 16384 + (wv & 7) * 16;
        const uint4 v = put_word(code[i], f.s9, f.lo);
        st_shared_v4((base + s * L::kTile + (value ? to_v : to_k)) ^ turn, v.x, v.y, v.z, v.w);
      }
      fetch_codes();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(full + s));
    }
  }
}

// Multiplies a row's P of the first 32 cols columns of S.
__device__ __forceinline__ void chunk_fall(uint32_t s_addr, int cols, float less) {
  tmem_wait_st();
#pragma unroll 1
  for (int w = 0; w < cols; ++w) {
    uint32_t old[16];
    tmem_ld_32x32b_x16(s_addr + 16 * w, old);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      asm volatile("" : "+r"(old[i]));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&old[i]));
      old[i] = pack_f16x2(v.x * less, v.y * less);
    }
    tmem_st_32x32b_x16(s_addr + 16 * w, old);
  }
}

// The softmax of a row over a tile of own units (`up`: the keys' units of K, then
// of V, times 2^-32): P of a key is its probability times V's unit over the row's,
// which moves where a product passes 2^15.  Columns from `left` on are hidden.
// Out of line, for tiles after the ordinary ones: as a part of their loop it cost
// that a tenth of its speed (1000-token chunk 403 -> 449 us).
struct OwnTile {
  float m, v_up, alpha, sum;  // alpha: for l and O
};
__device__ __noinline__ OwnTile chunk_own_tile(uint32_t s_addr, const float* up, const uint32_t* absent,
                                                  float factor, int left, float m, float v_up) {
  OwnTile r = {m, v_up, 1.f, 0.f};
  const float2 to_log2 = make_float2(factor * 0x1p32f, factor * 0x1p32f);
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t x[32];
    tmem_ld_32x32b_x32(s_addr + 32 * q, x);
    tmem_wait_ld_regs(x);
    const int here = min(max(left - 32 * q, 0), 32);  // columns before it are seen
    const uint32_t seen = (here == 32 ? ~0u : (1u << here) - 1u) & ~absent[q];
    float hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 u = *reinterpret_cast<const float2*>(up + 32 * q + i);
      const float2 v = mul_f32x2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                 mul_f32x2(u, to_log2));
      x[i] = (seen >> i) & 1u ? __float_as_uint(v.x) : 0xff800000u;
      x[i + 1] = (seen >> (i + 1)) & 1u ? __float_as_uint(v.y) : 0xff800000u;
      hi = fmax3(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), hi);
    }
    const bool over = hi - r.m > 14.f;
    if (__any_sync(0xffffffffu, over)) {
      const float less = over ? ex2_approx(r.m - hi) : 1.f;
      r.m = over ? hi : r.m;
      r.alpha *= less;
      r.sum *= less;
      chunk_fall(s_addr, q, less);
    }
    float top = 0.f;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 u = *reinterpret_cast<const float2*>(up + 128 + 32 * q + i);
      const float2 y = add_f32x2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                 make_float2(-r.m, -r.m));
      const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
      sum = add_f32x2(sum, e);
      const float2 v = mul_f32x2(e, u);
      top = fmax3(v.x, v.y, top);
      x[i] = __float_as_uint(v.x);
      x[i + 1] = __float_as_uint(v.y);
    }
    r.sum += sum.x + sum.y;
    const bool large = top > 32768.f * r.v_up;
    if (__any_sync(0xffffffffu, large)) {  // the largest to [8, 16)
      const float next = __uint_as_float((max(__float_as_uint(top) >> 23, 4u) - 3u) << 23);
      const float less = large ? r.v_up / next : 1.f;
      r.v_up = large ? next : r.v_up;
      chunk_fall(s_addr, q, less);
    }
    const float2 down = make_float2(1.f / r.v_up, 1.f / r.v_up);
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 v = mul_f32x2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), down);
      pk[i] = pack_f16x2(v.x, v.y);
    }
    tmem_st_32x32b_x16(s_addr + 16 * q, pk);
  }
  return r;
}

template <int D>
__global__ void __launch_bounds__(kChunkWarps * 32, 1)
    kv4_chunk_kernel(const __grid_constant__ Kv4AttendParams p) {
  using L = Kv4ChunkLayout<D>;
  using T = Kv4Tile<D>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Kv4Shared sh;
  __shared__ ChunkShared cs;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8u * static_cast<uint32_t>(i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = gridDim.x, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      // four warps lay out a tile, put K and V together, write P, find sizes
      const bool by_warps = i < L::kKEmpty || (i >= L::kVFull && i < L::kVEmpty) ||
                            (i >= L::kPFull && i < L::kPFull + 2) ||
                            (i >= L::kSize && i < L::kDrain);
      mbar_init(bar(i), by_warps ? 4 : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  kv4_locate<kChunkRows, kChunkUnit, kChunkWarps>(p, sh, cta, ctas);  // (a block barrier)
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const Kv4Share share(sh.total, ctas);
  const long long u_begin = share.start(cta), u_end = share.start(cta + 1);
  const bool any = u_begin < u_end;
  const uint64_t limit = p.limit_ns;
  if (threadIdx.x == 32) {  // (an idle warp's)
    if (any) {
      Kv4Walk<kChunkRows, kChunkUnit> walk(p, sh.found_b, sh.found_excl);
      walk.to(p, u_begin);
      const int row0 = walk.tile * kChunkRows;
      p.cuts[cta] = kv4_cut(share, cta, walk.job_start(), walk.job_start() + walk.units, walk.rq, row0,
                            min(kChunkRows, walk.rq.rows - row0), walk.h);
    } else {
      p.cuts[cta].rows = 0;
    }
  }

  if (warp < 4) {
    setmaxnreg_dec<L::kRegsOther>();  // (says how many; they are the launch's)
    if (warp == 0 && any) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t id_s = idesc_f16_f32(128, 128, false);
      constexpr uint32_t id_o = idesc_f16_f32(128, D, true);
      constexpr unsigned int err = kErrKv4 | kErrRoleMma;
      auto issue_s = [&](int t, int g) {  // S_t = Q_t K^T, K from ring position g
        const uint32_t qa = sb + L::kOffQ + t * L::kTile, ka = sb + L::kOffK + (g % S) * L::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_bf16_ss(tmem + L::kColS + t * 128, sw128_desc(qa + off, 16, 1024),
                      sw128_desc(ka + off, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(bar(L::kSFull + t));
      };
      auto issue_pv = [&](int t, int g, bool first) {  // O_t (+)= P_t V
        const uint32_t va = sb + L::kOffV + (g % S) * L::kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(tmem + L::kColO + t * D, tmem + L::kColS + t * 128 + kk * 8,
                      sw128_desc(va + kk * 2048, 16384, 1024), id_o, (!first || kk > 0) ? 1u : 0u);
      };
      Kv4Walk<kChunkRows, kChunkUnit> walk(p, sh.found_b, sh.found_excl);
      int g = 0, pieces[2] = {0, 0}, steps[2] = {0, 0};  // key tiles, Q tiles, P tiles so far
      bool ok = true;
      for (long long u = u_begin; u < u_end && ok;) {
        walk.to(p, u);
        const int units = static_cast<int>(min(static_cast<long long>(walk.units - walk.c0), u_end - u));
        const ChunkPiece c = chunk_piece(p, walk, units);
        u += units;
        if (c.most == 0) continue;
        for (int t = 0; t < 2 && ok; ++t)
          if (c.tiles[t] > 0) {
            ok = wait_bounded_warp(bar(L::kQFull + t), pieces[t] & 1, limit, abort_flag, err);
            ++pieces[t];
          }
        ok = ok && wait_bounded_warp(bar(L::kKFull + g % S), (g / S) & 1, limit, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < 2; ++t)
          if (c.tiles[t] > 0) issue_s(t, g);
        tc_commit(bar(L::kKEmpty + g % S));
        for (int j = 0; j < c.most && ok; ++j, ++g) {
          const int s = g % S, s1 = (g + 1) % S;
          ok = wait_bounded_warp(bar(L::kVFull + s), (g / S) & 1, limit, abort_flag, err);
          bool k_seen = false;
          for (int t = 0; t < 2 && ok; ++t) {
            if (j >= c.tiles[t]) continue;
            ok = wait_bounded_warp(bar(L::kPFull + t), steps[t] & 1, limit, abort_flag, err);
            if (!ok) break;
            ++steps[t];
            tc_fence_after();
            issue_pv(t, g, j == 0);
            if (j + 1 == c.tiles[t]) {
              tc_commit(bar(L::kOFinal + t));
            } else {
              if (!k_seen)
                ok = wait_bounded_warp(bar(L::kKFull + s1), ((g + 1) / S) & 1, limit, abort_flag, err);
              k_seen = true;
              if (!ok) break;
              tc_fence_after();
              issue_s(t, g + 1);
            }
          }
          if (!ok) break;
          tc_commit(bar(L::kVEmpty + s));
          if (j + 1 < c.most) tc_commit(bar(L::kKEmpty + s1));
        }
      }
      // every MMA issued above must finish before TMEM / smem are released
      tc_commit(bar(L::kDrain));
      drain_wait(bar(L::kDrain), 0, limit);
      __syncwarp();
    }
  } else if (warp < 12) {
    setmaxnreg_dec<L::kRegsPut>();
    if (any) chunk_put<D>(warp >= 8, p, sh, cs, sb, abort_flag, u_begin, u_end);
  } else {
    setmaxnreg_inc<L::kRegsSoftmax>();
    if (any) {
      // --------------------------------------------------- rows, softmax, output
      constexpr unsigned int err = kErrKv4 | kErrRoleSoftmax;
      const int t = warp >= 16 ? 1 : 0;
      const int r = threadIdx.x - 384 - 128 * t;  // row of the tile == TMEM lane
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_addr = tmem + lane_off + L::kColS + t * 128;
      const uint32_t o_addr = tmem + lane_off + L::kColO + t * D;
      Kv4Walk<kChunkRows, kChunkUnit> walk(p, sh.found_b, sh.found_excl);
      int g = 0, steps = 0, finals = 0;  // key tiles of the CTA, of this row tile; outputs
      bool ok = true;
      for (long long u = u_begin; u < u_end && ok;) {
        walk.to(p, u);
        const int units = static_cast<int>(min(static_cast<long long>(walk.units - walk.c0), u_end - u));
        const ChunkPiece c = chunk_piece(p, walk, units);
        float* part = p.part + (2LL * cta + (u == u_begin && c.head_cut ? 0 : 1)) * L::kPartFloats;
        u += units;
        const Kv4Req rq = walk.rq;
        const int in_tile = 128 * t + r, row = c.row0 + in_tile;
        const bool real = in_tile < c.rows;
        const int tok = p.by_group(row), head = c.h * p.group + row - tok * p.group;
        const int n = c.tiles[t];
        if (kDebugChecks) {
          ok = __all_sync(0xffffffffu, dbg_check(tmem_range_ok(s_addr, tmem, 128, L::kTmemCols) &&
                                                     tmem_range_ok(o_addr, tmem, D, L::kTmemCols) &&
                                                     (!real || (rq.first + tok < p.tokens && head < p.heads)) &&
                                                     part + L::kPartFloats <= p.part + p.part_floats,
                                                 err, abort_flag));
          if (!ok) break;
        }
        float factor = 0.f;  // from scores in the tile's units to base-2 exponents
        if (n > 0) {
          // ---- this row of Q: fp16 times a power of two, in the channel order
          // of the codes' pairs; a negative scale is taken into Q
          uint32_t raw[D / 2];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (real)
              x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                  (rq.first + tok) * p.q_st + head * p.q_sh + 8 * i);
            raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
          }
          auto pair = [&](int i) {
            return p.is_half ? __half22float2(*reinterpret_cast<const __half2*>(&raw[i]))
                             : make_float2(bf16_lo(raw[i]), bf16_hi(raw[i]));
          };
#pragma unroll
          for (int i = 0; i < D / 2; ++i) {
            const float2 v = pair(i);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
          const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 227);
          float down = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
          factor = __uint_as_float(static_cast<uint32_t>(e - 14) << 23) * fabsf(p.scale_log2);
          if (p.scale_log2 < 0.f) down = -down;
          const uint32_t q_row = sb + L::kOffQ + t * L::kTile + r * 128;
#pragma unroll
          for (int w = 0; w < D / 8; ++w) {
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = pair(4 * w + i);
              v[i].x *= down;
              v[i].y *= down;
            }
            // channels (0, 4), (1, 5), (2, 6), (3, 7)
            st_shared_v4(q_row + (w >> 3) * 16384 + (((w & 7) ^ (r & 7)) << 4),
                         pack_f16x2(v[0].x, v[2].x), pack_f16x2(v[0].y, v[2].y),
                         pack_f16x2(v[1].x, v[3].x), pack_f16x2(v[1].y, v[3].y));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kQFull + t));
        }
        const int lim = real ? kv4_sees(p, rq, row) : 0;
        // keys that every row of this warp sees (rows past the end do not count)
        const int all_see = __reduce_min_sync(0xffffffffu, real ? lim : 0x7fffffff);
        const int sure = kv4_sees(p, rq, c.row0);
        float m = -3.402823466e38f, l = 0.f;
        float v_up = 0.f;  // the unit of O times 2^-32, 0: none yet
        int v_size = 0;    // V's common unit, as the V warps find it
        auto begin = [&]() {  // the next tile's scores
          ok = wait_bounded_warp(bar(L::kSFull + t), steps & 1, limit, abort_flag, err);
          ++steps;
          tc_fence_after();
          return ok;
        };
        // P is written: O follows the reference (alpha) and its unit
        auto end = [&](int j, float alpha, float next_up) {
          if (next_up != v_up) {
            alpha *= v_up / next_up;
            v_up = next_up;
          }
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // (S of this tile was issued after the last P V, which is done)
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t oc[32];
              tmem_ld_32x32b_x32(o_addr + 32 * q, oc);
              tmem_wait_ld_regs(oc);
#pragma unroll
              for (int i = 0; i < 32; ++i) oc[i] = __float_as_uint(__uint_as_float(oc[i]) * alpha);
              tmem_st_32x32b_x32(o_addr + 32 * q, oc);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kPFull + t));
        };
        // tiles of own units are the last ones (see chunk_own)
        const int first_own = sure >= rq.len ? n : min(max(sure / 128 - c.k0, 0), n);
        for (int j = 0; j < first_own; ++j) {
          const int slot = (g + j) & 3;
          if (!begin()) break;
          const int key0 = (c.k0 + j) * 128;
          float alpha = 1.f;  // what l and O are to be multiplied by
#pragma unroll
          for (int w = 0; w < 4; ++w) v_size = max(v_size, cs.size[slot][w][1]);
          const float next_up = chunk_up(chunk_size(v_size)) * 0x1p-32f;
          // (not 0: a hidden key's score is minus infinity times it; scores in these
          // units stay below 2^31)
          const float f = fmaxf(factor * cs.k_up[slot], 1e-30f);
          const uint4 absent = *reinterpret_cast<const uint4*>(cs.absent[slot]);
          const bool masked = key0 + 128 > all_see || (absent.x | absent.y | absent.z | absent.w) != 0;
          // 32 columns at a time (one copy of this code: unrolled with the next
          // columns loading meanwhile it is 3 % slower, for the instruction cache):
          // exponentials against the reference, sums, fp16, and the maximum
          // alongside; where some row's passes its reference by 2^14 the reference
          // moves, the columns are done again, and the probabilities of this tile
          // already written, the sums, and below O follow
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(s_addr + 32 * q, x);
            tmem_wait_ld_regs(x);
            if (masked) {
              const int left = min(max(lim - key0 - 32 * q, 0), 32);  // columns before it are seen
              const uint32_t seen = (left == 32 ? ~0u : (1u << left) - 1u) & ~cs.absent[slot][q];
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((seen >> i) & 1u)) x[i] = 0xff800000u;
            }
            uint32_t pk[16];
            float2 before = sum;
            for (int pass = 0;; ++pass) {  // (a second time only where the reference moved)
              float hi[2] = {-INFINITY, -INFINITY};
              sum = before;
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 v = make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                hi[(i / 2) & 1] = fmax3(v.x, v.y, hi[(i / 2) & 1]);
                // (a product and a difference, not one fused: the row's largest is
                // then exactly 0 away from its reference, whatever its size)
                const float2 y = add_f32x2(mul_f32x2(v, make_float2(f, f)), make_float2(-m, -m));
                const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                sum = add_f32x2(sum, e);
                pk[i / 2] = pack_f16x2(e.x, e.y);
              }
              const float top = fmaxf(hi[0], hi[1]);
              const bool over = top > -INFINITY && top * f - m > 14.f;
              if (pass == 1 || !__any_sync(0xffffffffu, over)) break;
              float less = 1.f;
              if (over) {
                const float next = top * f;
                less = ex2_approx(m - next);
                m = next;
              }
              alpha *= less;
              before.x *= less;
              before.y *= less;
              chunk_fall(s_addr, q, less);
            }
            tmem_st_32x32b_x16(s_addr + 16 * q, pk);
          }
          l = fmaf(l, alpha, sum.x + sum.y);
          end(j, alpha, next_up);
        }
        for (int j = first_own; j < n && ok; ++j) {
          const int slot = (g + j) & 3;
          if (!begin()) break;
          const OwnTile own = chunk_own_tile(s_addr, cs.own_up[slot][0], cs.absent[slot], factor,
                                             lim - (c.k0 + j) * 128, m, v_up == 0.f ? 0x1p-126f : v_up);
          m = own.m;
          l = fmaf(l, own.alpha, own.sum);
          end(j, own.alpha, own.v_up);
        }
        if (!ok) break;
        g += c.most;
        // ---- output
        if (n > 0) {
          if (!(ok = wait_bounded_warp(bar(L::kOFinal + t), finals & 1, limit, abort_flag, err))) break;
          ++finals;
          tc_fence_after();
        }
        const float unit_o = v_up * 0x1p32f;
        const float scale_o = n == 0 || l == 0.f ? 0.f : c.whole ? unit_o / l : unit_o;
        const float m_out = m == -3.402823466e38f && l == 0.f ? -INFINITY : m;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t oc[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) oc[i] = 0;
          if (n > 0) {
            tmem_ld_32x32b_x32(o_addr + 32 * q, oc);
            tmem_wait_ld_regs(oc);
          }
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {  // column 8 w + (0 .. 7) is channel 0, 4, 1, 5, 2, 6, 3, 7
            const int ch = (i & ~7) + (i & 7) / 2 + 4 * (i & 1);
            // (a row that sees nothing gets 0, whatever its accumulator holds)
            v[ch] = scale_o == 0.f ? 0.f : __uint_as_float(oc[i]) * scale_o;
          }
          if (c.whole) {
            if (real) {
              uint16_t* to = static_cast<uint16_t*>(p.o) + (rq.first + tok) * p.o_st + head * p.o_sh + 32 * q;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = p.is_half ? pack_f16x2(v[i + 2 * k], v[i + 2 * k + 1])
                                   : pack_bf16x2(v[i + 2 * k], v[i + 2 * k + 1]);
                *reinterpret_cast<uint4*>(to + i) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          } else {
            // four channels of a row together, rows beside each other
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part + ((8 * q + i / 4) * kChunkRows + in_tile) * 4) =
                  make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
        if (c.whole) {
          if (real)
            p.lse[static_cast<long long>(rq.first + tok) * p.heads + head] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else {
          part[kChunkRows * D + in_tile] = m_out;
          part[kChunkRows * (D + 1) + in_tile] = l;
        }
        // the next piece's P V overwrites O only after P is written again, by
        // these threads
        tc_fence_before();
      }
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, L::kTmemCols);
}

// Joins the partial results of kv4_chunk_kernel: blocks (c, y) those of the job
// that CTA c + 1's range start cuts, if that is the first to cut it (its Kv4Cut
// says so), y = 32 rows each; a lane takes a row, a warp every eighth group of
// four channels.
constexpr int kChunkJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kChunkJoinWarps * 32)
    kv4_chunk_combine_kernel(const __grid_constant__ Kv4AttendParams p, int ctas) {
  using L = Kv4ChunkLayout<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Kv4Cut cut = p.cuts[blockIdx.x + 1];
  if (r >= cut.rows) return;
  if (!dbg_access(cut.first >= 0 && cut.first + cut.pieces <= ctas && cut.rows <= kChunkRows &&
                      2LL * ctas * L::kPartFloats <= p.part_floats,
                  kErrKv4))
    return;
  auto piece = [&](int k) {
    return p.part + (2LL * (cut.first + k) + (k == 0 ? cut.second : 0)) * L::kPartFloats;
  };
  float top = -INFINITY, sum = 0.f;
  for (int k = 0; k < cut.pieces; ++k) top = fmaxf(top, piece(k)[kChunkRows * D + r]);
  for (int k = 0; k < cut.pieces; ++k) {
    const float m = piece(k)[kChunkRows * D + r];
    if (m != -INFINITY) sum = fmaf(piece(k)[kChunkRows * (D + 1) + r], ex2_approx(m - top), sum);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int row = cut.row0 + r, i = p.by_group(row), head = cut.h * p.group + row - i * p.group;
  const long long tok = cut.token0 + i;
  if (!dbg_access(tok < p.tokens && head < p.heads, kErrKv4)) return;
  uint16_t* to = static_cast<uint16_t*>(p.o) + tok * p.o_st + head * p.o_sh;
  constexpr int kEach = D / 4 / kChunkJoinWarps;  // groups of four channels of a warp
  float4 o[kEach] = {};
  for (int k = 0; k < cut.pieces; ++k) {
    const float m = piece(k)[kChunkRows * D + r];
    if (m == -INFINITY) continue;
    const float w = ex2_approx(m - top);
#pragma unroll
    for (int c = 0; c < kEach; ++c) {
      const float4 v = *reinterpret_cast<const float4*>(
          piece(k) + ((c * kChunkJoinWarps + warp) * kChunkRows + r) * 4);
      o[c].x = fmaf(v.x, w, o[c].x);
      o[c].y = fmaf(v.y, w, o[c].y);
      o[c].z = fmaf(v.z, w, o[c].z);
      o[c].w = fmaf(v.w, w, o[c].w);
    }
  }
#pragma unroll
  for (int c = 0; c < kEach; ++c) {
    const float4 v = make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
    *reinterpret_cast<uint2*>(to + 4 * (c * kChunkJoinWarps + warp)) =
        p.is_half ? make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w))
                  : make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
  if (warp == 0)
    p.lse[tok * p.heads + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace fa
