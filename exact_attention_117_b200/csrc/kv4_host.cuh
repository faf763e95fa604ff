// kv4_host.cuh -- host side of the rotary and 4-bit cache entry points:
// argument checks, kernel selection and launch.  Included by fa_api.cu.
#pragma once

#include "kv4.cuh"
#include "kv4_attend.cuh"
#include "kv4_chunk.cuh"
#include "rotary.cuh"

namespace {

bool launched() { return cudaGetLastError() == cudaSuccess; }

bool strides_multiple(const long long* s, int n, long long of) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] % of) return false;
  return true;
}

template <typename T>
fa_status rotary_typed(fa::RotaryParams p, int B, bool interleaved, cudaStream_t st) {
  // Vectors of 16 bytes where the pairs, the channels behind them and every
  // row start allow it, else single pairs (2 to 8 times the instructions; an
  // odd number of rotated pairs is the usual cause).
  constexpr int kV = 16 / static_cast<int>(sizeof(T));
  bool wide = (interleaved ? p.rot : p.rot / 2) % kV == 0 && (p.d - p.rot) % kV == 0;
  for (int w = 0; w < 2; ++w) {
    if (!p.heads[w]) continue;
    wide = wide && aligned16(p.x[w]) && aligned16(p.y[w]) &&
           strides_multiple(p.xs[w], 3, kV) && strides_multiple(p.ys[w], 3, kV);
  }
  const int vec = wide ? kV : interleaved ? 2 : 1;
  const bool in_place = p.x[0] == p.y[0] && (!p.heads[1] || p.x[1] == p.y[1]);
  p.chunks = (interleaved ? p.rot : p.rot / 2) / vec + (in_place ? 0 : (p.d - p.rot) / vec);
  // A thread takes 1, 2, 4 or 8 vectors, as many as leave three blocks an SM, and
  // a block as many positions (512 sines, 256 vectors of a head at most), so that
  // sines are computed once for several heads and a block's latencies count once
  // for several vectors (2048 tokens of 40 heads, d = 128: 10.8 us, 23.7 with one
  // vector a thread).
  const int heads = p.heads[0] + p.heads[1], pairs = p.rot / 2;
  const long long all = static_cast<long long>(B) * p.n * heads * p.chunks;
  int per = 8;
  while (per > 1 && all < per * (fa::kRotaryThreads * 148LL * 3)) per /= 2;
  p.block_pos = std::max(1, std::min({per, fa::kRotaryPairs / pairs, fa::kRotaryThreads / p.chunks, p.n}));
  p.block_rows = p.block_pos * p.chunks;
  p.block_heads = std::min(heads, per * (fa::kRotaryThreads / p.block_rows));
  p.head_groups = (heads + p.block_heads - 1) / p.block_heads;
  p.block_heads = (heads + p.head_groups - 1) / p.head_groups;
  p.pos_blocks = (p.n + p.block_pos - 1) / p.block_pos;
  const long long blocks = static_cast<long long>(B) * p.pos_blocks * p.head_groups;
  if (blocks > 0x7fffffffLL) return FA_ERR_SHAPE;
  const unsigned grid = static_cast<unsigned>(blocks);
  {
    LaunchTimer timer(st, FA_KERNEL_ROTARY);
    if (wide && interleaved)
      fa::rotary_kernel<T, kV, true><<<grid, fa::kRotaryThreads, 0, st>>>(p);
    else if (wide)
      fa::rotary_kernel<T, kV, false><<<grid, fa::kRotaryThreads, 0, st>>>(p);
    else if (interleaved)
      fa::rotary_kernel<T, 2, true><<<grid, fa::kRotaryThreads, 0, st>>>(p);
    else
      fa::rotary_kernel<T, 1, false><<<grid, fa::kRotaryThreads, 0, st>>>(p);
  }
  return launched() ? FA_OK : FA_ERR_CUDA;
}

constexpr size_t kElemSize[3] = {2, 2, 4};

// Checks shared by append and gather; fills everything but x / y.
fa_status store_params(fa::Kv4StoreParams* p, const void* k, const void* v, const void* cache,
                       const long long* slots, long long tokens, int kv_heads, int d, int pages,
                       int page_size, const long long* strides) {
  if (tokens != 0 && (!k || !v || !slots)) return FA_ERR_NULL;  // no rows: no pointers
  if (!cache || !strides) return FA_ERR_NULL;
  if (tokens < 0 || kv_heads < 1 || pages < 1 || page_size < 16 || page_size % 16)
    return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  // tile numbers and the words of a block's tokens stay inside 31 bits
  if (static_cast<long long>(pages) * page_size >= (1LL << 35) || kv_heads > (1 << 20) ||
      tokens >= (1LL << 31))
    return FA_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) || !strides_multiple(strides, 4, 8))
    return FA_ERR_ALIGN;
  p->st[0] = strides[0];
  p->sh[0] = strides[1];
  p->st[1] = strides[2];
  p->sh[1] = strides[3];
  p->slots = slots;
  p->n_slots = static_cast<long long>(pages) * page_size;
  p->tokens = tokens;
  p->heads = kv_heads;
  p->page_tiles = page_size / 16;
  p->by_page_tiles = fa::FastDiv::of(static_cast<uint32_t>(page_size / 16));
  p->lanes = std::min(2 * kv_heads * (d / 16), fa::kStoreThreads);
  p->side_by_side = fa::kStoreThreads / p->lanes;
  p->by_lanes = fa::FastDiv::of(static_cast<uint32_t>(p->lanes));
  // as many tokens a block as still leave every SM 8 blocks: 1 for a decode
  // step, up to 16 for a prompt
  p->block_tokens = static_cast<int>(
      std::max<long long>(1, std::min<long long>(fa::kStoreTokens, tokens / (8LL * 148))));
  return FA_OK;
}

// The kernel for `max_tokens` queries a request: 1 to 4 row tiles of 8 on mma
// (kv4_attend.cuh), 0: 256 rows on tcgen05 (kv4_chunk.cuh), whose time hardly
// depends on the rows below 128.  us on one B200, mma / tcgen05, 16 requests of
// 4096 keys: d = 128, 8 heads, 32 rows 68 / 95, 48 rows 109 / 95, 64 rows 112 / 95,
// 128 rows 197 / 96; d = 64, 16 heads on 4, 64 rows 44 / 48, 96 rows 55 / 49, 128
// rows 69 / 49; 4 requests of 32768 keys cross at the same rows.  (One request
// of 4096 keys leaves most of the GPU idle either way, and mma is ahead up to 128
// rows, 35 / 35 us.)  The longest request chooses for the whole call: single tokens
// beside a prompt go with it.
int attend_kind(int max_tokens, int group, int d) {
  const long long rows = static_cast<long long>(max_tokens) * group;
  if (rows >= (d == 64 ? 80 : 48)) return 0;
  return rows <= 24 ? static_cast<int>((rows + 7) / 8) : 4;
}

// The kernel that joins partial results; it may start while the kernel before it
// still runs.
fa_status launch_join(void (*kernel)(fa::Kv4AttendParams, int), int ctas, int rows, int threads,
                      const fa::Kv4AttendParams& p, cudaStream_t st) {
  LaunchTimer timer(st, FA_KERNEL_KV4_COMBINE);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), static_cast<unsigned>(rows));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, ctas) == cudaSuccess && launched() ? FA_OK : FA_ERR_CUDA;
}

// Leading units of a job (kv4_attend.cuh): two, about what a job costs besides its
// keys.  us without / with them on one B200, d = 128, H=32/8: 64 requests of 200 to
// 8192 keys 86 / 76, 256 of 100 to 2000 118 / 95, 16 of 100 to 8000 33 / 26,
// 64 of 4096 71 / 71; chunks: 1000 queries on 16384 keys and on 3000 454 / 398, one
// of 1000 queries on 1000 keys 59 / 47.  With fewer jobs than CTAs one is enough, and
// where they are far fewer hardly a CTA has more than one job to begin, and leading
// units only take CTAs from the keys (one request of 4096 keys 13.4 / 13.8).
int attend_lead(const fa::Kv4AttendParams& p, int rows, int ctas, bool chunk) {
  const long long each = (static_cast<long long>(p.tokens) * p.group + p.requests - 1) / p.requests;
  const long long jobs = (each + rows - 1) / rows * p.requests * p.kv_heads;
  return jobs * 8 < ctas ? 0 : jobs < ctas && !chunk ? 1 : 2;
}

template <int D, int NT>
fa_status launch_attend(fa::Kv4AttendParams p, cudaStream_t st) {
  using L = fa::Kv4AttendLayout<D, NT>;
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  if (!attr_set[dev]) {
    if (!set_smem(fa::kv4_attend_kernel<D, NT>, L::kBytes)) return FA_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int ctas = sm_count(dev) * L::kCtas;
  p.lead = attend_lead(p, L::kRows, ctas, false);
  {
    LaunchTimer timer(st, FA_KERNEL_KV4_ATTEND);
    fa::kv4_attend_kernel<D, NT><<<ctas, fa::kKv4Warps * 32, L::kBytes, st>>>(p);
    if (!launched()) return FA_ERR_CUDA;
  }
  return launch_join(fa::kv4_combine_kernel<D, NT>, ctas, 2 * NT, fa::kKv4Warps * 32, p, st);
}

template <int D>
fa_status launch_chunk(fa::Kv4AttendParams p, cudaStream_t st) {
  using L = fa::Kv4ChunkLayout<D>;
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  if (!attr_set[dev]) {
    if (!set_smem(fa::kv4_chunk_kernel<D>, L::kSmemAlloc)) return FA_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int ctas = sm_count(dev);
  p.lead = attend_lead(p, fa::kChunkRows, ctas, true);
  {
    LaunchTimer timer(st, FA_KERNEL_KV4_ATTEND);
    fa::kv4_chunk_kernel<D><<<ctas, fa::kChunkWarps * 32, L::kSmemAlloc, st>>>(p);
    if (!launched()) return FA_ERR_CUDA;
  }
  return launch_join(fa::kv4_chunk_combine_kernel<D>, ctas, fa::kChunkRows / 32, fa::kChunkJoinWarps * 32, p, st);
}

// Workspace: two partial results a CTA, then (kind 0) a Kv4Cut a CTA.
struct AttendWorkspace {
  size_t cuts_at, bytes;
};
AttendWorkspace attend_workspace(int d, int kind) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  // CTAs an SM: kCtas of the layouts (up to 4, or 3 for more rows)
  const size_t ctas = static_cast<size_t>(sm_count(dev)) * (kind == 1 ? 4 : kind ? 3 : 1);
  const size_t rows = kind ? 8 * kind : fa::kChunkRows;
  const size_t part = 2 * ctas * rows * (d + 2) * sizeof(float);
  return {part, part + (kind ? 0 : ctas * sizeof(fa::Kv4Cut))};
}

}  // namespace

extern "C" {

fa_status fa_rotary(const void* q, const void* k, void* q_out, void* k_out, int B, int q_heads,
                    int k_heads, int N, int d, const long long* strides, const void* positions,
                    int positions_64, long long position_stride, const double* inv_freq,
                    int rotary_dim, int interleaved, float amplitude, int inverse, int dtype,
                    void* stream) {
  if (!inv_freq || !strides) return FA_ERR_NULL;
  if (N != 0 && (!q || !q_out || !positions)) return FA_ERR_NULL;  // no rows: no pointers
  if (N != 0 && k_heads > 0 && (!k || !k_out)) return FA_ERR_NULL;
  if (B < 1 || q_heads < 1 || k_heads < 0 || N < 0 || position_stride < 0) return FA_ERR_SHAPE;
  if (static_cast<long long>(B) * N > (1LL << 31) || q_heads > (1 << 20) || k_heads > (1 << 20))
    return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  if (rotary_dim < 2 || rotary_dim > d || rotary_dim % 2 || dtype < 0 || dtype > 2)
    return FA_ERR_SHAPE;
  if (!std::isfinite(amplitude)) return FA_ERR_SCALE;
  const uintptr_t el = kElemSize[dtype];
  // neighbouring pairs are read as one access of two elements
  const uintptr_t unit = interleaved ? 2 * el : el;
  const void* ptrs[4] = {q, q_out, k_heads ? k : q, k_heads ? k_out : q_out};
  for (const void* x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % unit) return FA_ERR_ALIGN;
  if (!strides_multiple(strides, k_heads ? 12 : 6, interleaved ? 2 : 1) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
      (reinterpret_cast<uintptr_t>(positions) & (positions_64 ? 7u : 3u)))
    return FA_ERR_ALIGN;
  if (N == 0) return FA_OK;
  // an output that is its input lies as the input does
  const long long sizes[2][3] = {{B, q_heads, N}, {B, k_heads, N}};
  for (int w = 0; w < (k_heads ? 2 : 1); ++w)
    for (int i = 0; i < 3; ++i)
      if (ptrs[2 * w] == ptrs[2 * w + 1] && sizes[w][i] > 1 &&
          strides[6 * w + i] != strides[6 * w + 3 + i])
        return FA_ERR_SHAPE;
  fa::RotaryParams p = {};
  p.x[0] = q;
  p.x[1] = k;
  p.y[0] = q_out;
  p.y[1] = k_out;
  for (int i = 0; i < 3; ++i) {
    p.xs[0][i] = strides[i];
    p.ys[0][i] = strides[3 + i];
    p.xs[1][i] = k_heads ? strides[6 + i] : 0;
    p.ys[1][i] = k_heads ? strides[9 + i] : 0;
  }
  p.heads[0] = q_heads;
  p.heads[1] = k_heads;
  p.positions = positions;
  p.pos64 = positions_64 != 0;
  p.pos_stride = position_stride;
  p.inv_freq = inv_freq;
  p.n = N;
  p.rot = rotary_dim;
  p.d = d;
  p.amplitude = amplitude;
  p.sin_sign = inverse ? -1.f : 1.f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == FA_BF16) return rotary_typed<__nv_bfloat16>(p, B, interleaved != 0, s);
  if (dtype == FA_FP16) return rotary_typed<__half>(p, B, interleaved != 0, s);
  return rotary_typed<float>(p, B, interleaved != 0, s);
}

size_t fa_kv4_cache_size(int pages, int kv_heads, int page_size, int d) {
  if (pages < 1 || kv_heads < 1 || page_size < 16 || page_size % 16 || (d != 64 && d != 128))
    return 0;
  return static_cast<size_t>(pages) * kv_heads * (page_size / 16) * 18 * d;
}

fa_status fa_kv4_plan(const int* lengths, const int* new_lengths, int* block_table,
                      long long table_stride, int width, int* free_pages, int ring_size,
                      const long long* free_range, int requests, int page_size, int max_tokens,
                      int* lengths_out, long long* free_range_out, int* cu_tokens,
                      long long* slots, int* positions, int* status, void* stream) {
  if (!lengths || !new_lengths || !block_table || !free_pages || !free_range || !lengths_out ||
      !free_range_out || !cu_tokens || !status || (max_tokens > 0 && (!slots || !positions)))
    return FA_ERR_NULL;
  if (requests < 1 || width < 1 || ring_size < 1 || page_size < 16 || page_size % 16 ||
      max_tokens < 0 || max_tokens > (1 << 30) || table_stride < width)
    return FA_ERR_SHAPE;
  if (static_cast<long long>(requests) * width > (1LL << 30) || requests > (1 << 30) ||
      static_cast<long long>(width) * page_size > (1LL << 30) || page_size > (1 << 30) ||
      ring_size > (1 << 30))
    return FA_ERR_SHAPE;
  const void* four[8] = {lengths, new_lengths, block_table, free_pages, lengths_out, cu_tokens,
                         positions, status};
  for (const void* x : four)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(free_range) & 7u) ||
      (reinterpret_cast<uintptr_t>(free_range_out) & 7u) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return FA_ERR_ALIGN;
  fa::Kv4PlanParams p = {};
  p.old_len = lengths;
  p.new_len = new_lengths;
  p.table = block_table;
  p.ring = free_pages;
  p.range = free_range;
  p.out_len = lengths_out;
  p.out_range = free_range_out;
  p.cu_tokens = cu_tokens;
  p.slots = slots;
  p.positions = positions;
  p.status = status;
  p.table_stride = table_stride;
  p.requests = requests;
  p.width = width;
  p.page_size = page_size;
  p.ring_size = ring_size;
  p.max_tokens = max_tokens;
  p.by_page = fa::FastDiv::of(static_cast<uint32_t>(page_size));
  // one CTA writes a few thousand tokens as fast as the launch of more takes
  const unsigned ctas = max_tokens > 2 * fa::kPlanThreads ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(fa::kPlanThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchTimer timer(cfg.stream, FA_KERNEL_KV4_PLAN);
  return cudaLaunchKernelEx(&cfg, fa::kv4_plan_kernel, p) == cudaSuccess && launched() ? FA_OK
                                                                                       : FA_ERR_CUDA;
}

fa_status fa_kv4_append(const void* k, const void* v, void* cache, const long long* slots,
                        long long tokens, int kv_heads, int d, int pages, int page_size,
                        const long long* strides, void* stream) {
  fa::Kv4StoreParams p = {};
  fa_status r = store_params(&p, k, v, cache, slots, tokens, kv_heads, d, pages, page_size, strides);
  if (r != FA_OK || tokens == 0) return r;
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.cache = static_cast<uint8_t*>(cache);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>((tokens + p.block_tokens - 1) / p.block_tokens);
  LaunchTimer timer(s, FA_KERNEL_KV4_APPEND);
  if (d == 64)
    fa::kv4_append_kernel<64><<<blocks, fa::kStoreThreads, 0, s>>>(p);
  else
    fa::kv4_append_kernel<128><<<blocks, fa::kStoreThreads, 0, s>>>(p);
  return launched() ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_kv4_gather(const void* cache, const long long* slots, void* k, void* v,
                        long long tokens, int kv_heads, int d, int pages, int page_size,
                        const long long* strides, void* stream) {
  fa::Kv4StoreParams p = {};
  fa_status r = store_params(&p, k, v, cache, slots, tokens, kv_heads, d, pages, page_size, strides);
  if (r != FA_OK || tokens == 0) return r;
  p.y[0] = static_cast<__nv_bfloat16*>(k);
  p.y[1] = static_cast<__nv_bfloat16*>(v);
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>((tokens + p.block_tokens - 1) / p.block_tokens);
  LaunchTimer timer(s, FA_KERNEL_KV4_GATHER);
  if (d == 64)
    fa::kv4_gather_kernel<64><<<blocks, fa::kStoreThreads, 0, s>>>(p);
  else
    fa::kv4_gather_kernel<128><<<blocks, fa::kStoreThreads, 0, s>>>(p);
  return launched() ? FA_OK : FA_ERR_CUDA;
}

size_t fa_kv4_attention_workspace_size(int heads, int kv_heads, int d, int max_tokens) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads || (d != 64 && d != 128) || max_tokens < 1)
    return 0;
  return attend_workspace(d, attend_kind(max_tokens, heads / kv_heads, d)).bytes;
}

fa_status fa_kv4_attention(const void* q, const void* cache, const int* block_table,
                           const int* lengths, const int* cu_tokens, void* o, float* lse,
                           int requests, int tokens, int heads, int kv_heads, int d, int pages,
                           int page_size, int width, long long table_stride,
                           const long long* strides, int max_tokens, int causal, float scale,
                           int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !block_table || !lengths || !cu_tokens || !strides) return FA_ERR_NULL;
  if (tokens != 0 && (!q || !o || !lse)) return FA_ERR_NULL;  // no rows: no pointers
  if (requests < 1 || tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || pages < 1 ||
      page_size < 16 || page_size % 16 || width < 1 || table_stride < width || max_tokens < 1)
    return FA_ERR_SHAPE;
  if (static_cast<long long>(tokens) * heads > 0x7fffffffLL - 1024 ||
      static_cast<long long>(width) * page_size > 0x7fffffffLL - 1024 ||
      (dtype != FA_BF16 && dtype != FA_FP16))
    return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_D;
  if (!std::isfinite(scale)) return FA_ERR_SCALE;
  const void* four[4] = {block_table, lengths, cu_tokens, lse};
  for (const void* x : four)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return FA_ERR_ALIGN;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !strides_multiple(strides, 4, 8))
    return FA_ERR_ALIGN;
  const int kind = attend_kind(max_tokens, heads / kv_heads, d);
  const AttendWorkspace ws = attend_workspace(d, kind);
  if (!workspace || workspace_bytes < ws.bytes) return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_ALIGN;
  if (tokens == 0) return FA_OK;
  fa::Kv4AttendParams p = {};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = block_table;
  p.lengths = lengths;
  p.cu_tokens = cu_tokens;
  p.part = static_cast<float*>(workspace);
  p.part_floats = static_cast<long long>(ws.cuts_at / sizeof(float));
  p.cuts = reinterpret_cast<fa::Kv4Cut*>(static_cast<char*>(workspace) + ws.cuts_at);
  p.q_st = strides[0];
  p.q_sh = strides[1];
  p.o_st = strides[2];
  p.o_sh = strides[3];
  p.table_stride = table_stride;
  p.requests = requests;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.tokens = tokens;
  p.pages = pages;
  p.page_size = page_size;
  p.width = width;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.causal = causal != 0;
  p.is_half = dtype == FA_FP16;
  p.limit_ns = kWaitLimitNs;
  p.page_tiles = fa::FastDiv::of(static_cast<uint32_t>(page_size / 16));
  p.by_group = fa::FastDiv::of(static_cast<uint32_t>(p.group));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (d == 64 ? kind : 8 + kind) {
    case 0: return launch_chunk<64>(p, s);
    case 1: return launch_attend<64, 1>(p, s);
    case 2: return launch_attend<64, 2>(p, s);
    case 3: return launch_attend<64, 3>(p, s);
    case 4: return launch_attend<64, 4>(p, s);
    case 8: return launch_chunk<128>(p, s);
    case 9: return launch_attend<128, 1>(p, s);
    case 10: return launch_attend<128, 2>(p, s);
    case 11: return launch_attend<128, 3>(p, s);
    default: return launch_attend<128, 4>(p, s);
  }
}

}  // extern "C"
