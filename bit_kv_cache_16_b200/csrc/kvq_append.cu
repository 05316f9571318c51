// kvq_append_chunk: a ragged chunk of new tokens into a cache that may already
// hold some.  The encoder is the prefill's (kvq_encode.cuh); what differs is
// where a group's tokens come from (the window ring, the chunk, or both), and
// that window slots are reused within the call.
#include "kvq_encode.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// A chunk of new tokens into a cache that may hold some already
// ---------------------------------------------------------------------------

// What a chunk does to sequence b: n, nq become n1, nq1; its rows start at
// row t0 of the chunk arrays.  m = 0 also for a chunk that is dropped (err).
struct ChunkPlan {
  int n, nq, m, n1, nq1, t0;
  uint32_t err;
};

// Every thread of the block calls this and gets the same plan: state and row
// checks here, the pages in check_pages.
__device__ __forceinline__ ChunkPlan chunk_plan(const kvq_cache& c, const int32_t* cu, int b, int total, int max_new) {
  const kvq_shape& s = c.shape;
  ChunkPlan p;
  p.t0 = cu[b];
  p.m = cu[b + 1] - p.t0;
  p.n = c.seq_len[b];
  p.nq = c.n_quant[b];
  p.err = 0u;
  if (state_bad(s, p.n, p.nq)) p.err = KVQ_DEVERR_STATE;
  else if (p.m < 0 || p.m > max_new || p.t0 < 0 || p.t0 > total - p.m) p.err = KVQ_DEVERR_PREFILL_LEN;
  else if (p.m > s.capacity - p.n) p.err = KVQ_DEVERR_APPEND_FULL;
  if (p.err) p.m = 0;
  p.n1 = p.n + p.m;
  p.nq1 = is_token_cache(s.format) ? p.n1 : max(p.nq, quantized_prefix(p.n1, s.residual, s.group));
  if (p.err) p.nq1 = p.nq;
  return p;
}

// One page per group: a bad page id drops the sequence's whole chunk.
__device__ __forceinline__ void check_pages(const kvq_cache& c, int b, ChunkPlan& p) {
  const kvq_shape& s = c.shape;
  if (s.page_size == 0 || p.nq1 <= p.nq) return;
  bool ok = true;
  const int32_t* table = c.page_table + (size_t)b * s.max_pages_per_seq;
  for (int g = p.nq / kTile + threadIdx.x; g < p.nq1 / kTile; g += blockDim.x)
    ok = ok && table[g] >= 0 && table[g] < s.num_pages;
  if (__syncthreads_and(ok)) return;
  p.err = KVQ_DEVERR_PAGE_RANGE;
  p.m = 0;
  p.n1 = p.n;
  p.nq1 = p.nq;
}

// Key and value row of new token t of (b, h) into its window slot (16-byte
// pieces e = 0 ... 15, one per thread).
__device__ __forceinline__ void ring_put(const kvq_cache& c, const uint16_t* k, const uint16_t* v, const ChunkPlan& p,
                                         int b, int h, int t, int e) {
  const kvq_shape& s = c.shape;
  const int64_t src = ((int64_t)(p.t0 + t - p.n) * s.num_kv_heads + h) * kHeadDim + 8 * e;
  const size_t dst = Addr::ring_row(s, b, h, t % window_slots(s)) + 8 * e;
  *reinterpret_cast<uint4*>((uint16_t*)c.k_res + dst) = *reinterpret_cast<const uint4*>(k + src);
  *reinterpret_cast<uint4*>((uint16_t*)c.v_res + dst) = *reinterpret_cast<const uint4*>(v + src);
}

// Grid ((groups + tail) x H_kv, B), 128 threads; the heads are neighbours in the
// grid, as their rows are in memory.  The tokens [nq1, n1) end up in
// the window, the whole groups of [nq, nq1) are quantized; a group's tokens
// come from the ring (t < n) and from the chunk (t >= n).
//  * item < groups: one group of (b, h), with the prefill's team of
//    four warps.  A window slot that held one of the group's tokens is free
//    only now: this CTA also stores the new token that takes the slot, after
//    its last read of the group (a slot's old token is always in a group that
//    this launch quantizes: t - (R + G) < nq1 for every t < n1).
//  * the others: 32 new window tokens each whose slots held nothing.
// seq_len, n_quant and the MIXED window classes are read by every CTA of the
// sequence here and change in append_chunk_commit_kernel.
// 8 x 1048 INT4 tokens (8 heads) joining 1000 each: 22 us, 44 MB (floor 6.7).
// No limit of the machine is reached (issue slots 50 %, DRAM 23 %, 30 % of the
// warps): a CTA loads, reduces, encodes and stores one group with nothing of
// the next on its way, in 2.7 waves.  65536 tokens of one sequence: 75 us, 4.6
// TB/s, 0.71 of the copy.
// FMT: 2, 4 or 6 (MIXED).
template <int FMT, int G, bool SPARSE>
__global__ void __launch_bounds__(128, SPARSE ? 5 : (G <= 32 ? 6 : 5))
    append_chunk_int_kernel(kvq_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                            const uint8_t* __restrict__ cls, const int32_t* __restrict__ cu, int total, int max_new,
                            int groups) {
  grid_dependents_launch();   // the commit kernel may be scheduled; it waits for this grid
  const kvq_shape& s = c.shape;
  const int item = blockIdx.x / s.num_kv_heads, h = blockIdx.x % s.num_kv_heads, b = blockIdx.y, tid = threadIdx.x;
  const int Ws = window_slots(s);
  ChunkPlan p = chunk_plan(c, cu, b, total, max_new);
  // A group of new tokens alone touches nothing that is in use yet, so it looks
  // at its own page only (34.8 -> 30.7 us for 16 sequences of up to 1301 tokens
  // in 16-token pages); what frees or fills window slots needs the whole chunk
  // to be good.
  const int gs = p.nq + item * G;
  const bool fresh_group = item < groups && gs >= p.n && item > 0;
  if (!fresh_group) check_pages(c, b, p);
  if (p.err && item == 0 && h == 0 && tid == 0) set_err(c.err_word, p.err);
  const int lo = max(p.n, p.nq1);                    // new window tokens: [lo, n1)
  if (item >= groups) {
    const int t = lo + 32 * (item - groups);
    for (int e = tid; e < 32 * 16; e += 128) {
      const int tt = t + e / 16;
      if (tt < p.n1 && p.nq + (tt - p.nq) % Ws >= p.n) ring_put(c, k, v, p, b, h, tt, e % 16);
    }
    return;
  }
  if (gs >= p.nq1) return;
  GroupDst d;
  if (!group_dst(c, b, h, gs / G, d)) return;        // (reported with the other pages)
  const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
  const int held = min(max(p.n - gs, 0), G);         // tokens of the group that are in the ring
  const int64_t fresh = ((int64_t)(p.t0 + gs + held - p.n) * s.num_kv_heads + h) * kHeadDim;
  bool four = FMT == 4;
  if constexpr (FMT == 6) {
    bool mine = false;
    if (tid < G)
      mine = tid < held ? c.window_class[(size_t)b * Ws + (gs + tid) % Ws] == 4 : cls[p.t0 + gs + tid - p.n] == 4;
    four = __syncthreads_or(mine) != 0;
    if (h == 0 && tid == 0) c.group_bits[(size_t)b * (s.capacity / G) + gs / G] = four ? 4 : 2;
  }
  if (held == 0) {
    const RowSrc ks{k + fresh, stride, 0, 0}, vs{v + fresh, stride, 0, 0};
    if constexpr (FMT == 6) quantize_group_mixed<G>(four, ks, vs, d);
    else quantize_group_cta<FMT, G, SPARSE>(ks, vs, d);
    return;
  }
  const uint16_t* kr = (const uint16_t*)c.k_res + Addr::ring_row(s, b, h, 0);
  const uint16_t* vr = (const uint16_t*)c.v_res + Addr::ring_row(s, b, h, 0);
  const JoinSrc ks{kr, k + fresh, stride, gs % Ws, Ws, held}, vs{vr, v + fresh, stride, gs % Ws, Ws, held};
  if constexpr (FMT == 6) quantize_group_mixed<G>(four, ks, vs, d);
  else quantize_group_cta<FMT, G, SPARSE>(ks, vs, d);
  __syncthreads();                                   // the group's slots are read for the last time
  for (int e = tid; e < held * 16; e += 128) {
    const int o = gs + e / 16;                       // the slot's old token
    int t = lo + (o - lo) % Ws;                      // the new window token of the same slot
    if (t < lo) t += Ws;
    if (t < p.n1) ring_put(c, k, v, p, b, h, t, e % 16);
  }
}

// One 16-token tile of FP8 rows (layouts as int8_token_tile): codes of tokens
// [first, valid) with the stored static scale, saturating.
template <bool KEY>
__device__ __forceinline__ void fp8_token_tile(const uint16_t* rows, int64_t stride, int first, int valid,
                                               uint8_t* codes, float inv) {
  const int lane = threadIdx.x & 31;
  const int n = lane >> 2, l = lane & 3;
  const int tok[4] = {2 * l, 2 * l + 1, 2 * l + 8, 2 * l + 9};
  uint32_t w[16];                                    // KEY: word 4q + i; else word j, byte q
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (tok[q] < first || tok[q] >= valid) continue;
    const uint16_t* r = rows + (int64_t)tok[q] * stride + 16 * n;
    const uint4 a = *reinterpret_cast<const uint4*>(r);
    const uint4 b = *reinterpret_cast<const uint4*>(r + 8);
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t e = e4m3_encode(__fmul_rn((j & 1) ? bf16_hi(x[j >> 1]) : bf16_lo(x[j >> 1]), inv));
      if (KEY) w[4 * q + (j >> 2)] |= e << (8 * (j & 3));
      else w[j] |= e << (8 * q);
    }
  }
  if (KEY) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (tok[q] >= first && tok[q] < valid)
        *reinterpret_cast<uint4*>(codes + (size_t)tok[q] * kHeadDim + 16 * n) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  } else {
    if (first > 0 || valid < kTile) merge_tile_words(w, codes, tok, first, valid);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(codes + 16 * lane + 512 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2],
                                                                          w[4 * i + 3]);
  }
}

// Grid (ceil(tiles / 2) x H_kv, B), 128 threads: the 16-token tiles that the
// chunk's tokens [n, n1) of an FP8 or INT8 cache fall into, two per CTA
// (warps 0 and 1 the key rows, warps 2 and 3 the value rows).  One warp owns
// a whole value tile, so the tokens that a partly filled first tile already
// holds are merged back without a race.
template <bool I8>
__global__ void __launch_bounds__(128, I8 ? 6 : 8)
    append_chunk_token_kernel(kvq_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                              const int32_t* __restrict__ cu, int total, int max_new) {
  grid_dependents_launch();
  const kvq_shape& s = c.shape;
  const int item = blockIdx.x / s.num_kv_heads, h = blockIdx.x % s.num_kv_heads, b = blockIdx.y;
  const int warp = threadIdx.x >> 5;
  const ChunkPlan p = chunk_plan(c, cu, b, total, max_new);
  if (p.err && blockIdx.x == 0 && threadIdx.x == 0) set_err(c.err_word, p.err);
  const int tile = p.n / kTile + 2 * item + (warp & 1);
  if (p.m == 0 || tile * kTile >= p.n1) return;
  const int first = max(p.n - tile * kTile, 0), valid = min(kTile, p.n1 - tile * kTile);
  const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
  // row of the tile's token 0 (before the chunk's first row when first > 0: never read)
  const int64_t row0 = ((int64_t)(p.t0 + tile * kTile - p.n) * s.num_kv_heads + h) * kHeadDim;
  uint8_t* kc = (uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h) + (size_t)tile * kTile * kHeadDim;
  uint8_t* vt = (uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, tile);
  if constexpr (I8) {
    __half* km = (__half*)c.k_meta + Addr::k_meta_token(s, b, h, tile * kTile);
    __half* vm = (__half*)c.v_meta + Addr::v_meta_token(s, b, h, tile * kTile);
    if (warp < 2) int8_token_tile<true, true>(k + row0, stride, valid, kc, km, first);
    else int8_token_tile<false, true>(v + row0, stride, valid, vt, vm, first);
  } else {
    if (warp < 2) fp8_token_tile<true>(k + row0, stride, first, valid, kc, __frcp_rn(c.fp8_scale[h]));
    else fp8_token_tile<false>(v + row0, stride, first, valid, vt, __frcp_rn(c.fp8_scale[s.num_kv_heads + h]));
  }
}

// Grid (B), 128 threads: after the chunk kernel, the window classes (MIXED)
// and the counters of every sequence whose chunk was taken.
__global__ void __launch_bounds__(128) append_chunk_commit_kernel(kvq_cache c, const uint8_t* __restrict__ cls,
                                                                  const int32_t* __restrict__ cu, int total,
                                                                  int max_new) {
  grid_dependency_wait();     // every CTA of the chunk kernel has read the state
  const kvq_shape& s = c.shape;
  const int b = blockIdx.x;
  ChunkPlan p = chunk_plan(c, cu, b, total, max_new);
  check_pages(c, b, p);
  if (p.err) return;
  if (is_mixed(s.format)) {
    const int Ws = window_slots(s);
    for (int t = max(p.n, p.nq1) + (int)threadIdx.x; t < p.n1; t += blockDim.x)
      c.window_class[(size_t)b * Ws + t % Ws] = cls[p.t0 + t - p.n] == 4 ? 4 : 2;
  }
  __syncthreads();            // every thread has read the counters
  if (threadIdx.x == 0) {
    c.seq_len[b] = p.n1;
    c.n_quant[b] = p.nq1;
  }
}

cudaError_t launch_append_chunk(const kvq_cache& c, const void* k, const void* v, const uint8_t* cls,
                                const int32_t* cu, int total, int max_new, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  const uint16_t* kk = (const uint16_t*)k;
  const uint16_t* vv = (const uint16_t*)v;
  const int most = min(max_new, s.capacity);         // longer chunks are rejected on the device
  if (is_token_cache(s.format)) {
    // a chunk of m tokens touches at most (m + 30) / 16 tiles
    const long long x = max(1, ((most + 2 * kTile - 2) / kTile + 1) / 2) * (long long)s.num_kv_heads;
    if (x > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    dim3 grid((unsigned)x, s.batch);
    if (is_int8(s.format)) append_chunk_token_kernel<true><<<grid, 128, 0, st>>>(c, kk, vv, cu, total, max_new);
    else append_chunk_token_kernel<false><<<grid, 128, 0, st>>>(c, kk, vv, cu, total, max_new);
  } else {
    // n - nq <= R + G and nq1 <= n1 - R: at most (G + m) / G groups; the new
    // window tokens are at most m and at most R + G
    const int groups = 1 + most / s.group;
    const int tail = (min(most, window_slots(s)) + 31) / 32;
    const long long x = (long long)(groups + tail) * s.num_kv_heads;
    if (x > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    dim3 grid((unsigned)x, s.batch);
#define KVQ_CHUNK_CASE(B, GG, SP) \
  if (s.format == B && s.group == GG && (bool)s.sparse == SP) \
    append_chunk_int_kernel<B, GG, SP><<<grid, 128, 0, st>>>(c, kk, vv, cls, cu, total, max_new, groups);
    KVQ_CHUNK_CASE(4, 16, false) KVQ_CHUNK_CASE(4, 32, false) KVQ_CHUNK_CASE(4, 64, false)
    KVQ_CHUNK_CASE(4, 128, false) KVQ_CHUNK_CASE(2, 16, false) KVQ_CHUNK_CASE(2, 32, false)
    KVQ_CHUNK_CASE(2, 64, false) KVQ_CHUNK_CASE(2, 128, false) KVQ_CHUNK_CASE(4, 16, true)
    KVQ_CHUNK_CASE(4, 32, true) KVQ_CHUNK_CASE(2, 16, true) KVQ_CHUNK_CASE(2, 32, true)
    KVQ_CHUNK_CASE(6, 32, false) KVQ_CHUNK_CASE(6, 64, false) KVQ_CHUNK_CASE(6, 128, false)
#undef KVQ_CHUNK_CASE
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.batch);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_chunk_commit_kernel, c, cls, cu, total, max_new);
}

}  // namespace kvq
