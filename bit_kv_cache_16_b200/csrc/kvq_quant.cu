// Write side of the cache: prefill quantization, append, flush (INT2/INT4),
// and the FP8-E4M3 comparison cache.
//
// INT prefill and flush: one CTA of four warps quantizes one block of
// TB = max(G, 32) tokens of one (sequence, kv head).
// The four warps' roles and the encoder's arithmetic are in kvq_encode.cuh.
#include "kvq_encode.cuh"

namespace kvq {

// Grid (ceil(max_len / TB), H_kv, B), 128 threads; TB = max(G, 32) tokens
// per CTA (two key groups when G = 16, one value warp per group).
// Registers are cut for 8 CTAs per SM at G = 16 and 32 (64 registers,
// some spill; more CTAs keep more of the short per-CTA loads in flight).
// Means of 20 calls: the paged ragged batch (G = 16) 1585 us at 5 CTAs,
// 1432 at 6, 1353 at 7, 1260 at 8, 1602 at 10, 1943 at 12; the 8B layer
// (G = 32) 78.0 us at 6 against 71.5 at 8, the 70B layer 134.6 against
// 124.5 (INT4) and 133.6 against 128.4 (INT2).  The dense-and-sparse
// kernel keeps 6 at G = 32 (5 or 8 were slower) and 5 at G = 16; G = 64
// and 128 keep 5 (no spill).
template <int BITS, int G, bool SPARSE>
__global__ void __launch_bounds__(128, SPARSE ? (G == 32 ? 6 : 5) : ((G == 16 || G == 32) ? 8 : 5)) prefill_int_kernel(kvq_cache c, const uint16_t* __restrict__ k,
                                                          const uint16_t* __restrict__ v,
                                                          const int32_t* __restrict__ cu, int max_len) {
  constexpr int TB = G < 32 ? 32 : G;
  const kvq_shape& s = c.shape;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int Ws = window_slots(s);
  const int t0 = cu[b];
  int n = cu[b + 1] - t0;
  const bool too_long = n > s.capacity || n < 0 || n > max_len;
  if (too_long) n = 0;
  const int nq = quantized_prefix(n, s.residual, G);
  if (blk == 0 && h == 0 && threadIdx.x == 0) {
    c.seq_len[b] = n;
    c.n_quant[b] = nq;
    if (too_long) set_err(c.err_word, KVQ_DEVERR_PREFILL_LEN);
  }
  const int tb0 = blk * TB;
  if (tb0 >= n) return;
  const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
  bool page_bad = false;
  if constexpr (G == 16 && !SPARSE) {
    // the block's two 16-token groups: each key warp loads both groups'
    // words before quantizing either (twice the loads in flight); value
    // warp 2 + gi takes group gi's tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    GroupDst d[2];
    bool ok[2] = {false, false};
#pragma unroll
    for (int gi = 0; gi < 2; ++gi) {
      const int g = 2 * blk + gi;
      if ((g + 1) * G > nq) break;
      ok[gi] = group_dst(c, b, h, g, d[gi]);
      page_bad = page_bad || !ok[gi];
    }
    if (warp < 2) {
      const int p = 32 * warp + lane;
      uint32_t x0[16], x1[16];
      const uint16_t* r0 = k + ((int64_t)(t0 + 32 * blk) * s.num_kv_heads + h) * kHeadDim + 2 * p;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x0[i] = ok[0] ? *reinterpret_cast<const uint32_t*>(r0 + i * stride) : 0u;
        x1[i] = ok[1] ? *reinterpret_cast<const uint32_t*>(r0 + (16 + i) * stride) : 0u;
      }
      if (ok[0]) k_group_x<BITS, 16>(x0, p, d[0].k_codes, d[0].k_meta);
      if (ok[1]) k_group_x<BITS, 16>(x1, p, d[1].k_codes, d[1].k_meta);
    } else if (ok[warp - 2]) {
      const int gi = warp - 2;
      const RowSrc vs{v + ((int64_t)(t0 + 32 * blk + 16 * gi) * s.num_kv_heads + h) * kHeadDim, stride, 0, 0};
      v_tile<BITS>(vs, 0, d[gi].v_tiles, d[gi].v_meta);
    }
  } else {
#pragma unroll 1
  for (int gi = 0; gi < TB / G; ++gi) {
    const int g = blk * (TB / G) + gi;
    if ((g + 1) * G > nq) break;
    GroupDst d;
    if (!group_dst(c, b, h, g, d)) {
      page_bad = true;
      continue;
    }
    const RowSrc ks{k + ((int64_t)(t0 + g * G) * s.num_kv_heads + h) * kHeadDim, stride, 0, 0};
    const RowSrc vs{v + ((int64_t)(t0 + g * G) * s.num_kv_heads + h) * kHeadDim, stride, 0, 0};
    if (G == 16) {
      // a 16-token group has one value tile: value warp 2 + gi takes group
      // gi's, so both value warps work while the key warps take both groups
      const int warp = threadIdx.x >> 5;
      if constexpr (SPARSE) {
        if (warp < 2) k_group_sparse<BITS, 16>(ks, 32 * warp + (threadIdx.x & 31), d.k_codes, d.k_meta, d.k_sparse);
        else if (warp - 2 == gi) v_tile_sparse<BITS>(vs, 0, d.v_tiles, d.v_meta, d.v_sparse);
      } else {
        if (warp < 2) k_group<BITS, G>(ks, 32 * warp + (threadIdx.x & 31), d.k_codes, d.k_meta);
        else if (warp - 2 == gi) v_tile<BITS>(vs, 0, d.v_tiles, d.v_meta);
      }
    } else {
      quantize_group_cta<BITS, G, SPARSE>(ks, vs, d);
    }
  }
  }
  if (page_bad && threadIdx.x == 0) set_err(c.err_word, KVQ_DEVERR_PAGE_RANGE);
  // window tokens of this block -> ring slots t mod (R + G)
  const int lo = max(tb0, nq), hi = min(tb0 + TB, n);
  uint16_t* kr = (uint16_t*)c.k_res;
  uint16_t* vr = (uint16_t*)c.v_res;
  for (int e = threadIdx.x; e < (hi - lo) * 16; e += blockDim.x) {
    const int t = lo + e / 16, piece = e % 16;
    const int64_t src = ((int64_t)(t0 + t) * s.num_kv_heads + h) * kHeadDim + piece * 8;
    const size_t dst = Addr::ring_row(s, b, h, t % Ws) + piece * 8;
    *reinterpret_cast<uint4*>(kr + dst) = *reinterpret_cast<const uint4*>(k + src);
    *reinterpret_cast<uint4*>(vr + dst) = *reinterpret_cast<const uint4*>(v + src);
  }
}

// Grid (H_kv, B), 128 threads: quantizes the oldest G window tokens of
// (b, h) when the window of sequence b holds R + G tokens.  n_quant is left
// alone here (other heads' CTAs of the sequence still read it);
// flush_commit_kernel, next on the stream, advances it.
template <int BITS, int G, bool SPARSE>
__global__ void __launch_bounds__(128) flush_int_kernel(kvq_cache c) {
  grid_dependents_launch();   // the commit kernel may be scheduled; it waits for this grid
  const kvq_shape& s = c.shape;
  const int h = blockIdx.x, b = blockIdx.y;
  const int Ws = window_slots(s);
  const int n = c.seq_len[b], nq = c.n_quant[b];
  if (n - nq != Ws) return;
  if (nq < 0 || nq + G > s.capacity || nq % G) {
    if (threadIdx.x == 0 && h == 0) set_err(c.err_word, KVQ_DEVERR_STATE);
    return;
  }
  GroupDst d;
  if (!group_dst(c, b, h, nq / G, d)) {
    if (threadIdx.x == 0) set_err(c.err_word, KVQ_DEVERR_PAGE_RANGE);
    return;
  }
  const RowSrc ks{(const uint16_t*)c.k_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
  const RowSrc vs{(const uint16_t*)c.v_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
  quantize_group_cta<BITS, G, SPARSE>(ks, vs, d);
}

// Grid (B), 32 threads: after flush_int_kernel, advance n_quant of every
// sequence whose window was full and whose group pages were all valid.
__global__ void flush_commit_kernel(kvq_cache c) {
  grid_dependency_wait();     // every flush CTA has read n_quant and written its group
  const kvq_shape& s = c.shape;
  const int b = blockIdx.x;
  const int G = s.group, Ws = window_slots(s);
  const int n = c.seq_len[b], nq = c.n_quant[b];
  if (n - nq != Ws || nq < 0 || nq + G > s.capacity || nq % G) return;
  bool ok = true;
  if (s.page_size != 0) {
    const int page = c.page_table[(size_t)b * s.max_pages_per_seq + nq / G];
    ok = page >= 0 && page < s.num_pages;
  }
  if (ok && threadIdx.x == 0) c.n_quant[b] = nq + G;
}

// Grid (B); block H_kv * 32 threads.  INT formats: token -> window slot
// (MIXED: cls[b], the token's class, into window_class).
__global__ void append_int_kernel(kvq_cache c, const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn,
                                  const uint8_t* __restrict__ cls) {
  const kvq_shape& s = c.shape;
  const int b = blockIdx.x;
  const int n = c.seq_len[b], nq = c.n_quant[b];
  const int Ws = window_slots(s);
  if (n >= s.capacity || n - nq >= Ws || n < nq) {
    if (threadIdx.x == 0) set_err(c.err_word, KVQ_DEVERR_APPEND_FULL);
    return;
  }
  uint16_t* kr = (uint16_t*)c.k_res;
  uint16_t* vr = (uint16_t*)c.v_res;
  for (int e = threadIdx.x; e < s.num_kv_heads * 16; e += blockDim.x) {
    const int h = e / 16, piece = e % 16;
    const size_t src = ((size_t)b * s.num_kv_heads + h) * kHeadDim + piece * 8;
    const size_t dst = Addr::ring_row(s, b, h, n % Ws) + piece * 8;
    *reinterpret_cast<uint4*>(kr + dst) = *reinterpret_cast<const uint4*>(kn + src);
    *reinterpret_cast<uint4*>(vr + dst) = *reinterpret_cast<const uint4*>(vn + src);
  }
  if (cls && threadIdx.x == 0) c.window_class[(size_t)b * Ws + n % Ws] = cls[b] == 4 ? 4 : 2;
  __syncthreads();
  if (threadIdx.x == 0) c.seq_len[b] = n + 1;
}

// Grid (H_kv, B) in clusters of (H_kv, 1): the CTAs of one sequence form a
// cluster.  Append, then flush when due, in one launch: CTA (h, b) writes the
// new token of kv head h to window slot seq_len mod (R + G); if the window
// now holds R + G tokens it quantizes the oldest G of them (the same group
// kvq_flush_group would take); after a cluster barrier (every CTA of the
// sequence has read seq_len and n_quant) CTA 0 advances seq_len and, after a
// flush, n_quant.  The states, codes and errors equal those of
// kvq_append_token followed by kvq_flush_group.
template <int BITS, int G, bool SPARSE>
__global__ void __launch_bounds__(128) append_flush_int_kernel(kvq_cache c, const uint16_t* __restrict__ kn,
                                                               const uint16_t* __restrict__ vn) {
  const kvq_shape& s = c.shape;
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  const int Ws = window_slots(s);
  // the new token's row is loaded first: its address does not depend on the
  // state, so both loads are in flight together
  const int piece = t & 15;
  uint4 row = make_uint4(0u, 0u, 0u, 0u);
  if (t < 32)
    row = *reinterpret_cast<const uint4*>((t < 16 ? kn : vn) + ((size_t)b * s.num_kv_heads + h) * kHeadDim + piece * 8);
  const int n = c.seq_len[b], nq = c.n_quant[b];
  // append (as kvq_append_token)
  const bool appended = !(n >= s.capacity || n - nq >= Ws || n < nq);
  if (appended) {
    if (t < 32) {
      const size_t dst = Addr::ring_row(s, b, h, n % Ws) + piece * 8;
      *reinterpret_cast<uint4*>((uint16_t*)(t < 16 ? c.k_res : c.v_res) + dst) = row;
    }
  } else if (t == 0 && h == 0) {
    set_err(c.err_word, KVQ_DEVERR_APPEND_FULL);
  }
  // flush (as kvq_flush_group, on the state after the append)
  const int n1 = appended ? n + 1 : n;
  bool flushed = false;
  if (n1 - nq == Ws) {
    if (nq < 0 || nq + G > s.capacity || nq % G) {
      if (t == 0 && h == 0) set_err(c.err_word, KVQ_DEVERR_STATE);
    } else {
      GroupDst d;
      if (!group_dst(c, b, h, nq / G, d)) {
        if (t == 0) set_err(c.err_word, KVQ_DEVERR_PAGE_RANGE);
      } else {
        __syncthreads();   // the appended row is visible to the whole team
        const RowSrc ks{(const uint16_t*)c.k_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
        const RowSrc vs{(const uint16_t*)c.v_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
        quantize_group_cta<BITS, G, SPARSE>(ks, vs, d);
        flushed = true;   // the page is the sequence's, so every CTA of the cluster agrees
      }
    }
  }
  // every CTA of the sequence has read seq_len and n_quant before they change
  // (the reads have returned: their values decided the branches above, so a
  // relaxed arrive orders them; the ring and group writes need no ordering
  // against the state update within this launch, the next launch sees them all)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  if (h == 0 && t == 0) {
    if (appended) c.seq_len[b] = n1;
    if (flushed) c.n_quant[b] = nq + G;
  }
}

// ---------------------------------------------------------------------------
// FP8-E4M3 cache
// ---------------------------------------------------------------------------

// Grid (ceil(max_len/64), H_kv, B): amax |x| over a 64-token chunk of one kv
// head, folded into fp8_amax[0|1][h] (non-negative floats order like their bits).
__global__ void fp8_amax_kernel(kvq_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                                const int32_t* __restrict__ cu, int max_len) {
  const kvq_shape& s = c.shape;
  const int h = blockIdx.y, b = blockIdx.z;
  const int t0 = cu[b];
  const int n = cu[b + 1] - t0;
  if (n > s.capacity || n < 0 || n > max_len) return;
  float ak = 0.f, av = 0.f;
  const int lo = blockIdx.x * 64, hi = min(lo + 64, n);
  for (int e = threadIdx.x; e < (hi - lo) * 16; e += blockDim.x) {
    const int t = lo + e / 16, piece = e % 16;
    const int64_t off = ((int64_t)(t0 + t) * s.num_kv_heads + h) * kHeadDim + piece * 8;
    const uint4 a = *reinterpret_cast<const uint4*>(k + off);
    const uint4 bb = *reinterpret_cast<const uint4*>(v + off);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {bb.x, bb.y, bb.z, bb.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      ak = fmaxf(ak, fmaxf(fabsf(bf16_lo(wa[p])), fabsf(bf16_hi(wa[p]))));
      av = fmaxf(av, fmaxf(fabsf(bf16_lo(wb[p])), fabsf(bf16_hi(wb[p]))));
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, off));
    av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, off));
  }
  if ((threadIdx.x & 31) == 0 && hi > lo) {
    atomicMax(&c.fp8_amax[h], __float_as_uint(ak));
    atomicMax(&c.fp8_amax[s.num_kv_heads + h], __float_as_uint(av));
  }
}

__device__ __forceinline__ void fp8_write_words(const kvq_cache& c, int b, int h, int t, uint2 kx, uint2 vx,
                                                float inv_k, float inv_v, int lane) {
  // lane handles channels 4*lane .. 4*lane+3 (kx, vx: their bf16 words)
  const kvq_shape& s = c.shape;
  const float kf[4] = {bf16_lo(kx.x), bf16_hi(kx.x), bf16_lo(kx.y), bf16_hi(kx.y)};
  const float vf[4] = {bf16_lo(vx.x), bf16_hi(vx.x), bf16_lo(vx.y), bf16_hi(vx.y)};
  uint32_t kw = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) kw |= e4m3_encode(__fmul_rn(kf[i], inv_k)) << (8 * i);
  uint8_t* kc = (uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h) + (size_t)t * kHeadDim;
  *reinterpret_cast<uint32_t*>(kc + 4 * lane) = kw;
  uint8_t* vt = (uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, t / kTile);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    vt[fp8_vtile_offset(t % kTile, 4 * lane + i)] = (uint8_t)e4m3_encode(__fmul_rn(vf[i], inv_v));
}

__device__ __forceinline__ void fp8_write_token(const kvq_cache& c, int b, int h, int t, const uint16_t* krow,
                                                const uint16_t* vrow, float inv_k, float inv_v, int lane) {
  fp8_write_words(c, b, h, t, *reinterpret_cast<const uint2*>(krow + 4 * lane),
                  *reinterpret_cast<const uint2*>(vrow + 4 * lane), inv_k, inv_v, lane);
}

// Grid (ceil(max_len/16), H_kv, B); block 16 warps: warp i encodes token
// 16*blockIdx.x + i (zeros for tokens past the end of the sequence).
__global__ void __launch_bounds__(512) fp8_prefill_kernel(kvq_cache c, const uint16_t* __restrict__ k,
                                                          const uint16_t* __restrict__ v,
                                                          const int32_t* __restrict__ cu, int max_len) {
  const kvq_shape& s = c.shape;
  const int tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int t0 = cu[b];
  int n = cu[b + 1] - t0;
  const bool too_long = n > s.capacity || n < 0 || n > max_len;
  if (too_long) n = 0;
  const float Sk = fp8_scale_from_amax(__uint_as_float(c.fp8_amax[h]));
  const float Sv = fp8_scale_from_amax(__uint_as_float(c.fp8_amax[s.num_kv_heads + h]));
  if (tile == 0 && threadIdx.x == 0) {
    if (b == 0) {
      c.fp8_scale[h] = Sk;
      c.fp8_scale[s.num_kv_heads + h] = Sv;
    }
    if (h == 0) {
      c.seq_len[b] = n;
      c.n_quant[b] = n;
      if (too_long) set_err(c.err_word, KVQ_DEVERR_PREFILL_LEN);
    }
  }
  if (tile * kTile >= n) return;
  const float inv_k = __frcp_rn(Sk), inv_v = __frcp_rn(Sv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = tile * kTile + warp;
  if (t < n) {
    const int64_t off = ((int64_t)(t0 + t) * s.num_kv_heads + h) * kHeadDim;
    fp8_write_token(c, b, h, t, k + off, v + off, inv_k, inv_v, lane);
  } else {
    uint8_t* vt = (uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, tile);
#pragma unroll
    for (int i = 0; i < 4; ++i) vt[fp8_vtile_offset(t % kTile, 4 * lane + i)] = 0;
  }
}

// Grid (B); block H_kv warps.
__global__ void fp8_append_kernel(kvq_cache c, const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn) {
  const kvq_shape& s = c.shape;
  const int b = blockIdx.x;
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the new rows and the head's scales do not depend on the state: their
  // loads are issued with the state's
  uint2 kx = make_uint2(0u, 0u), vx = make_uint2(0u, 0u);
  float Sk = 1.f, Sv = 1.f;
  if (h < s.num_kv_heads) {
    const size_t off = ((size_t)b * s.num_kv_heads + h) * kHeadDim;
    kx = *reinterpret_cast<const uint2*>(kn + off + 4 * lane);
    vx = *reinterpret_cast<const uint2*>(vn + off + 4 * lane);
    Sk = c.fp8_scale[h];
    Sv = c.fp8_scale[s.num_kv_heads + h];
  }
  const int n = c.seq_len[b];
  if (n >= s.capacity || n < 0) {
    if (threadIdx.x == 0) set_err(c.err_word, KVQ_DEVERR_APPEND_FULL);
    return;
  }
  if (h < s.num_kv_heads) fp8_write_words(c, b, h, n, kx, vx, __frcp_rn(Sk), __frcp_rn(Sv), lane);
  __syncthreads();
  if (threadIdx.x == 0) {
    c.seq_len[b] = n + 1;
    c.n_quant[b] = n + 1;
  }
}

// ---------------------------------------------------------------------------
// MIXED cache: INT4 or INT2 per group by the classes of its tokens
// ---------------------------------------------------------------------------

// Grid (ceil(max_len / G), H_kv, B), 128 threads: one group per CTA (G >= 32),
// stored at 4 bits if any of its tokens has class 4, else at 2; then the
// block's window tokens and their classes.  Registers are cut for 7 CTAs
// per SM (72 registers, some spill): 73.8 against 82.1 us at 5 on the 8B
// layer, no better at 8 or 10.
template <int G>
__global__ void __launch_bounds__(128, 7) prefill_mixed_kernel(kvq_cache c, const uint16_t* __restrict__ k,
                                                               const uint16_t* __restrict__ v,
                                                               const uint8_t* __restrict__ cls,
                                                               const int32_t* __restrict__ cu, int max_len) {
  static_assert(G >= 32, "one group per CTA");
  const kvq_shape& s = c.shape;
  const int g = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int Ws = window_slots(s);
  const int t0 = cu[b];
  int n = cu[b + 1] - t0;
  const bool too_long = n > s.capacity || n < 0 || n > max_len;
  if (too_long) n = 0;
  const int nq = quantized_prefix(n, s.residual, G);
  if (g == 0 && h == 0 && threadIdx.x == 0) {
    c.seq_len[b] = n;
    c.n_quant[b] = nq;
    if (too_long) set_err(c.err_word, KVQ_DEVERR_PREFILL_LEN);
  }
  const int tb0 = g * G;
  if (tb0 >= n) return;
  if ((g + 1) * G <= nq) {
    const bool four = __syncthreads_or(threadIdx.x < G && cls[t0 + tb0 + threadIdx.x] == 4) != 0;
    if (h == 0 && threadIdx.x == 0) c.group_bits[(size_t)b * (s.capacity / G) + g] = four ? 4 : 2;
    GroupDst d;
    group_dst(c, b, h, g, d);     // contiguous: always valid
    const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
    const RowSrc ks{k + ((int64_t)(t0 + tb0) * s.num_kv_heads + h) * kHeadDim, stride, 0, 0};
    const RowSrc vs{v + ((int64_t)(t0 + tb0) * s.num_kv_heads + h) * kHeadDim, stride, 0, 0};
    quantize_group_mixed<G>(four, ks, vs, d);
  }
  // window tokens of this block -> ring slots t mod (R + G), with their classes
  const int lo = max(tb0, nq), hi = min(tb0 + G, n);
  uint16_t* kr = (uint16_t*)c.k_res;
  uint16_t* vr = (uint16_t*)c.v_res;
  for (int e = threadIdx.x; e < (hi - lo) * 16; e += blockDim.x) {
    const int t = lo + e / 16, piece = e % 16;
    const int64_t src = ((int64_t)(t0 + t) * s.num_kv_heads + h) * kHeadDim + piece * 8;
    const size_t dst = Addr::ring_row(s, b, h, t % Ws) + piece * 8;
    *reinterpret_cast<uint4*>(kr + dst) = *reinterpret_cast<const uint4*>(k + src);
    *reinterpret_cast<uint4*>(vr + dst) = *reinterpret_cast<const uint4*>(v + src);
  }
  if (h == 0)
    for (int t = lo + (int)threadIdx.x; t < hi; t += blockDim.x)
      c.window_class[(size_t)b * Ws + t % Ws] = cls[t0 + t] == 4 ? 4 : 2;
}

// Grid (H_kv, B), 128 threads: the flush of a MIXED cache (as
// flush_int_kernel), the group stored at the widest class of its G window
// tokens; flush_commit_kernel advances n_quant.
template <int G>
__global__ void __launch_bounds__(128) flush_mixed_kernel(kvq_cache c) {
  grid_dependents_launch();
  const kvq_shape& s = c.shape;
  const int h = blockIdx.x, b = blockIdx.y;
  const int Ws = window_slots(s);
  const int n = c.seq_len[b], nq = c.n_quant[b];
  if (n - nq != Ws) return;
  if (nq < 0 || nq + G > s.capacity || nq % G) {
    if (threadIdx.x == 0 && h == 0) set_err(c.err_word, KVQ_DEVERR_STATE);
    return;
  }
  const bool four =
      __syncthreads_or(threadIdx.x < G && c.window_class[(size_t)b * Ws + (nq + threadIdx.x) % Ws] == 4) != 0;
  if (h == 0 && threadIdx.x == 0) c.group_bits[(size_t)b * (s.capacity / G) + nq / G] = four ? 4 : 2;
  GroupDst d;
  group_dst(c, b, h, nq / G, d);
  const RowSrc ks{(const uint16_t*)c.k_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
  const RowSrc vs{(const uint16_t*)c.v_res + Addr::ring_row(s, b, h, 0), kHeadDim, nq % Ws, Ws};
  quantize_group_mixed<G>(four, ks, vs, d);
}

// ---------------------------------------------------------------------------
// INT8 per-token cache: every key and value row quantized over its 128
// channels at 8 bits when it is written (no window)
// ---------------------------------------------------------------------------

// Grid (ceil(max_len / 32), H_kv, B), 128 threads: warps 0 and 1 quantize
// the key rows of the block's two 16-token tiles, warps 2 and 3 the value
// rows.  Tokens of a sequence's last tile past its length are stored as
// code 0 with scale and zero 0.  Registers are cut for 6 CTAs per SM (80,
// some spill): 84.0 against 88.1 us at 5 on the 8B layer; 8 is slower.
__global__ void __launch_bounds__(128, 6) prefill_int8_kernel(kvq_cache c, const uint16_t* __restrict__ k,
                                                           const uint16_t* __restrict__ v,
                                                           const int32_t* __restrict__ cu, int max_len) {
  const kvq_shape& s = c.shape;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int t0 = cu[b];
  int n = cu[b + 1] - t0;
  const bool too_long = n > s.capacity || n < 0 || n > max_len;
  if (too_long) n = 0;
  if (blk == 0 && h == 0 && threadIdx.x == 0) {
    c.seq_len[b] = n;
    c.n_quant[b] = n;
    if (too_long) set_err(c.err_word, KVQ_DEVERR_PREFILL_LEN);
  }
  const int tile = 2 * blk + (warp & 1);
  if (tile * kTile >= n) return;
  const int valid = min(kTile, n - tile * kTile);
  const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
  const int64_t row0 = ((int64_t)(t0 + tile * kTile) * s.num_kv_heads + h) * kHeadDim;
  if (warp < 2) {
    uint8_t* kc = (uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h) + (size_t)tile * kTile * kHeadDim;
    __half* km = (__half*)c.k_meta + Addr::k_meta_token(s, b, h, tile * kTile);
    int8_token_tile<true>(k + row0, stride, valid, kc, km);
  } else {
    uint8_t* vt = (uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, tile);
    __half* vm = (__half*)c.v_meta + Addr::v_meta_token(s, b, h, tile * kTile);
    int8_token_tile<false>(v + row0, stride, valid, vt, vm);
  }
}

// One token row of 128 channels quantized by one warp (lane: channels
// 4 lane .. 4 lane + 3): returns the four codes in the bytes of a word and
// the (scale, zero) pair as a word.
__device__ __forceinline__ uint32_t int8_encode_words(uint2 xw, uint32_t& meta) {
  const float xf[4] = {bf16_lo(xw.x), bf16_hi(xw.x), bf16_lo(xw.y), bf16_hi(xw.y)};
  float mn = fminf(fminf(xf[0], xf[1]), fminf(xf[2], xf[3]));   // fminf/fmaxf ignore NaN
  float mx = fmaxf(fmaxf(xf[0], xf[1]), fmaxf(xf[2], xf[3]));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  }
  const QParams qp = quant_params(mn, mx, 8);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= encode(xf[i], qp.z, qp.inv, 255) << (8 * i);
  meta = (uint32_t)__half_as_ushort(qp.s16) | ((uint32_t)__half_as_ushort(qp.z16) << 16);
  return w;
}

// Grid (B); block H_kv warps: warp h quantizes sequence b's new key and
// value rows of kv head h into token seq_len[b]; then seq_len and n_quant
// advance together.  The rows are loaded and encoded before the state is
// needed (only the stores depend on it), so the row and state loads are in
// flight together.
__global__ void append_int8_kernel(kvq_cache c, const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn) {
  const kvq_shape& s = c.shape;
  const int b = blockIdx.x;
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint2 kx = make_uint2(0u, 0u), vx = make_uint2(0u, 0u);
  const size_t off = ((size_t)b * s.num_kv_heads + h) * kHeadDim;
  if (h < s.num_kv_heads) {
    kx = *reinterpret_cast<const uint2*>(kn + off + 4 * lane);
    vx = *reinterpret_cast<const uint2*>(vn + off + 4 * lane);
  }
  const int n = c.seq_len[b], nq = c.n_quant[b];
  uint32_t km = 0, vm = 0, kw = 0, vw = 0;
  if (h < s.num_kv_heads) {
    kw = int8_encode_words(kx, km);
    vw = int8_encode_words(vx, vm);
  }
  if (n >= s.capacity || n < 0 || nq != n) {
    if (threadIdx.x == 0) set_err(c.err_word, KVQ_DEVERR_APPEND_FULL);
    return;
  }
  if (h < s.num_kv_heads) {
    uint8_t* kc = (uint8_t*)c.k_codes + Addr::k_codes_unit(s, b, h) + (size_t)n * kHeadDim;
    *reinterpret_cast<uint32_t*>(kc + 4 * lane) = kw;
    uint8_t* vt = (uint8_t*)c.v_codes + Addr::v_codes_tile(s, b, h, n / kTile);
#pragma unroll
    for (int i = 0; i < 4; ++i) vt[fp8_vtile_offset(n % kTile, 4 * lane + i)] = (uint8_t)(vw >> (8 * i));
    if (lane == 0) {
      *reinterpret_cast<uint32_t*>((__half*)c.k_meta + Addr::k_meta_token(s, b, h, n)) = km;
      *reinterpret_cast<uint32_t*>((__half*)c.v_meta + Addr::v_meta_token(s, b, h, n)) = vm;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    c.seq_len[b] = n + 1;
    c.n_quant[b] = n + 1;
  }
}

// ---------------------------------------------------------------------------
// Host launchers (called by kvq_api.cu after validation)
// ---------------------------------------------------------------------------

cudaError_t launch_prefill(const kvq_cache& c, const void* k, const void* v, const int32_t* cu, int max_len,
                           cudaStream_t st) {
  const kvq_shape& s = c.shape;
  const int limit = max_len;           // longer sequences are rejected on the device
  if (max_len <= 0) max_len = 1;
  if (is_int8(s.format)) {
    dim3 g8((max_len + 2 * kTile - 1) / (2 * kTile), s.num_kv_heads, s.batch);
    prefill_int8_kernel<<<g8, 128, 0, st>>>(c, (const uint16_t*)k, (const uint16_t*)v, cu, limit);
    return cudaGetLastError();
  }
  if (is_fp8(s.format)) {
    cudaError_t e = cudaMemsetAsync(c.fp8_amax, 0, sizeof(uint32_t) * 2 * s.num_kv_heads, st);
    if (e != cudaSuccess) return e;
    dim3 ga((max_len + 63) / 64, s.num_kv_heads, s.batch);
    fp8_amax_kernel<<<ga, 128, 0, st>>>(c, (const uint16_t*)k, (const uint16_t*)v, cu, limit);
    dim3 gp((max_len + kTile - 1) / kTile, s.num_kv_heads, s.batch);
    fp8_prefill_kernel<<<gp, 32 * kTile, 0, st>>>(c, (const uint16_t*)k, (const uint16_t*)v, cu, limit);
    return cudaGetLastError();
  }
  const int TB = s.group < 32 ? 32 : s.group;
  dim3 grid((max_len + TB - 1) / TB, s.num_kv_heads, s.batch);
  const uint16_t* kk = (const uint16_t*)k;
  const uint16_t* vv = (const uint16_t*)v;
#define KVQ_PREFILL_CASE(B, GG) \
  if (s.format == B && s.group == GG && !s.sparse) prefill_int_kernel<B, GG, false><<<grid, 128, 0, st>>>(c, kk, vv, cu, limit);
#define KVQ_PREFILL_SPARSE_CASE(B, GG) \
  if (s.format == B && s.group == GG && s.sparse) prefill_int_kernel<B, GG, true><<<grid, 128, 0, st>>>(c, kk, vv, cu, limit);
  KVQ_PREFILL_CASE(4, 16) KVQ_PREFILL_CASE(4, 32) KVQ_PREFILL_CASE(4, 64) KVQ_PREFILL_CASE(4, 128)
  KVQ_PREFILL_CASE(2, 16) KVQ_PREFILL_CASE(2, 32) KVQ_PREFILL_CASE(2, 64) KVQ_PREFILL_CASE(2, 128)
  KVQ_PREFILL_SPARSE_CASE(4, 16) KVQ_PREFILL_SPARSE_CASE(4, 32) KVQ_PREFILL_SPARSE_CASE(2, 16) KVQ_PREFILL_SPARSE_CASE(2, 32)
#undef KVQ_PREFILL_CASE
#undef KVQ_PREFILL_SPARSE_CASE
  return cudaGetLastError();
}

cudaError_t launch_prefill_mixed(const kvq_cache& c, const void* k, const void* v, const uint8_t* cls,
                                 const int32_t* cu, int max_len, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  const int limit = max_len;
  if (max_len <= 0) max_len = 1;
  dim3 grid((max_len + s.group - 1) / s.group, s.num_kv_heads, s.batch);
  const uint16_t* kk = (const uint16_t*)k;
  const uint16_t* vv = (const uint16_t*)v;
  if (s.group == 32) prefill_mixed_kernel<32><<<grid, 128, 0, st>>>(c, kk, vv, cls, cu, limit);
  else if (s.group == 64) prefill_mixed_kernel<64><<<grid, 128, 0, st>>>(c, kk, vv, cls, cu, limit);
  else if (s.group == 128) prefill_mixed_kernel<128><<<grid, 128, 0, st>>>(c, kk, vv, cls, cu, limit);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

cudaError_t launch_append_mixed(const kvq_cache& c, const void* kn, const void* vn, const uint8_t* cls,
                                cudaStream_t st) {
  const kvq_shape& s = c.shape;
  append_int_kernel<<<s.batch, 32 * min(s.num_kv_heads, 32), 0, st>>>(c, (const uint16_t*)kn, (const uint16_t*)vn,
                                                                      cls);
  return cudaGetLastError();
}

cudaError_t launch_append(const kvq_cache& c, const void* kn, const void* vn, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  if (is_fp8(s.format))
    fp8_append_kernel<<<s.batch, 32 * s.num_kv_heads, 0, st>>>(c, (const uint16_t*)kn, (const uint16_t*)vn);
  else if (is_int8(s.format))
    append_int8_kernel<<<s.batch, 32 * s.num_kv_heads, 0, st>>>(c, (const uint16_t*)kn, (const uint16_t*)vn);
  else
    append_int_kernel<<<s.batch, 32 * min(s.num_kv_heads, 32), 0, st>>>(c, (const uint16_t*)kn,
                                                                        (const uint16_t*)vn, nullptr);
  return cudaGetLastError();
}

cudaError_t launch_flush(const kvq_cache& c, cudaStream_t st);

// Append and flush in one launch (one cluster of H_kv CTAs per sequence)
// when the kv heads fit a portable cluster; otherwise the two calls.
cudaError_t launch_append_flush(const kvq_cache& c, const void* kn, const void* vn, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  if (is_token_cache(s.format) || s.num_kv_heads > 8) {
    cudaError_t e = launch_append(c, kn, vn, st);
    return e != cudaSuccess ? e : launch_flush(c, st);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.num_kv_heads, s.batch);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = s.num_kv_heads;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint16_t* k16 = (const uint16_t*)kn;
  const uint16_t* v16 = (const uint16_t*)vn;
#define KVQ_APPEND_FLUSH_CASE(B, GG, SP) \
  if (s.format == B && s.group == GG && (bool)s.sparse == SP) \
    return cudaLaunchKernelEx(&cfg, append_flush_int_kernel<B, GG, SP>, c, k16, v16);
  KVQ_APPEND_FLUSH_CASE(4, 16, false) KVQ_APPEND_FLUSH_CASE(4, 32, false) KVQ_APPEND_FLUSH_CASE(4, 64, false)
  KVQ_APPEND_FLUSH_CASE(4, 128, false) KVQ_APPEND_FLUSH_CASE(2, 16, false) KVQ_APPEND_FLUSH_CASE(2, 32, false)
  KVQ_APPEND_FLUSH_CASE(2, 64, false) KVQ_APPEND_FLUSH_CASE(2, 128, false)
  KVQ_APPEND_FLUSH_CASE(4, 16, true) KVQ_APPEND_FLUSH_CASE(4, 32, true) KVQ_APPEND_FLUSH_CASE(2, 16, true)
  KVQ_APPEND_FLUSH_CASE(2, 32, true)
#undef KVQ_APPEND_FLUSH_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_flush(const kvq_cache& c, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  if (is_token_cache(s.format)) return cudaSuccess;
  dim3 grid(s.num_kv_heads, s.batch);
  if (is_mixed(s.format)) {
    if (s.group == 32) flush_mixed_kernel<32><<<grid, 128, 0, st>>>(c);
    else if (s.group == 64) flush_mixed_kernel<64><<<grid, 128, 0, st>>>(c);
    else if (s.group == 128) flush_mixed_kernel<128><<<grid, 128, 0, st>>>(c);
  }
#define KVQ_FLUSH_CASE(B, GG, SP) \
  if (s.format == B && s.group == GG && (bool)s.sparse == SP) flush_int_kernel<B, GG, SP><<<grid, 128, 0, st>>>(c);
  KVQ_FLUSH_CASE(4, 16, false) KVQ_FLUSH_CASE(4, 32, false) KVQ_FLUSH_CASE(4, 64, false) KVQ_FLUSH_CASE(4, 128, false)
  KVQ_FLUSH_CASE(2, 16, false) KVQ_FLUSH_CASE(2, 32, false) KVQ_FLUSH_CASE(2, 64, false) KVQ_FLUSH_CASE(2, 128, false)
  KVQ_FLUSH_CASE(4, 16, true) KVQ_FLUSH_CASE(4, 32, true) KVQ_FLUSH_CASE(2, 16, true) KVQ_FLUSH_CASE(2, 32, true)
#undef KVQ_FLUSH_CASE
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the commit is launched early (programmatic dependent launch) and waits
  // on the device, which hides its launch latency behind the flush
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.batch);
  cfg.blockDim = dim3(32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, flush_commit_kernel, c);
}

}  // namespace kvq
