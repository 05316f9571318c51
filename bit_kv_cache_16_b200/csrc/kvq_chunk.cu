// kvq_chunk_attention, general form: a chunk of new tokens attends to the
// packed cache and causally to itself, in fp32 on the CUDA cores.
#include "kvq_chunk.cuh"
#include "kvq_rows.cuh"

namespace kvq {

constexpr int kGenRows = 32;                 // query rows per CTA
constexpr int kGenKeys = 32;                 // keys per step: two 16-token tiles
constexpr int kGenPad = kHeadDim + 4;        // floats per row (16-byte aligned, rows in different banks)

struct GenSmem {
  float q[kGenRows][kGenPad];
  float k[kGenKeys][kGenPad];
  float v[kGenKeys][kGenPad];
  float p[kGenRows][kGenKeys + 1];
  double freq[kHeadDim / 2];                 // RoPE pair frequencies
  int skipped[2];                            // the step's tiles whose page id is bad
};

// Grid (row blocks, H_kv, B), 128 threads.  Row r of a unit is head r % gq of
// new token r / gq.  Each step brings 32 keys and values as fp32 into shared
// memory (warps 0, 1 keys, warps 2, 3 values; one 16-token tile each): from the
// packed tiles, the window ring or the chunk, keys stored before RoPE rotated
// by their position.  Four threads share a row: scores of every fourth key,
// then 32 channels each of the value sum.  Softmax online, everything in fp32.
// Bound by the fp32 rate of the two products.
template <int FMT>
__global__ void __launch_bounds__(128) chunk_general_kernel(ChunkAttnArgs A) {
  extern __shared__ __align__(16) uint8_t raw[];
  GenSmem& sm = *reinterpret_cast<GenSmem*>(raw);
  const kvq_cache& c = A.c;
  const kvq_shape& s = c.shape;
  const int kv = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = s.num_q_heads / s.num_kv_heads;
  const ChunkSeq sq = chunk_seq(A, b);
  if (sq.err && blockIdx.x == 0 && kv == 0 && tid == 0) atomicOr(c.err_word, sq.err);
  const int r0 = blockIdx.x * kGenRows, rows = sq.m * gq;
  if (r0 >= rows) return;
  const bool rope = s.rope_theta > 0.f;
  if (rope && tid < kHeadDim / 2)
    sm.freq[tid] = pow((double)s.rope_theta, -2.0 * (double)tid / (double)kHeadDim);
  for (int e = tid; e < kGenRows * kHeadDim / 2; e += 128) {
    const int r = e / (kHeadDim / 2), w = e % (kHeadDim / 2), R = r0 + r;
    uint32_t x = 0u;
    if (R < rows)
      x = reinterpret_cast<const uint32_t*>(
          A.q + ((size_t)(sq.t0 + R / gq) * s.num_q_heads + kv * gq + R % gq) * kHeadDim)[w];
    sm.q[r][2 * w] = bf16_lo(x);
    sm.q[r][2 * w + 1] = bf16_hi(x);
  }
  const int row = tid >> 2, l = tid & 3;
  const int p_row = sq.p0 + min(r0 + row, rows - 1) / gq;               // this row's position
  const TileRange range(sq.p0 + r0 / gq, sq.p0 + (min(r0 + kGenRows, rows) - 1) / gq, A.window, A.sinks, kGenKeys);
  const int Ws = window_slots(s);
  float m = -INFINITY, sum = 0.f, o[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) o[i] = 0.f;

  for (int it = 0; it < range.count; ++it) {
    const int t0 = range.tile(it) * kGenKeys;
    __syncthreads();                         // the last step's tiles are used up
    {
      const bool key = warp < 2;
      const int base = 16 * (warp & 1), tile = t0 / kTile + (warp & 1);
      float(*dst)[kGenPad] = key ? sm.k : sm.v;
      auto put = [&](int r, int ch, const float (&x)[8]) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        if (key && rope) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float cs, sn;
            rope_cos_sin(tile * kTile + r, sm.freq[ch / 2 + i], cs, sn);
            y[2 * i] = x[2 * i] * cs - x[2 * i + 1] * sn;
            y[2 * i + 1] = x[2 * i] * sn + x[2 * i + 1] * cs;
          }
        }
        float4* d4 = reinterpret_cast<float4*>(&dst[base + r][ch]);
        d4[0] = make_float4(y[0], y[1], y[2], y[3]);
        d4[1] = make_float4(y[4], y[5], y[6], y[7]);
      };
      const int quant = min(max(sq.nq - tile * kTile, 0), kTile);      // the tile's quantized rows come first
      bool ok = true;
      if (quant > 0) {
        TileSrc d;
        ok = tile_src<FMT>(c, b, kv, tile, d);
        if (ok) {
          if (key) key_rows<FMT>(d, 0, quant, put);
          else value_rows<FMT>(d, 0, quant, put);
        } else if (lane == 0 && key) atomicOr(c.err_word, KVQ_DEVERR_PAGE_RANGE);
      }
      if (lane == 0 && key) sm.skipped[warp] = ok ? 0 : 1;
      for (int r = quant + (lane >> 4); r < kTile; r += 2) {
        const int t = tile * kTile + r, ch = 8 * (lane & 15);
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (t < sq.n)
          w = *reinterpret_cast<const uint4*>((const uint16_t*)(key ? c.k_res : c.v_res) +
                                              Addr::ring_row(s, b, kv, t % Ws) + ch);
        else if (t < sq.total)
          w = *reinterpret_cast<const uint4*>((key ? A.k : A.v) +
                                              ((size_t)(sq.t0 + t - sq.n) * s.num_kv_heads + kv) * kHeadDim + ch);
        const float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                            bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
        put(r, ch, x);
      }
    }
    __syncthreads();
    float sc[8], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = l + 4 * i, t = t0 + j;
      sc[i] = -INFINITY;
      if (!key_visible(t, p_row, A.window, A.sinks) || (t < sq.nq && sm.skipped[j / kTile])) continue;
      float d = 0.f;
      const float4* qr = reinterpret_cast<const float4*>(sm.q[row]);
      const float4* kr = reinterpret_cast<const float4*>(sm.k[j]);
#pragma unroll 8
      for (int e = 0; e < kHeadDim / 4; ++e) {
        const float4 x = qr[e], y = kr[e];
        d = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, d))));
      }
      sc[i] = d * A.scale_log2;
      top = fmaxf(top, sc[i]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref);            // 0 while m is -inf
    sum *= f;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= f;
    m = mn;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = ex2(sc[i] - ref);
      sum += e;
      sm.p[row][l + 4 * i] = e;
    }
    __syncwarp();
#pragma unroll 1
    for (int j = 0; j < kGenKeys; ++j) {
      const float p = sm.p[row][j];
      if (p == 0.f) continue;                // hidden keys' values may be anything, infinities too
      const float4* vr = reinterpret_cast<const float4*>(sm.v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = vr[l + 4 * i];
        o[4 * i] = fmaf(p, x.x, o[4 * i]); o[4 * i + 1] = fmaf(p, x.y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(p, x.z, o[4 * i + 2]); o[4 * i + 3] = fmaf(p, x.w, o[4 * i + 3]);
      }
    }
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  if (r0 + row >= rows) return;
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  const int R = r0 + row;
  if (A.out32) {
    const size_t at = (size_t)(sq.t0 + R / gq) * s.num_q_heads + kv * gq + R % gq;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(A.out32 + at * kHeadDim + 4 * (l + 4 * i)) =
          make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
    if (A.lse && l == 0) A.lse[at] = (m + log2f(sum)) * 0.69314718055994531f;
    return;
  }
  uint16_t* dst = A.out + ((size_t)(sq.t0 + R / gq) * s.num_q_heads + kv * gq + R % gq) * kHeadDim;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint2*>(dst + 4 * (l + 4 * i)) =
        make_uint2(pack_bf2(o[4 * i] * inv, o[4 * i + 1] * inv), pack_bf2(o[4 * i + 2] * inv, o[4 * i + 3] * inv));
}

template <int FMT>
static cudaError_t launch_general(const ChunkAttnArgs& A, cudaStream_t st) {
  const kvq_shape& s = A.c.shape;
  const int gq = s.num_q_heads / s.num_kv_heads;
  cudaError_t e = cudaFuncSetAttribute(chunk_general_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(GenSmem));
  if (e != cudaSuccess) return e;
  const long long blocks = ((long long)min(A.max_new, A.rows) * gq + kGenRows - 1) / kGenRows;
  dim3 grid((unsigned)max(blocks, 1ll), s.num_kv_heads, s.batch);
  chunk_general_kernel<FMT><<<grid, 128, sizeof(GenSmem), st>>>(A);
  return cudaGetLastError();
}

size_t chunk_workspace_bytes(const kvq_shape& s, int num_splits, int rows) { return 0; }
int chunk_default_splits(const kvq_shape& s, int rows, int max_new, int max_len, int window, int sinks) { return 1; }

cudaError_t launch_chunk_attention(const ChunkAttnArgs& A, cudaStream_t st) {
  switch (A.c.shape.format) {
    case KVQ_FORMAT_INT2: return launch_general<2>(A, st);
    case KVQ_FORMAT_INT4: return launch_general<4>(A, st);
    case KVQ_FORMAT_MIXED: return launch_general<6>(A, st);
    case KVQ_FORMAT_FP8_E4M3: return launch_general<8>(A, st);
    default: return launch_general<16>(A, st);
  }
}

}  // namespace kvq
