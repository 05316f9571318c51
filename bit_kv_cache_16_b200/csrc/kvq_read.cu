// kvq_read_tokens: token ranges of the cache as bf16 rows.
#include "kvq_rows.cuh"

namespace kvq {

struct ReadArgs {
  kvq_cache c;
  const int32_t* start;    // [B] first token per sequence, or null (0)
  const int32_t* cu;       // [B + 1] output rows
  uint16_t* k;             // bf16 [rows][H_kv][128], or null
  uint16_t* v;             // same, or null
  int rows;                // of k and v
  int max_len;
};

// Grid (pairs of tiles x H_kv, B), 128 threads: two 16-token tiles of one
// (sequence, kv head), warps 0 and 1 their keys, warps 2 and 3 their values.  A
// tile is either quantized (tokens below n_quant, a multiple of 16 where there
// is a window) or held in the window ring.  Bound by the bf16 rows it writes:
// the heads are neighbours in the grid, as their rows are in memory, and every
// store of a value row is 32 bytes, a whole sector.  131072 INT2 tokens of 8
// heads: 117 to 119 us, 5.3 TB/s (147 with a head's tiles side by side and
// 16-byte stores); 16 x 4096 FP8 tokens: 77 us, 5.2 TB/s.  Several tile pairs per CTA
// took 141 to 160 us, 8 CTAs per SM 139.
template <int FMT>
__global__ void __launch_bounds__(128, 16) read_tokens_kernel(ReadArgs A) {
  const kvq_cache& c = A.c;
  const kvq_shape& s = c.shape;
  const int h = blockIdx.x % s.num_kv_heads, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = A.cu[b], len = A.cu[b + 1] - row0;
  const int first = A.start ? A.start[b] : 0;
  const int n = c.seq_len[b], nq = c.n_quant[b];
  const bool lead = blockIdx.x == 0 && threadIdx.x == 0;
  if (state_bad(s, n, nq)) {
    if (lead) atomicOr(c.err_word, KVQ_DEVERR_STATE);
    return;
  }
  if (len < 0 || len > A.max_len || row0 < 0 || row0 > A.rows - len || first < 0 || first > n || len > n - first) {
    if (lead) atomicOr(c.err_word, KVQ_DEVERR_PREFILL_LEN);
    return;
  }
  const bool key = warp < 2;
  uint16_t* rows = key ? A.k : A.v;
  if (!rows) return;
  const int64_t stride = (int64_t)s.num_kv_heads * kHeadDim;
  const int tile = first / kTile + 2 * (blockIdx.x / s.num_kv_heads) + (warp & 1);
  const int lo = max(first - tile * kTile, 0), hi = min(kTile, first + len - tile * kTile);
  if (lo >= hi) return;
  // row of the tile's token 0 (never written when lo > 0)
  uint16_t* out = rows + ((int64_t)(row0 + tile * kTile - first) * s.num_kv_heads + h) * kHeadDim;
  if (!is_token_cache(FMT) && tile * kTile >= nq) {
    const int Ws = window_slots(s);
    const uint16_t* ring = (const uint16_t*)(key ? c.k_res : c.v_res) + Addr::ring_row(s, b, h, 0);
    for (int r = lo + (lane >> 4); r < hi; r += 2)
      *reinterpret_cast<uint4*>(out + r * stride + 8 * (lane & 15)) =
          *reinterpret_cast<const uint4*>(ring + (size_t)((tile * kTile + r) % Ws) * kHeadDim + 8 * (lane & 15));
    return;
  }
  TileSrc d;
  if (!tile_src<FMT>(c, b, h, tile, d)) {
    if (lane == 0) atomicOr(c.err_word, KVQ_DEVERR_PAGE_RANGE);
    return;
  }
  if (key) {
    key_rows<FMT>(d, lo, hi, [&](int r, int ch, const float (&x)[8]) {
      *reinterpret_cast<uint4*>(out + r * stride + ch) =
          make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
    });
  } else {
    // a whole sector per store where the caller's rows start on one
    const bool sectors = ((uintptr_t)rows & 31u) == 0;
    value_rows<FMT>(d, lo, hi, [&](int r, int ch, const float (&x)[16]) {
      const uint4 a = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
      const uint4 e = make_uint4(pack_bf2(x[8], x[9]), pack_bf2(x[10], x[11]), pack_bf2(x[12], x[13]), pack_bf2(x[14], x[15]));
      uint16_t* to = out + r * stride + ch;
      if (sectors) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(e.x), "r"(e.y), "r"(e.z), "r"(e.w)
                     : "memory");
      } else {
        *reinterpret_cast<uint4*>(to) = a;
        *reinterpret_cast<uint4*>(to + 8) = e;
      }
    });
  }
}

cudaError_t launch_read_tokens(const kvq_cache& c, const int32_t* start, const int32_t* cu, int rows, int max_len,
                               void* k, void* v, cudaStream_t st) {
  const kvq_shape& s = c.shape;
  const ReadArgs A{c, start, cu, (uint16_t*)k, (uint16_t*)v, rows, max_len};
  const int most = min(max_len, s.capacity);         // longer ranges are rejected on the device
  // a range of m tokens touches at most (m + 30) / 16 tiles
  const long long pairs = max(1, ((most + 2 * kTile - 2) / kTile + 1) / 2);
  if (pairs * s.num_kv_heads > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  dim3 grid((unsigned)(pairs * s.num_kv_heads), s.batch);
  switch (s.format) {
    case KVQ_FORMAT_INT2: read_tokens_kernel<2><<<grid, 128, 0, st>>>(A); break;
    case KVQ_FORMAT_INT4: read_tokens_kernel<4><<<grid, 128, 0, st>>>(A); break;
    case KVQ_FORMAT_MIXED: read_tokens_kernel<6><<<grid, 128, 0, st>>>(A); break;
    case KVQ_FORMAT_FP8_E4M3: read_tokens_kernel<8><<<grid, 128, 0, st>>>(A); break;
    default: read_tokens_kernel<16><<<grid, 128, 0, st>>>(A); break;
  }
  return cudaGetLastError();
}

}  // namespace kvq
