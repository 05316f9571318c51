// What the chunk attention kernels (kvq_chunk.cu) and its host code share.
#pragma once

#include "kvq_common.cuh"

namespace kvq {

struct ChunkAttnArgs {
  kvq_cache c;
  const uint16_t* q;      // bf16 [rows][H_q][128]
  const uint16_t* k;      // bf16 [rows][H_kv][128]: the chunk's own keys
  const uint16_t* v;      // bf16 [rows][H_kv][128]
  const int32_t* cu;      // [B + 1] chunk rows of each sequence
  uint16_t* out;          // bf16 [rows][H_q][128]
  float* ws_o;            // [splits][rows][H_q][128] (splits > 1)
  float* ws_ml;           // [splits][rows][H_q][2]
  float scale_log2;       // softmax_scale * log2(e)
  int rows;               // rows of the chunk arrays
  int max_new;
  int window, sinks;      // window 0: every earlier token is visible
  int splits;
};

// The sequence's share of a call: n cached tokens (nq quantized), m new ones
// from row t0 on at positions n, n + 1, ..., `total` together.  err: the bit
// to report for a state, length or row range that fails the checks (then m =
// 0 and nothing is computed).
struct ChunkSeq {
  int n, nq, m, t0, total;
  uint32_t err;
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkAttnArgs& A, int b) {
  ChunkSeq q;
  q.t0 = A.cu[b];
  q.m = A.cu[b + 1] - q.t0;
  q.n = A.c.seq_len[b];
  q.nq = A.c.n_quant[b];
  q.err = 0u;
  if (state_bad(A.c.shape, q.n, q.nq)) q.err = KVQ_DEVERR_STATE;
  else if (q.m < 0 || q.m > A.max_new || q.t0 < 0 || q.t0 > A.rows - q.m) q.err = KVQ_DEVERR_PREFILL_LEN;
  if (q.err) q.m = 0;
  q.total = q.n + q.m;
  return q;
}

// Key tiles of TS tokens that rows at positions [p0, p1] can see, in order:
// the tiles of the first `sinks` tokens, then those from the first row's
// window to p1.  tile(i) for 0 <= i < count.
struct TileRange {
  int lead, skip, count;
  TileRange() = default;
  __device__ __forceinline__ TileRange(int p0, int p1, int window, int sinks, int TS) {
    const int lo = window > 0 ? max(0, p0 - window + 1) : 0;
    skip = lo / TS;
    lead = min(skip, (min(sinks, lo) + TS - 1) / TS);
    count = lead + p1 / TS + 1 - skip;
  }
  __device__ __forceinline__ int tile(int i) const { return i < lead ? i : skip + i - lead; }
};

}  // namespace kvq
