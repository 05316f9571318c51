// kvq_decode_attention and kvq_merge_partials: the decode kernels
// (kvq_decode.cuh) over every token, and the merge of partial attentions.
#include "kvq_decode.cuh"

namespace kvq {

// Grid (rows); block 128: merge of `parts` partial attentions of the same
// rows over disjoint token sets (section 3.2 of the arganzheng page attends
// the window and the quantized part apart and merges them the same way):
// out = sum_p e^(lse_p - L) out_p with L = ln sum_p e^(lse_p).  A part with
// lse = -inf has no tokens; a row with no tokens anywhere gets zeros.
__global__ void __launch_bounds__(kHeadDim) merge_partials_kernel(const float* __restrict__ outs,
                                                                  const float* __restrict__ lses, int parts,
                                                                  long long rows, float* __restrict__ out,
                                                                  float* __restrict__ lse_out) {
  const long long r = blockIdx.x;
  const int ch = threadIdx.x;
  float M = -INFINITY;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, lses[p * rows + r]);
  float o = 0.f, L = 0.f;
  if (M != -INFINITY) {
    for (int p = 0; p < parts; ++p) {
      const float lp = lses[p * rows + r];
      const float w = lp == -INFINITY ? 0.f : expf(lp - M);
      L += w;
      o = fmaf(w, outs[(p * rows + r) * kHeadDim + ch], o);
    }
  }
  out[r * kHeadDim + ch] = L > 0.f ? o / L : 0.f;
  if (lse_out && ch == 0) lse_out[r] = L > 0.f ? M + logf(L) : -INFINITY;
}

int decode_default_splits(const kvq_shape& s, int max_len) { return decode_splits_rule(s, max_len); }

size_t decode_workspace_bytes(const kvq_shape& s, int num_splits) { return decode_workspace_rule(s, num_splits); }

cudaError_t launch_decode(const kvq_cache& c, const void* q, float* out, float* lse, float softmax_scale, void* ws,
                          int num_splits, cudaStream_t st) {
  return launch_decode_form<false>(c, q, out, lse, softmax_scale, WindowSpec{0, 0}, ws, num_splits, st);
}

cudaError_t launch_merge(const float* outs, const float* lses, int parts, long long rows, float* out, float* lse_out,
                         cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  merge_partials_kernel<<<(unsigned)rows, kHeadDim, 0, st>>>(outs, lses, parts, rows, out, lse_out);
  return cudaGetLastError();
}

}  // namespace kvq
