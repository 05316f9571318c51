// kvq_decode_attention_window: the decode kernels (kvq_decode.cuh) over the
// last `window` tokens and the first `sinks`.  Only the 32-token chunks that
// hold visible tokens enter the list the warps stream; a chunk at an edge has
// its hidden tokens' scores set to -inf and their scales, zeros and codes to
// zero, so that nothing stored there (NaN and infinities too) reaches a sum.
// 65000 + 128 of 131072 INT8 tokens, batch 2, 64 / 8 heads: 68 us, 4.1 TB/s,
// bound as the full decode by each chunk's chain of conversions; 1024 + 4 of
// 8192 INT4 tokens, batch 8, 32 / 8 heads: 16 us, one or two chunks a warp and
// so the fixed part of both kernels (alone under ncu 13 and 7 us).
#include "kvq_decode.cuh"

namespace kvq {

// The split count for the tokens that can be visible.
int window_default_splits(const kvq_shape& s, int max_len, int window, int sinks) {
  const long long seen = window > 0 ? min((long long)max_len, (long long)window + sinks) : max_len;
  return decode_splits_rule(s, (int)max(seen, 1ll));
}

cudaError_t launch_window_decode(const kvq_cache& c, const void* q, float* out, float* lse, float softmax_scale,
                                 int window, int sinks, void* ws, int num_splits, cudaStream_t st) {
  return launch_decode_form<true>(c, q, out, lse, softmax_scale, WindowSpec{window, sinks}, ws, num_splits, st);
}

}  // namespace kvq
