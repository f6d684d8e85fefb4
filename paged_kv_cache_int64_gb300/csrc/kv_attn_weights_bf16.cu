// kv_attn_weights_bf16.cu - the kernels of pkv_kv_attn_weights over a cache of this type (a file each, compiled side by side).
#include "kv_attn_weights.cuh"

namespace pkv {
pkv_status run_attn_weights_bf16(const WeightParams& p, int ctas, cudaStream_t stream) {
  return run_attn_weights<PKV_KV_BF16>(p, ctas, stream);
}
}  // namespace pkv
