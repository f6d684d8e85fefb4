// kv_attn_weights.cu - pkv_kv_attn_weights: the attention weight that each cached key collects.
//
//   weights[r][h][pos] = prev + sum over the counted tokens t and the query heads of KV head h of exp(s - lse),
// s = softmax_scale q . k, lse the query row's log-sum-exp (of the verify partials, or computed here first).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

constexpr int kD = 256;
constexpr int kMaxCols = 128;  // query columns of one pass

struct WeightParams {
  const __nv_bfloat16* q;
  const uint8_t* k;
  const float* k_scale;
  int64_t num_blocks, stride_blk, stride_tok, stride_head, s_stride_blk, s_stride_tok;  // elements
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  const int32_t* q_valid;
  int32_t num_reqs, T, num_q_heads, num_kv_heads, block_size;
  float softmax_scale;
  const float* part_lse;
  int32_t split_tokens, max_splits;
  const float* prev;
  const int32_t* prev_lens;
  float* weights;
  int64_t w_stride_req, w_stride_head, max_ctx;
  float* lse;  // workspace
  int* dev_err;
};

__device__ __forceinline__ int keys_of(const WeightParams& p, int len) {
  return (int)max((int64_t)0, min((int64_t)len, (int64_t)p.max_blocks * p.block_size));
}

// The warp's dot product of a query row with the key at `pos`, times the key's scale; lane l has 8 elements.
template <int kFmt>
__device__ float score(const WeightParams& p, int r, int h, int pos, const float (&q)[8], int lane) {
  const int col = pos / p.block_size;
  const int blk = __ldg(p.block_table + (int64_t)r * p.bt_stride + col);
  if (blk < 0 || blk >= p.num_blocks) {
    if (lane == 0) record_error(p.dev_err, kErrDeviceBounds);
    return 0.0f;
  }
  const int slot = pos - col * p.block_size;
  const int64_t at = blk * p.stride_blk + slot * p.stride_tok + h * p.stride_head + lane * 8;
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float k;
    if (kFmt == PKV_KV_BF16) k = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.k)[at + e]);
    if (kFmt == PKV_KV_INT8) k = (float)reinterpret_cast<const int8_t*>(p.k)[at + e];
    if (kFmt == PKV_KV_FP8) k = (float)reinterpret_cast<const __nv_fp8_e4m3*>(p.k)[at + e];
    s = fmaf(q[e], k, s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (kFmt == PKV_KV_INT8) s *= __ldg(p.k_scale + blk * p.s_stride_blk + slot * p.s_stride_tok + h);
  if (kFmt == PKV_KV_FP8) s *= __ldg(p.k_scale);
  return s * p.softmax_scale;
}

__device__ __forceinline__ void load_q(const WeightParams& p, int64_t row, float (&q)[8], int lane) {
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = __bfloat162float(p.q[row * kD + lane * 8 + e]);
}

template <int kFmt>
__global__ void lse_kernel(const WeightParams p) {
  const int64_t row = blockIdx.x;  // (r * T + t) * Hq + head
  const int head = (int)(row % p.num_q_heads), rt = (int)(row / p.num_q_heads), r = rt / p.T, t = rt % p.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int len = p.seq_lens[r], n = min(keys_of(p, len), len - p.T + t + 1);
  __shared__ float s_m[32], s_l[32];
  float m = -INFINITY, l = 0.0f;
  if (p.part_lse) {
    if (warp == 0) {
      const int splits = len > 0 ? min((len - 1) / p.split_tokens + 1, p.max_splits) : 0;
      const int64_t rows = (int64_t)p.num_reqs * p.T * p.num_q_heads;
      for (int s = 0; s < splits; ++s) {
        const float x = p.part_lse[s * rows + row];
        const float m2 = fmaxf(m, x);
        if (m2 != -INFINITY) l = l * expf(m - m2) + expf(x - m2);
        m = m2;
      }
    }
  } else {
    float q[8];
    load_q(p, row, q, lane);
    for (int pos = warp; pos < n; pos += warps) {
      const float x = score<kFmt>(p, r, head / (p.num_q_heads / p.num_kv_heads), pos, q, lane);
      const float m2 = fmaxf(m, x);
      if (m2 != -INFINITY) l = l * expf(m - m2) + expf(x - m2);
      m = m2;
    }
  }
  s_m[warp] = m;
  s_l[warp] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < warps; ++w) mm = fmaxf(mm, s_m[w]);
    for (int w = 0; w < warps; ++w)
      if (s_l[w] != 0.0f) ll += s_l[w] * expf(s_m[w] - mm);
    p.lse[row] = ll == 0.0f ? -INFINITY : mm + logf(ll);
  }
}

template <int kFmt>
__global__ void weights_kernel(const WeightParams p) {
  const int r = blockIdx.y, h = blockIdx.z;
  const int lane = threadIdx.x & 31;
  const int group = p.num_q_heads / p.num_kv_heads;
  const int len = p.seq_lens[r], n = keys_of(p, len);
  const int valid = p.q_valid ? max(0, min(p.q_valid[r], p.T)) : p.T;
  if (blockIdx.x == 0 && threadIdx.x == 0 && h == 0 && (len < 0 || len > n || n > p.max_ctx)) record_error(p.dev_err, kErrDeviceBounds);
  const int n_out = (int)min((int64_t)n, p.max_ctx);
  const int prev_len = p.prev && p.prev_lens ? p.prev_lens[r] : p.prev ? n : 0;
  for (int pos = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); pos < n_out; pos += gridDim.x * (blockDim.x >> 5)) {
    float sum = 0.0f;
    for (int t = max(0, pos - (len - p.T)); t < valid; ++t)
      for (int g = 0; g < group; ++g) {
        const int64_t row = ((int64_t)r * p.T + t) * p.num_q_heads + h * group + g;
        const float lse = p.lse[row];
        if (lse == -INFINITY) continue;
        float q[8];
        load_q(p, row, q, lane);
        sum += expf(score<kFmt>(p, r, h, pos, q, lane) - lse);
      }
    if (lane == 0) {
      const int64_t at = (int64_t)r * p.w_stride_req + (int64_t)h * p.w_stride_head + pos;
      p.weights[at] = pos < prev_len ? p.prev[at] + sum : sum;
    }
  }
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_kv_attn_weights_workspace_bytes(int32_t num_rows, int32_t num_q_heads, int32_t num_ctas) {
  if (num_rows <= 0 || num_q_heads <= 0 || num_ctas <= 0) return 0;
  return ((size_t)num_rows * (size_t)num_q_heads * 4 + 255) & ~(size_t)255;
}

extern "C" pkv_status pkv_kv_attn_weights(const void* q, const void* k_cache, int32_t kv_dtype, const float* k_scale,
                                          int64_t num_blocks, int64_t stride_blk, int64_t stride_tok, int64_t stride_head,
                                          int64_t scale_stride_blk, int64_t scale_stride_tok, const int32_t* block_table,
                                          int64_t bt_stride, int32_t max_blocks, const int32_t* seq_lens,
                                          const int32_t* q_valid, int32_t num_reqs, int32_t T, int32_t num_q_heads,
                                          int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float softmax_scale,
                                          const float* part_lse, int32_t split_tokens, int32_t max_splits,
                                          const float* prev, const int32_t* prev_lens, float* weights,
                                          int64_t w_stride_req, int64_t w_stride_head, int64_t max_ctx, void* workspace,
                                          int64_t workspace_bytes, int32_t* dev_err, void* stream) {
  using namespace pkv;
  clear_error();
  const char* name = "kv_attn_weights";
  PKV_UNSUP(head_dim == kD, "%s: head_dim must be 256 (got %d)", name, head_dim);
  PKV_ARG(kv_dtype >= PKV_KV_BF16 && kv_dtype <= PKV_KV_FP8, "%s: kv_dtype must be bf16, int8 or fp8 (got %d)", name, kv_dtype);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(q && k_cache && block_table && seq_lens && weights && workspace && (kv_dtype == PKV_KV_BF16 || k_scale),
          "%s: null pointer argument", name);
  PKV_ARG(num_reqs > 0 && T > 0 && num_q_heads > 0 && num_kv_heads > 0 && num_blocks > 0 && block_size > 0 &&
              max_blocks > 0 && bt_stride >= max_blocks && max_ctx > 0 && w_stride_req >= 0 && w_stride_head >= 0 &&
              (!part_lse || (split_tokens > 0 && max_splits > 0)),
          "%s: bad size argument", name);
  PKV_UNSUP(num_q_heads % num_kv_heads == 0, "%s: num_q_heads %% num_kv_heads != 0", name);
  PKV_UNSUP(num_q_heads / num_kv_heads <= kMaxCols, "%s: num_q_heads / num_kv_heads must be at most %d (got %d)", name, kMaxCols,
            num_q_heads / num_kv_heads);
  PKV_UNSUP(block_size % 8 == 0, "%s: block_size must be a multiple of 8", name);
  PKV_UNSUP((int64_t)max_blocks * block_size <= INT32_MAX - 127, "%s: max_blocks * block_size must be at most 2^31 - 128", name);
  PKV_UNSUP((int64_t)num_reqs * T * num_q_heads <= INT32_MAX, "%s: too many query rows", name);
  const int64_t es = kv_dtype == PKV_KV_BF16 ? 2 : 1;
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0, "%s: strides must be positive", name);
  PKV_ARG(aligned16(q) && aligned16(k_cache) && stride_blk * es % 16 == 0 && stride_tok * es % 16 == 0 && stride_head * es % 16 == 0,
          "%s: q, the cache and its strides must be 16-byte aligned", name);
  PKV_ARG(((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(prev) | reinterpret_cast<uintptr_t>(part_lse) |
            reinterpret_cast<uintptr_t>(k_scale)) & 3) == 0,
          "%s: fp32 arrays must be 4-byte aligned", name);
  PKV_ARG(kv_dtype != PKV_KV_INT8 || (scale_stride_blk > 0 && scale_stride_tok >= num_kv_heads),
          "%s: scale strides must be positive, with scale_stride_tok >= num_kv_heads", name);
  PKV_ARG(softmax_scale > 0.0f && softmax_scale <= 3.4e38f, "%s: softmax_scale must be positive and finite", name);
  const int64_t need = (int64_t)pkv_kv_attn_weights_workspace_bytes(num_reqs * T, num_q_heads, 1);
  PKV_ARG(aligned16(workspace) && workspace_bytes >= need, "%s: workspace must be 16-byte aligned and hold %lld bytes (got %lld)",
          name, (long long)need, (long long)workspace_bytes);
  WeightParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(k_cache), k_scale, num_blocks, stride_blk,
                 stride_tok, stride_head, scale_stride_blk, scale_stride_tok, block_table, bt_stride, max_blocks, seq_lens,
                 q_valid, num_reqs, T, num_q_heads, num_kv_heads, block_size, softmax_scale, part_lse, split_tokens,
                 max_splits, prev, prev_lens, weights, w_stride_req, w_stride_head, max_ctx,
                 static_cast<float*>(workspace), dev_err};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned rows = (unsigned)num_reqs * T * num_q_heads;
  const dim3 grid(1024, num_reqs, num_kv_heads);
  if (kv_dtype == PKV_KV_BF16) {
    lse_kernel<PKV_KV_BF16><<<rows, 256, 0, st>>>(p);
    weights_kernel<PKV_KV_BF16><<<grid, 256, 0, st>>>(p);
  } else if (kv_dtype == PKV_KV_INT8) {
    lse_kernel<PKV_KV_INT8><<<rows, 256, 0, st>>>(p);
    weights_kernel<PKV_KV_INT8><<<grid, 256, 0, st>>>(p);
  } else {
    lse_kernel<PKV_KV_FP8><<<rows, 256, 0, st>>>(p);
    weights_kernel<PKV_KV_FP8><<<grid, 256, 0, st>>>(p);
  }
  return check_launch(name);
}
