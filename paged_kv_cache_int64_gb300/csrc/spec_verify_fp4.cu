// spec_verify_fp4.cu - pkv_spec_verify_attn_fp4: decode / speculative-verify attention over the paged
// 4-bit cache.
//
// One CTA per query row (token, head): its 8 warps stride over the keys, each with a running maximum
// and sum; a lane holds 8 of the 256 dimensions. The warps' partials are merged in shared memory.
#include <cuda_bf16.h>

#include "host_common.h"
#include "kv_fp4.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;

struct Args {
  const __nv_bfloat16* q;
  const uint8_t* k_fp4;
  const uint8_t* v_fp4;
  const uint8_t* k_bscale;
  const uint8_t* v_bscale;
  const float* k_scale;
  const float* v_scale;
  int64_t num_blocks, stride_blk, stride_tok, stride_head;
  int64_t scale_stride_blk, scale_stride_tok, scale_stride_head;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t T, num_q_heads, group, block_size;
  float scale_log2;
  __nv_bfloat16* out;
  int* dev_err;
};

__device__ __forceinline__ void row8(const uint8_t* codes, const uint8_t* scales, int lane, float (&x)[8]) {
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + lane);
  const uint32_t s2 = e4m3_dup_f16(__ldg(scales + (lane >> 1)));
  uint32_t v[4];
  e2m1x8_to_f16(w, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = hmul2_u32(v[i], s2);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__global__ void __launch_bounds__(kWarps * 32) spec_verify_fp4_kernel(const Args a) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kFp4D];
  const int64_t row = blockIdx.x;
  const int qh = (int)(row % a.num_q_heads);
  const int64_t tok = row / a.num_q_heads;
  const int r = (int)(tok / a.T), t = (int)(tok % a.T);
  const int h = qh / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = __ldg(a.seq_lens + r) - a.T + t + 1;  // visible keys
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __bfloat162float(a.q[row * kFp4D + lane * 8 + i]);
  const float f = a.scale_log2 * __ldg(a.k_scale);
  float m = -INFINITY, l = 0.0f, o[8] = {};
  for (int pos = warp; pos < n; pos += kWarps) {
    const int col = pos / a.block_size, slot = pos % a.block_size;
    const int64_t blk = col < a.max_blocks ? (int64_t)__ldg(a.block_table + (int64_t)r * a.bt_stride + col) : -1;
    float s = 0.0f, v[8] = {};
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) record_error(a.dev_err, kErrDeviceBounds);
    } else {
      const int64_t off = blk * a.stride_blk + slot * a.stride_tok + (int64_t)h * a.stride_head;
      const int64_t soff = blk * a.scale_stride_blk + slot * a.scale_stride_tok + (int64_t)h * a.scale_stride_head;
      float k[8];
      row8(a.k_fp4 + off, a.k_bscale + soff, lane, k);
      row8(a.v_fp4 + off, a.v_bscale + soff, lane, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += q[i] * k[i];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    }
    s *= f;
    const float m_new = fmaxf(m, s);
    const float alpha = exp2f(m - m_new), p = exp2f(s - m_new);
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * alpha + p * v[i];
    m = m_new;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s_o[warp][lane * 8 + i] = o[i];
  __syncthreads();
  const int d = threadIdx.x;
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  float L = 0.0f, O = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    if (s_m[w] == -INFINITY) continue;
    const float e = exp2f(s_m[w] - M);
    L += e * s_l[w];
    O += e * s_o[w][d];
  }
  a.out[row * kFp4D + d] = __float2bfloat16(n > 0 ? O / L * __ldg(a.v_scale) : 0.0f);
}

constexpr size_t kWorkspacePerCta = 2 * (32 * kFp4D + 32) * sizeof(float) + 256;

}  // namespace

}  // namespace pkv

extern "C" size_t pkv_spec_verify_fp4_workspace_bytes(int32_t num_ctas) {
  return num_ctas > 0 ? (size_t)num_ctas * pkv::kWorkspacePerCta : 0;
}

extern "C" pkv_status pkv_spec_verify_attn_fp4(
    const void* q, const uint8_t* k_fp4, const uint8_t* v_fp4, const uint8_t* k_bscale, const uint8_t* v_bscale,
    const float* k_scale, const float* v_scale, int64_t num_blocks, int64_t stride_blk, int64_t stride_tok,
    int64_t stride_head, int64_t scale_stride_blk, int64_t scale_stride_tok, int64_t scale_stride_head,
    const int32_t* block_table, int64_t bt_stride, int32_t max_blocks, const int32_t* seq_lens, int32_t num_reqs,
    int32_t T, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float softmax_scale,
    void* out, void* workspace, int64_t workspace_bytes, int32_t* dev_err, void* stream) {
  using namespace pkv;
  constexpr const char* name = "spec_verify_attn_fp4";
  clear_error();
  PKV_UNSUP(head_dim == kFp4D, "%s: head_dim must be 256 (got %d)", name, head_dim);
  if (num_reqs == 0) return PKV_OK;  // nothing to do, nothing read
  PKV_ARG(q && k_fp4 && v_fp4 && k_bscale && v_bscale && k_scale && v_scale && block_table && seq_lens && out &&
              workspace,
          "%s: null pointer argument", name);
  PKV_ARG(num_reqs > 0 && T > 0 && num_q_heads > 0 && num_kv_heads > 0 && num_blocks > 0 && block_size > 0 &&
              max_blocks > 0 && bt_stride >= max_blocks,
          "%s: bad size argument", name);
  PKV_UNSUP(num_q_heads % num_kv_heads == 0, "%s: num_q_heads %% num_kv_heads != 0", name);
  const int group = num_q_heads / num_kv_heads;
  PKV_UNSUP(group <= 32, "%s: num_q_heads / num_kv_heads must be at most 32 (got %d)", name, group);
  PKV_UNSUP(block_size % 8 == 0, "%s: block_size must be a multiple of 8", name);
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0 && scale_stride_blk > 0 && scale_stride_tok > 0 &&
              scale_stride_head > 0,
          "%s: strides must be positive", name);
  PKV_ARG(aligned16(q) && aligned16(out) && aligned16(workspace) && aligned16(k_fp4) && aligned16(v_fp4) &&
              aligned16(k_bscale) && aligned16(v_bscale) && stride_blk % 16 == 0 && stride_tok % 16 == 0 &&
              stride_head % 16 == 0 && scale_stride_blk % 16 == 0 && scale_stride_tok % 16 == 0 &&
              scale_stride_head % 16 == 0,
          "%s: q, out, workspace, caches, scale caches and their strides must be 16-byte aligned", name);
  PKV_ARG(softmax_scale > 0.0f, "%s: softmax_scale must be positive", name);
  PKV_ARG(workspace_bytes >= (int64_t)kWorkspacePerCta, "%s: the workspace needs at least %zu bytes", name,
          kWorkspacePerCta);
  const int64_t rows = (int64_t)num_reqs * T * num_q_heads;
  PKV_ARG(rows < (1ll << 31), "%s: num_reqs * T * num_q_heads too large", name);
  Args a{static_cast<const __nv_bfloat16*>(q), k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale, num_blocks,
         stride_blk, stride_tok, stride_head, scale_stride_blk, scale_stride_tok, scale_stride_head, block_table,
         bt_stride, max_blocks, seq_lens, T, num_q_heads, group, block_size, softmax_scale * 1.4426950408889634f,
         static_cast<__nv_bfloat16*>(out), dev_err};
  spec_verify_fp4_kernel<<<(unsigned)rows, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch(name);
}
