// kv_fp4_write.cu - pkv_kv_cache_write_fp4: quantize a chunk's new K/V rows to 4 bits and store them
// into the paged cache through the block table.
//
// Per group of 16 elements x, with g the tensor's fp32 scale:
//   a = max |x|;  s = e4m3(a / (6 g)), to nearest even, at most 448;  d = s g;
//   code = e2m1(x / d), to nearest even, magnitudes past 6 stored as 6; the sign is x's.
// All divisions and products are single fp32 roundings. d = 0, subnormal or infinite: the magnitudes
// are 0. A NaN in the group: the scale is NaN, the codes 0.
//
// One lane holds one group: 32 bytes in (one 256-bit load), 8 bytes of codes and 1 byte of scale
// out, so nothing crosses lanes; a warp covers a K row and its V row (same token and head) at once.
// The quotient is q0 = x inv with inv = 1 / d, corrected by its exact remainder: r = x - q0 d is
// exact in one fma, and q0 + r inv is within 2^-46 of x / d before its one rounding, so the code is
// that of the correctly rounded quotient at less than half the price of 16 divisions; groups where
// an intermediate could overflow or underflow take the division itself.
#include <cuda_bf16.h>

#include "host_common.h"
#include "kv_fp4.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kIter = 4;  // (token, head) pairs a warp has in flight

struct WriteArgs {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t new_stride_tok;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  const int32_t* qsl;
  uint8_t* k_fp4;
  uint8_t* v_fp4;
  int64_t num_blocks, stride_blk, stride_tok, stride_head;  // bytes
  uint8_t* k_bscale;
  uint8_t* v_bscale;
  int64_t scale_stride_blk, scale_stride_tok, scale_stride_head;
  const float* k_scale;
  const float* v_scale;
  int32_t block_size, num_kv_heads, chunks;
  int* dev_err;
};

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// 16 bf16 elements -> 8 bytes of codes and the group's scale byte.
__device__ __forceinline__ uint2 quantize_group(const Bytes32& in, float g, float g6, uint32_t& scale_byte) {
  // |x| as bf16 bit patterns: their unsigned order is the order of the magnitudes, and a pattern past
  // 0x7f80 is a NaN
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, in.w[i] & 0x7fff7fffu);
  const uint32_t mx = max(m & 0xffffu, m >> 16);
  if (mx > 0x7f80u) {
    scale_byte = 0x7fu;
    return make_uint2(0, 0);
  }
  const float amax = __uint_as_float(mx << 16);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(__fdiv_rn(amax, g6)));
  scale_byte = s2 & 0xffu;
  const uint32_t sh = e4m3_dup_f16(scale_byte);
  const float d = __fmul_rn(__low2float(*reinterpret_cast<const __half2*>(&sh)), g);
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(in.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(in.w[i] & 0xffff0000u);
  }
  if (d >= 0x1p-80f && d <= 0x1p100f && amax <= __fmul_rn(16.0f, d)) {
    const float inv = __fdiv_rn(1.0f, d);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q0 = __fmul_rn(x[i], inv);
      x[i] = copysignf(__fmaf_rn(__fmaf_rn(-q0, d, x[i]), inv, q0), x[i]);
    }
  } else {
    const bool zero = !(d >= 0x1p-126f && d <= 3.4028234e38f);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = copysignf(zero ? 0.0f : __fdiv_rn(x[i], d), x[i]);
  }
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = e2m1x2(x[8 * h + 2 * i], x[8 * h + 2 * i + 1]);
    c[h] = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
  }
  return make_uint2(c[0], c[1]);
}

__global__ void __launch_bounds__(kWarps * 32) kv_fp4_write_kernel(const WriteArgs a) {
  const int r = blockIdx.x / a.chunks;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int q0 = __ldg(a.qsl + r);
  const int q_len = __ldg(a.qsl + r + 1) - q0;
  const int seq_len = __ldg(a.seq_lens + r);
  const int chunk = blockIdx.x - r * a.chunks;
  if (q_len <= 0) return;
  if (q_len > seq_len) {  // the chunk would start before position 0: nothing is written
    if (chunk == 0 && threadIdx.x == 0) record_error(a.dev_err, kErrDeviceBounds);
    return;
  }
  const int hkv = a.num_kv_heads;
  const int which = lane >> 4, grp = lane & 15;  // lanes 0-15: the K row's groups, 16-31: the V row's
  const float g = __ldg(which ? a.v_scale : a.k_scale);
  const float g6 = __fmul_rn(6.0f, g);
  const __nv_bfloat16* src = which ? a.v_new : a.k_new;
  uint8_t* codes = which ? a.v_fp4 : a.k_fp4;
  uint8_t* scales = which ? a.v_bscale : a.k_bscale;
  const int64_t nrows = (int64_t)q_len * hkv;  // (token, head) pairs
  const int64_t stride = (int64_t)a.chunks * kWarps * kIter;
  for (int64_t base = ((int64_t)chunk * kWarps + warp) * kIter; base < nrows; base += stride) {
    Bytes32 raw[kIter];
    int64_t off[kIter], soff[kIter];
#pragma unroll
    for (int u = 0; u < kIter; ++u) {
      const int64_t row = base + u;
      off[u] = -1;
      if (row >= nrows) continue;
      const int h = (int)(row % hkv);
      const int i = (int)(row / hkv);
      const int64_t pos = (int64_t)seq_len - q_len + i;
      const int64_t col = pos / a.block_size;
      const int64_t blk = col < a.max_blocks ? (int64_t)__ldg(a.block_table + (int64_t)r * a.bt_stride + col) : -1;
      if (blk < 0 || blk >= a.num_blocks) {
        if (lane == 0) record_error(a.dev_err, kErrDeviceBounds);
        continue;  // not written
      }
      const int64_t slot = pos % a.block_size;
      off[u] = blk * a.stride_blk + slot * a.stride_tok + (int64_t)h * a.stride_head + grp * 8;
      soff[u] = blk * a.scale_stride_blk + slot * a.scale_stride_tok + (int64_t)h * a.scale_stride_head + grp;
      raw[u] = ldg_bytes32(src + (int64_t)(q0 + i) * a.new_stride_tok + (int64_t)h * kFp4D + grp * kFp4Group);
    }
#pragma unroll
    for (int u = 0; u < kIter; ++u) {
      if (off[u] < 0) continue;  // warp-uniform: one table entry per pair
      uint32_t sb;
      const uint2 c = quantize_group(raw[u], g, g6, sb);
      *reinterpret_cast<uint2*>(codes + off[u]) = c;
      scales[soff[u]] = (uint8_t)sb;
    }
  }
}

}  // namespace

}  // namespace pkv

extern "C" pkv_status pkv_kv_cache_write_fp4(
    const void* k_new, const void* v_new, int64_t new_stride_tok, const int32_t* block_table, int64_t bt_stride,
    int32_t max_blocks, const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_reqs, int32_t max_q_len,
    uint8_t* k_fp4, uint8_t* v_fp4, uint8_t* k_bscale, uint8_t* v_bscale, const float* k_scale, const float* v_scale,
    int64_t num_blocks, int64_t stride_blk, int64_t stride_tok, int64_t stride_head, int64_t scale_stride_blk,
    int64_t scale_stride_tok, int64_t scale_stride_head, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
    int32_t* dev_err, void* stream) {
  using namespace pkv;
  clear_error();
  PKV_UNSUP(head_dim == kFp4D, "kv_cache_write_fp4: head_dim must be 256 (got %d)", head_dim);
  PKV_ARG(num_reqs >= 0 && max_q_len >= 0, "kv_cache_write_fp4: bad size argument");
  if (num_reqs == 0 || max_q_len == 0) return PKV_OK;  // nothing to do, nothing read
  PKV_ARG(k_new && v_new && block_table && seq_lens && query_start_loc && k_fp4 && v_fp4 && k_bscale && v_bscale &&
              k_scale && v_scale,
          "kv_cache_write_fp4: null pointer argument");
  PKV_ARG(num_blocks > 0 && block_size > 0 && num_kv_heads > 0 && max_blocks > 0 && bt_stride >= max_blocks &&
              new_stride_tok >= (int64_t)num_kv_heads * kFp4D,
          "kv_cache_write_fp4: bad size argument");
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0 && scale_stride_blk > 0 && scale_stride_tok > 0 &&
              scale_stride_head > 0,
          "kv_cache_write_fp4: strides must be positive");
  // a lane reads 32 bytes and writes 8 bytes of codes
  PKV_ARG((reinterpret_cast<uintptr_t>(k_new) & 31) == 0 && (reinterpret_cast<uintptr_t>(v_new) & 31) == 0 &&
              new_stride_tok % 16 == 0,
          "kv_cache_write_fp4: new rows must be 32-byte aligned, with a token stride of a multiple of 16 elements");
  PKV_ARG(aligned16(k_fp4) && aligned16(v_fp4) && aligned16(k_bscale) && aligned16(v_bscale) && stride_blk % 16 == 0 &&
              stride_tok % 16 == 0 && stride_head % 16 == 0 && scale_stride_blk % 16 == 0 &&
              scale_stride_tok % 16 == 0 && scale_stride_head % 16 == 0,
          "kv_cache_write_fp4: caches, scale caches and their strides must be 16-byte aligned");
  WriteArgs a{static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new), new_stride_tok,
              block_table, bt_stride, max_blocks, seq_lens, query_start_loc, k_fp4, v_fp4, num_blocks, stride_blk,
              stride_tok, stride_head, k_bscale, v_bscale, scale_stride_blk, scale_stride_tok, scale_stride_head,
              k_scale, v_scale, block_size, num_kv_heads, 0, dev_err};
  const int64_t rows = (int64_t)max_q_len * num_kv_heads, per_cta = (int64_t)kWarps * kIter;
  const int64_t want = (rows + per_cta - 1) / per_cta;
  const int64_t cap = ((1ll << 30) - 1) / num_reqs + 1;  // the grid's x extent stays below 2^31
  a.chunks = (int32_t)(want < cap ? want : cap);
  PKV_ARG((int64_t)a.chunks * num_reqs < (1ll << 31), "kv_cache_write_fp4: grid too large");
  kv_fp4_write_kernel<<<(unsigned)(a.chunks * num_reqs), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch("kv_cache_write_fp4");
}
