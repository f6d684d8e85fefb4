// kv_fp4_dequant.cu - pkv_kv_fp4_dequant_dense: rows of the paged 4-bit cache back to dense bf16.
//
//   dense[r][pos][h][i] = bf16_rn((e2m1(code) * e4m3(group)) * scale) for pos_begin[r] <= pos < pos_end[r]
// The first product is exact (6 significant bits); the second is one fp32 rounding.
//
// One lane holds one group: 8 bytes of codes and a scale byte in, 32 bytes out (one 256-bit store);
// a warp covers the K row and the V row of one (position, head), four of them in flight. Their places are found
// side by side, a lane each, and handed round: with a walk from one pair to the next, 2.6 million pairs
// took 554 us.
//
// Bound by memory, four fifths of it the stores. Measured: 2.6 million pairs of rows 536 us, 6.4 TB/s in and
// out (0.94 of the measured copy rate); 188,416 pairs 41 us (46 with a cold L2); the smallest calls 2.1 us.
#include <cuda_bf16.h>

#include "host_common.h"
#include "kv_fp4.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 16;  // of an SM: all the warps it holds, 32 registers (2.6 million pairs 535 us; 545 without the bound)

struct ReadArgs {
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
  const int32_t* pos_begin;
  const int32_t* pos_end;
  int32_t block_size, num_kv_heads, chunks;
  __nv_bfloat16* k_dense;
  __nv_bfloat16* v_dense;
  int64_t max_ctx;
  int* dev_err;
};

template <int kPairs>
__global__ void __launch_bounds__(kWarps * 32, kCtas) kv_fp4_dequant_kernel(const ReadArgs a) {
  const int r = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x - r * a.chunks;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t begin = max(__ldg(a.pos_begin + r), 0);
  int64_t end = __ldg(a.pos_end + r);
  if (end > a.max_ctx) {
    if (chunk == 0 && threadIdx.x == 0) record_error(a.dev_err, kErrDeviceBounds);
    end = a.max_ctx;
  }
  if (begin >= end) return;
  const int hkv = a.num_kv_heads;
  const int which = lane >> 4, grp = lane & 15;
  const uint8_t* codes = which ? a.v_fp4 : a.k_fp4;
  const uint8_t* scales = which ? a.v_bscale : a.k_bscale;
  __nv_bfloat16* dense = which ? a.v_dense : a.k_dense;
  const float g = __ldg(which ? a.v_scale : a.k_scale);
  const uint64_t nrows = (uint64_t)(end - begin) * hkv;
  const uint64_t stride = (uint64_t)a.chunks * kWarps * kPairs;
  const int32_t* table = a.block_table + (int64_t)r * a.bt_stride;
  for (uint64_t base = ((uint64_t)chunk * kWarps + warp) * kPairs; base < nrows; base += stride) {
    // lane u finds pair u's place (no table entry past the request's last is read); a warp-uniform offset then
    int64_t off = -1, soff = 0;
    if (lane < kPairs && base + lane < nrows) {
      uint32_t tok, head;
      split_pair(base + lane, hkv, tok, head);
      const uint32_t pos = (uint32_t)begin + tok, col = pos / (uint32_t)a.block_size, slot = pos - col * a.block_size;
      const int64_t blk = col < (uint32_t)a.max_blocks ? __ldg(table + col) : -1;
      if (blk < 0 || blk >= a.num_blocks) {  // reads as zero
        record_error(a.dev_err, kErrDeviceBounds);
      } else {
        off = blk * a.stride_blk + (int64_t)slot * a.stride_tok + (int64_t)head * a.stride_head;
        soff = blk * a.scale_stride_blk + (int64_t)slot * a.scale_stride_tok + (int64_t)head * a.scale_stride_head;
      }
    }
    // the pairs of a request are consecutive rows of the dense tensor
    __nv_bfloat16* dst = dense + (((int64_t)r * a.max_ctx + begin) * hkv + (int64_t)base) * kFp4D + grp * kFp4Group;
    uint2 c[kPairs];
    uint32_t sb[kPairs];
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      c[u] = make_uint2(0, 0);
      sb[u] = 0;
      const int64_t o = __shfl_sync(0xffffffffu, off, u), so = __shfl_sync(0xffffffffu, soff, u);
      if (o >= 0) {
        c[u] = __ldg(reinterpret_cast<const uint2*>(codes + o + grp * 8));
        sb[u] = __ldg(scales + so + grp);
      }
    }
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      if (base + u >= nrows) break;
      const uint32_t s2 = e4m3_dup_f16(sb[u]);
      Bytes32 o;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[4];
        e2m1x8_to_f16(half ? c[u].y : c[u].x, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = hmul2_u32(v[i], s2);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
          o.w[4 * half + i] = pack_bf16x2(__fmul_rn(f.x, g), __fmul_rn(f.y, g));
        }
      }
      stg_bytes32(dst + (int64_t)u * kFp4D, o);
    }
  }
}

}  // namespace

}  // namespace pkv

extern "C" pkv_status pkv_kv_fp4_dequant_dense(
    const uint8_t* k_fp4, const uint8_t* v_fp4, const uint8_t* k_bscale, const uint8_t* v_bscale, const float* k_scale,
    const float* v_scale, int64_t num_blocks, int64_t stride_blk, int64_t stride_tok, int64_t stride_head,
    int64_t scale_stride_blk, int64_t scale_stride_tok, int64_t scale_stride_head, const int32_t* block_table,
    int64_t bt_stride, int32_t max_blocks, const int32_t* pos_begin, const int32_t* pos_end, int32_t num_reqs,
    int32_t max_tokens, int32_t block_size, int32_t num_kv_heads, int32_t head_dim, void* k_dense, void* v_dense,
    int64_t max_ctx, int32_t* dev_err, void* stream) {
  using namespace pkv;
  clear_error();
  PKV_UNSUP(head_dim == kFp4D, "kv_fp4_dequant_dense: head_dim must be 256 (got %d)", head_dim);
  PKV_ARG(num_reqs >= 0 && max_tokens >= 0, "kv_fp4_dequant_dense: bad size argument");
  if (num_reqs == 0 || max_tokens == 0) return PKV_OK;  // nothing to do, nothing read
  PKV_ARG(k_fp4 && v_fp4 && k_bscale && v_bscale && k_scale && v_scale && block_table && pos_begin && pos_end &&
              k_dense && v_dense,
          "kv_fp4_dequant_dense: null pointer argument");
  PKV_ARG(num_blocks > 0 && block_size > 0 && num_kv_heads > 0 && max_blocks > 0 && bt_stride >= max_blocks &&
              max_ctx > 0,
          "kv_fp4_dequant_dense: bad size argument");
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0 && scale_stride_blk > 0 && scale_stride_tok > 0 &&
              scale_stride_head > 0,
          "kv_fp4_dequant_dense: strides must be positive");
  PKV_ARG(aligned16(k_fp4) && aligned16(v_fp4) && aligned16(k_bscale) && aligned16(v_bscale) && stride_blk % 16 == 0 &&
              stride_tok % 16 == 0 && stride_head % 16 == 0 && scale_stride_blk % 16 == 0 &&
              scale_stride_tok % 16 == 0 && scale_stride_head % 16 == 0,
          "kv_fp4_dequant_dense: caches, scale caches and their strides must be 16-byte aligned");
  PKV_ARG((reinterpret_cast<uintptr_t>(k_dense) & 31) == 0 && (reinterpret_cast<uintptr_t>(v_dense) & 31) == 0,
          "kv_fp4_dequant_dense: dense outputs must be 32-byte aligned");
  ReadArgs a{k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale, num_blocks, stride_blk, stride_tok, stride_head,
             scale_stride_blk, scale_stride_tok, scale_stride_head, block_table, bt_stride, max_blocks, pos_begin,
             pos_end, block_size, num_kv_heads, 0, static_cast<__nv_bfloat16*>(k_dense),
             static_cast<__nv_bfloat16*>(v_dense), max_ctx, dev_err};
  // pairs of a warp: 4 in flight where there are enough for every warp the device holds (2.6 million pairs:
  // 535 us against 1,072 with one, 562 with three, 587 with five), else 1 (256 pairs: 2.1 us against 2.8 with
  // four)
  const int64_t rows = (int64_t)max_tokens * num_kv_heads;
  const bool many = rows * num_reqs > (int64_t)num_sms() * kCtas * kWarps * 4;
  const int64_t per_cta = (int64_t)kWarps * (many ? 4 : 1);
  const int64_t want = (rows + per_cta - 1) / per_cta;
  const int64_t cap = ((1ll << 30) - 1) / num_reqs + 1;
  a.chunks = (int32_t)(want < cap ? want : cap);
  PKV_ARG((int64_t)a.chunks * num_reqs < (1ll << 31), "kv_fp4_dequant_dense: grid too large");
  const unsigned grid = (unsigned)(a.chunks * num_reqs);
  if (many)
    kv_fp4_dequant_kernel<4><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  else
    kv_fp4_dequant_kernel<1><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch("kv_fp4_dequant_dense");
}
