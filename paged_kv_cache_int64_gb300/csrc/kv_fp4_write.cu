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
// The quotient is q0 = x inv with inv = 1 / d, corrected by its remainder e = q0 d - x (Markstein's method):
// q0 is within 2^-22 of x / d, e has one rounding of its own, so q0 - e inv is within 2^-45 of x / d before
// its one rounding, at less than half the price of 16 divisions. The code is that of the correctly
// rounded quotient: over all mantissas of d and x the two are equal. Where this could fail by range:
//   - |x| >= d / 8, the elements that a threshold (d / 4 or more) can concern: for d in [2^-80, 2^100] and x at
//     most 16 d, q0 and inv are normal and e is a multiple of 2^-129, so nothing underflows or overflows;
//   - smaller elements: e may underflow, which moves the quotient by 2^-70 at most, and the code is 0 with the
//     sign of x either way.
// Groups outside these ranges of d and x take the division itself.
//
// Measured (pairs of a K and a V row of 256): 570,184 pairs 137 us, 5.5 TB/s in and out; 8,192 pairs 4.6
// us; the smallest calls 2.2 to 2.5 us, launch and three dependent loads. Large calls are bound by the
// instructions of the conversion, small ones by latency.
#include <cuda_bf16.h>

#include "host_common.h"
#include "kv_fp4.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;
constexpr int kDepth = 2;  // (token, head) pairs a warp has in flight
// CTAs of an SM: 64 registers, one more warp of four to a scheduler than without the bound (570,184 pairs:
// 137 us against 143; three pairs in flight instead 146, ten CTAs 141)
constexpr int kCtas = 8;

// Pairs of a warp: as many as leave the device the warps that it holds, at most 16. Long walks spread a
// warp's start (launch, lengths, table: three dependent loads) over more rows; short ones are all that
// small calls have (570,184 pairs: 137 us with 16, 139 with 12, 357 with one; 8,192 pairs: 4.6 us with
// two, 5.5 with one, 8.1 with 16).
constexpr int64_t kPairsMost = 16;
int32_t pairs_per_warp(int64_t pairs) {
  const int64_t device_warps = (int64_t)num_sms() * kCtas * kWarps;
  const int64_t per = (pairs + device_warps - 1) / device_warps;
  return (int32_t)(per < 1 ? 1 : per > kPairsMost ? kPairsMost : per);
}

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
  int32_t block_size, num_kv_heads, chunks, per;
  int* dev_err;
};

// The division itself, for groups outside the range of the corrected product: 8 elements. By value and
// out of line: its registers are not the common path's.
__device__ __noinline__ uint32_t quantize8_slow(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float d) {
  const bool zero = !(d >= 0x1p-126f && d <= 3.4028234e38f);
  const uint32_t w[4] = {w0, w1, w2, w3};
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    x[i] = copysignf(zero ? 0.0f : __fdiv_rn(v, d), v);
  }
  return e2m1x8_rn(x);
}

// 16 bf16 elements -> 8 bytes of codes and the group's scale byte.
__device__ __forceinline__ uint2 quantize_group(const Bytes32& in, float g, float g6, uint32_t& scale_byte) {
  // |x| as bf16 bit patterns: their unsigned order is the order of the magnitudes, and a pattern past
  // 0x7f80 is a NaN
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, in.w[i] & 0x7fff7fffu);
  const uint32_t mx = max(m & 0xffffu, m >> 16);
  const float amax = __uint_as_float(mx << 16);
  uint16_t s2;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(__fdiv_rn(amax, g6)));
  const uint32_t sh = e4m3_dup_f16(s2);
  const float d = __fmul_rn(__low2float(*reinterpret_cast<const __half2*>(&sh)), g);
  scale_byte = s2 & 0xffu;
  if (!(d >= 0x1p-80f && d <= 0x1p100f && amax <= __fmul_rn(16.0f, d))) {
    if (mx > 0x7f80u) {
      scale_byte = 0x7fu;
      return make_uint2(0, 0);
    }
    return make_uint2(quantize8_slow(in.w[0], in.w[1], in.w[2], in.w[3], d), quantize8_slow(in.w[4], in.w[5], in.w[6], in.w[7], d));
  }
  // (with e = q0 d - x, not x - q0 d, a negative zero keeps its sign)
  const float inv = __fdiv_rn(1.0f, d);
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = in.w[4 * h + i / 2];
      const float v = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
      const float q0 = __fmul_rn(v, inv);
      x[i] = __fmaf_rn(-__fmaf_rn(q0, d, -v), inv, q0);
    }
    c[h] = e2m1x8_rn(x);
  }
  return make_uint2(c[0], c[1]);
}

__global__ void __launch_bounds__(kWarps * 32, kCtas) kv_fp4_write_kernel(const WriteArgs a) {
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
  const uint64_t nrows = (uint64_t)q_len * hkv;  // (token, head) pairs
  const uint64_t stride = (uint64_t)a.chunks * kWarps * a.per;
  const int32_t* table = a.block_table + (int64_t)r * a.bt_stride;
  for (uint64_t base = ((uint64_t)chunk * kWarps + warp) * a.per; base < nrows; base += stride) {
    const int n = (int)min((uint64_t)a.per, nrows - base);
    PairWalk at(table, hkv, a.block_size, a.max_blocks, (uint32_t)(seq_len - q_len), (uint32_t)seq_len, base);
    Bytes32 raw[kDepth];
    int64_t off[kDepth], soff[kDepth];
    auto fetch = [&](int u, bool live) {
      off[u] = -1;
      if (!live) return;
      raw[u] = ldg_bytes32(src + (int64_t)(q0 + at.i) * a.new_stride_tok + (int64_t)at.h * kFp4D + grp * kFp4Group);
      if (at.blk < 0 || at.blk >= a.num_blocks) {
        if (lane == 0) record_error(a.dev_err, kErrDeviceBounds);  // not written
      } else {
        off[u] = (int64_t)at.blk * a.stride_blk + (int64_t)at.slot * a.stride_tok + (int64_t)at.h * a.stride_head + grp * 8;
        soff[u] = (int64_t)at.blk * a.scale_stride_blk + (int64_t)at.slot * a.scale_stride_tok +
                  (int64_t)at.h * a.scale_stride_head + grp;
      }
      at.next();
    };
#pragma unroll
    for (int u = 0; u < kDepth; ++u) fetch(u, u < n);
    for (int k = 0; k < n; k += kDepth) {
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        if (off[u] >= 0) {  // warp-uniform: one table entry a pair
          uint32_t sb;
          const uint2 c = quantize_group(raw[u], g, g6, sb);
          *reinterpret_cast<uint2*>(codes + off[u]) = c;
          scales[soff[u]] = (uint8_t)sb;
        }
        fetch(u, k + kDepth + u < n);
      }
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
              k_scale, v_scale, block_size, num_kv_heads, 0, 0, dev_err};
  const int64_t rows = (int64_t)max_q_len * num_kv_heads;
  a.per = pairs_per_warp(rows * num_reqs);
  const int64_t per_cta = (int64_t)kWarps * a.per;
  const int64_t want = (rows + per_cta - 1) / per_cta;
  const int64_t cap = ((1ll << 30) - 1) / num_reqs + 1;  // the grid's x extent stays below 2^31
  a.chunks = (int32_t)(want < cap ? want : cap);
  PKV_ARG((int64_t)a.chunks * num_reqs < (1ll << 31), "kv_cache_write_fp4: grid too large");
  kv_fp4_write_kernel<<<(unsigned)(a.chunks * num_reqs), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return check_launch("kv_cache_write_fp4");
}
