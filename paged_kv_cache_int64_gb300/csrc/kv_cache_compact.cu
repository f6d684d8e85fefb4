// kv_cache_compact.cu - pkv_kv_cache_compact: the rows that stay move to the front of their cache.
//
// Row j of (request r, KV head h) becomes row keep[r][h][j], in K, in V, in the scale caches and in the weights; in
// place, or into other blocks. keep ascends, so keep[j] >= j: a row moves down or stays.
#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;  // rows of a chunk

struct CompactParams {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  int64_t num_blocks, stride_blk, stride_tok, stride_head;        // bytes
  int64_t s_stride_blk, s_stride_tok, s_stride_head;              // bytes
  const int32_t* src_table;
  const int32_t* dst_table;
  int64_t src_stride, dst_stride;
  int32_t src_blocks, dst_blocks;
  const int32_t* keep;
  const int32_t* new_lens;
  int32_t num_kv_heads, budget, block_size;
  float* weights;
  int64_t w_stride_req, w_stride_head, max_ctx;
  int* dev_err;
};

struct Row {
  int blk, slot;  // blk < 0: the row does not move
};

// kPieces: 16-byte pieces of a row; kScale: bytes of a row's scales (0, 4 or 16).
template <int kPieces, int kScale>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p) {
  constexpr int kPer = 2 * kRows * kPieces / kThreads;  // pieces a thread, K and V
  __shared__ Row s_src[kRows], s_dst[kRows];
  const int unit = blockIdx.x;
  const int r = unit / p.num_kv_heads, h = unit - r * p.num_kv_heads;
  const int tid = threadIdx.x;
  const int32_t* keep = p.keep + (int64_t)unit * p.budget;
  const int32_t* src_table = p.src_table + (int64_t)r * p.src_stride;
  const int32_t* dst_table = p.dst_table + (int64_t)r * p.dst_stride;
  const int len = __ldg(p.new_lens + r);
  const int n = max(0, min(len, p.budget));
  if (tid == 0 && (len < 0 || len > p.budget)) record_error(p.dev_err, kErrDeviceBounds);
  float* w = p.weights ? p.weights + (int64_t)r * p.w_stride_req + (int64_t)h * p.w_stride_head : nullptr;
  for (int j0 = 0; j0 < n; j0 += kRows) {
    float wv = 0.0f;
    bool w_moves = false;
    if (tid < kRows) {
      Row a{-1, 0}, b{-1, 0};
      const int j = j0 + tid;
      if (j < n) {
        const int from = __ldg(keep + j);
        const int col = from / p.block_size, dcol = j / p.block_size;
        bool ok = from >= j && (j == 0 || from > __ldg(keep + j - 1)) && col < p.src_blocks && dcol < p.dst_blocks;
        if (ok) {
          a = {__ldg(src_table + col), from - col * p.block_size};
          b = {__ldg(dst_table + dcol), j - dcol * p.block_size};
          ok = a.blk >= 0 && a.blk < p.num_blocks && b.blk >= 0 && b.blk < p.num_blocks;
        }
        if (ok && w) {
          ok = from < p.max_ctx;
          if (ok && from != j) {
            wv = w[from];
            w_moves = true;
          }
        }
        if (!ok) record_error(p.dev_err, kErrDeviceBounds);
        if (!ok || (a.blk == b.blk && a.slot == b.slot)) a.blk = -1;
      }
      s_src[tid] = a;
      s_dst[tid] = b;
    }
    __syncthreads();
    uint4 x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int piece = i * kThreads + tid;
      const int row = piece / kPieces & (kRows - 1);
      const uint8_t* pool = i < kPer / 2 ? p.k : p.v;
      const Row a = s_src[row];
      if (a.blk >= 0)
        x[i] = *reinterpret_cast<const uint4*>(pool + a.blk * p.stride_blk + a.slot * p.stride_tok + h * p.stride_head +
                                               piece % kPieces * 16);
    }
    uint4 sx = make_uint4(0, 0, 0, 0);
    const int srow = tid & (kRows - 1);
    uint8_t* spool = tid < kRows ? p.ks : p.vs;
    const bool scales = kScale && tid < 2 * kRows && s_src[srow].blk >= 0;
    if (scales) {
      const Row a = s_src[srow];
      const uint8_t* at = spool + a.blk * p.s_stride_blk + a.slot * p.s_stride_tok + h * p.s_stride_head;
      if (kScale == 4) sx.x = *reinterpret_cast<const uint32_t*>(at);
      if (kScale == 16) sx = *reinterpret_cast<const uint4*>(at);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int piece = i * kThreads + tid;
      const int row = piece / kPieces & (kRows - 1);
      uint8_t* pool = i < kPer / 2 ? p.k : p.v;
      const Row b = s_dst[row];
      if (s_src[row].blk >= 0)
        *reinterpret_cast<uint4*>(pool + b.blk * p.stride_blk + b.slot * p.stride_tok + h * p.stride_head +
                                  piece % kPieces * 16) = x[i];
    }
    if (scales) {
      const Row b = s_dst[srow];
      uint8_t* at = spool + b.blk * p.s_stride_blk + b.slot * p.s_stride_tok + h * p.s_stride_head;
      if (kScale == 4) *reinterpret_cast<uint32_t*>(at) = sx.x;
      if (kScale == 16) *reinterpret_cast<uint4*>(at) = sx;
    }
    if (w_moves) w[j0 + tid] = wv;
    __syncthreads();
  }
}

template <int kPieces, int kScale>
pkv_status launch(const CompactParams& p, int units, cudaStream_t st) {
  compact_kernel<kPieces, kScale><<<units, kThreads, 0, st>>>(p);
  return check_launch("kv_cache_compact");
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_kv_cache_compact_workspace_bytes(int32_t num_reqs, int32_t num_kv_heads, int32_t budget) {
  if (num_reqs <= 0 || num_kv_heads <= 0 || budget <= 0) return 0;
  const size_t chunks = ((size_t)budget + pkv::kRows - 1) / pkv::kRows;
  return ((size_t)num_reqs * (size_t)num_kv_heads * chunks * 4 + 255) & ~(size_t)255;
}

extern "C" pkv_status pkv_kv_cache_compact(void* k_cache, void* v_cache, int32_t kv_dtype, int64_t num_blocks,
                                           int64_t stride_blk, int64_t stride_tok, int64_t stride_head, void* k_scale,
                                           void* v_scale, int64_t scale_stride_blk, int64_t scale_stride_tok,
                                           int64_t scale_stride_head, const int32_t* src_table, int64_t src_stride,
                                           int32_t src_blocks, const int32_t* dst_table, int64_t dst_stride,
                                           int32_t dst_blocks, const int32_t* keep, const int32_t* new_lens,
                                           int32_t num_reqs, int32_t num_kv_heads, int32_t budget, int32_t block_size,
                                           int32_t head_dim, float* weights, int64_t w_stride_req, int64_t w_stride_head,
                                           int64_t max_ctx, void* workspace, int64_t workspace_bytes, int32_t* dev_err,
                                           void* stream) {
  using namespace pkv;
  clear_error();
  const char* name = "kv_cache_compact";
  PKV_UNSUP(head_dim == 256, "%s: head_dim must be 256 (got %d)", name, head_dim);
  PKV_ARG(kv_dtype >= PKV_KV_BF16 && kv_dtype <= PKV_KV_FP4, "%s: kv_dtype must be one of pkv_kv_dtype (got %d)", name, kv_dtype);
  PKV_ARG(num_reqs >= 0 && num_kv_heads > 0 && num_blocks > 0 && block_size > 0 && src_blocks > 0 && dst_blocks > 0 &&
              src_stride >= src_blocks && dst_stride >= dst_blocks && budget > 0,
          "%s: bad size argument", name);
  const bool scaled = kv_dtype == PKV_KV_INT8 || kv_dtype == PKV_KV_FP4;
  PKV_UNSUP((int64_t)num_reqs * num_kv_heads <= INT32_MAX, "%s: too many requests", name);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(k_cache && v_cache && src_table && dst_table && keep && new_lens && workspace && (!scaled || (k_scale && v_scale)),
          "%s: null pointer argument", name);
  const int64_t es = kv_dtype == PKV_KV_BF16 ? 2 : 1, ss = kv_dtype == PKV_KV_INT8 ? 4 : 1;
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0 &&
              (!scaled || (scale_stride_blk > 0 && scale_stride_tok > 0 && scale_stride_head > 0)),
          "%s: strides must be positive", name);
  PKV_ARG(aligned16(k_cache) && aligned16(v_cache) && stride_blk * es % 16 == 0 && stride_tok * es % 16 == 0 &&
              stride_head * es % 16 == 0,
          "%s: caches and their strides must be 16-byte aligned", name);
  if (kv_dtype == PKV_KV_INT8)
    PKV_ARG(((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3) == 0,
            "%s: scale caches must be 4-byte aligned", name);
  if (kv_dtype == PKV_KV_FP4)
    PKV_ARG(aligned16(k_scale) && aligned16(v_scale) && scale_stride_blk % 16 == 0 && scale_stride_tok % 16 == 0 &&
                scale_stride_head % 16 == 0,
            "%s: scale caches and their strides must be 16-byte aligned", name);
  PKV_ARG(!weights || (max_ctx > 0 && w_stride_req >= 0 && w_stride_head >= 0 && (reinterpret_cast<uintptr_t>(weights) & 3) == 0),
          "%s: bad weights", name);
  const int64_t need = (int64_t)pkv_kv_cache_compact_workspace_bytes(num_reqs, num_kv_heads, budget);
  PKV_ARG((reinterpret_cast<uintptr_t>(workspace) & 3) == 0 && workspace_bytes >= need,
          "%s: workspace must be 4-byte aligned and hold %lld bytes (got %lld)", name, (long long)need, (long long)workspace_bytes);
  CompactParams p{};
  p.k = static_cast<uint8_t*>(k_cache);
  p.v = static_cast<uint8_t*>(v_cache);
  p.ks = static_cast<uint8_t*>(k_scale);
  p.vs = static_cast<uint8_t*>(v_scale);
  p.num_blocks = num_blocks;
  p.stride_blk = stride_blk * es, p.stride_tok = stride_tok * es, p.stride_head = stride_head * es;
  p.s_stride_blk = scale_stride_blk * ss, p.s_stride_tok = scale_stride_tok * ss, p.s_stride_head = scale_stride_head * ss;
  p.src_table = src_table, p.dst_table = dst_table;
  p.src_stride = src_stride, p.dst_stride = dst_stride;
  p.src_blocks = src_blocks, p.dst_blocks = dst_blocks;
  p.keep = keep, p.new_lens = new_lens;
  p.num_kv_heads = num_kv_heads, p.budget = budget, p.block_size = block_size;
  p.weights = weights, p.w_stride_req = w_stride_req, p.w_stride_head = w_stride_head, p.max_ctx = max_ctx;
  p.dev_err = dev_err;
  const int units = num_reqs * num_kv_heads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (kv_dtype) {
    case PKV_KV_BF16: return launch<32, 0>(p, units, st);
    case PKV_KV_INT8: return launch<16, 4>(p, units, st);
    case PKV_KV_FP8: return launch<16, 0>(p, units, st);
    default: return launch<8, 16>(p, units, st);
  }
}
