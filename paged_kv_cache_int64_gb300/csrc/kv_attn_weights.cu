// kv_attn_weights.cu - pkv_kv_attn_weights: the attention weight that each cached key collects (checks, tensor maps and
// passes; the kernel is in kv_attn_weights.cuh).
#include "kv_attn_weights.cuh"

namespace pkv {
namespace {

constexpr size_t kStatBytes = 2 * kWMaxCols * sizeof(float2);  // a CTA's

size_t lse_bytes(int64_t rows) { return ((size_t)rows * 4 + 255) & ~(size_t)255; }

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_kv_attn_weights_workspace_bytes(int32_t num_rows, int32_t num_q_heads, int32_t num_ctas) {
  if (num_rows <= 0 || num_q_heads <= 0 || num_ctas <= 0) return 0;
  return pkv::lse_bytes((int64_t)num_rows * num_q_heads) + (size_t)num_ctas * pkv::kStatBytes;
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
  PKV_UNSUP(head_dim == kWD, "%s: head_dim must be 256 (got %d)", name, head_dim);
  PKV_ARG(kv_dtype >= PKV_KV_BF16 && kv_dtype <= PKV_KV_FP8, "%s: kv_dtype must be bf16, int8 or fp8 (got %d)", name, kv_dtype);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(q && k_cache && block_table && seq_lens && weights && workspace && (kv_dtype == PKV_KV_BF16 || k_scale),
          "%s: null pointer argument", name);
  PKV_ARG(num_reqs > 0 && T > 0 && num_q_heads > 0 && num_kv_heads > 0 && num_blocks > 0 && block_size > 0 &&
              max_blocks > 0 && bt_stride >= max_blocks && max_ctx > 0 && w_stride_req >= 0 && w_stride_head >= 0 &&
              (!part_lse || (split_tokens > 0 && max_splits > 0)),
          "%s: bad size argument", name);
  PKV_UNSUP(num_q_heads % num_kv_heads == 0, "%s: num_q_heads %% num_kv_heads != 0", name);
  const int group = num_q_heads / num_kv_heads;
  PKV_UNSUP(group <= kWMaxCols, "%s: num_q_heads / num_kv_heads must be at most %d (got %d)", name, kWMaxCols, group);
  PKV_UNSUP(block_size % 8 == 0, "%s: block_size must be a multiple of 8", name);
  PKV_UNSUP((int64_t)max_blocks * block_size <= INT32_MAX - 127, "%s: max_blocks * block_size must be at most 2^31 - 128", name);
  PKV_UNSUP((int64_t)num_reqs * T <= INT32_MAX / num_q_heads, "%s: too many query rows", name);
  PKV_UNSUP(((int64_t)max_blocks * block_size / kWTile + 1) * num_reqs <= INT32_MAX / 2, "%s: too many keys", name);
  PKV_ARG(rows_apart(num_reqs, w_stride_req, num_kv_heads, w_stride_head, max_ctx), "%s: rows of weights must not overlap", name);
  // (each key's earlier weight is read by the thread that writes the new one, at its own time)
  PKV_ARG(!prev || prev == weights ||
              !rows_meet(num_reqs, w_stride_req, num_kv_heads, w_stride_head, max_ctx,
                         ((int64_t)reinterpret_cast<uintptr_t>(prev) - (int64_t)reinterpret_cast<uintptr_t>(weights)) / 4),
          "%s: prev must be weights itself or share no element with it", name);
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
  const size_t lse = lse_bytes((int64_t)num_reqs * T * num_q_heads);
  PKV_ARG(aligned16(workspace) && workspace_bytes >= (int64_t)(lse + kStatBytes),
          "%s: workspace must be 16-byte aligned and hold %lld bytes at least (got %lld)", name, (long long)(lse + kStatBytes),
          (long long)workspace_bytes);

  WeightParams p{};
  int seg = kWTile;
  while (block_size % seg) seg >>= 1;  // gcd with 128: 8 at least
  p.seg = seg;
  p.big_ok = block_size >= kWTile;
  {
    const uint64_t head = (uint64_t)(stride_head * es), tok = (uint64_t)(stride_tok * es), blk = (uint64_t)(stride_blk * es);
    const uint64_t hkv = (uint64_t)num_kv_heads, bs = (uint64_t)block_size, nb = (uint64_t)num_blocks;
    const bool wide = kv_dtype == PKV_KV_BF16;
    const uint64_t dims4[4] = {(uint64_t)kWD, hkv, bs, nb}, strides4[3] = {head, tok, blk};
    const uint64_t dims5[5] = {128, bs, 2, hkv, nb}, strides5[4] = {tok, 128, head, blk};
    auto encode = [&](CUtensorMap* map, uint32_t rows) {
      const uint32_t box4[4] = {64, 1, rows, 1}, box5[5] = {128, rows, 2, 1, 1};
      return wide ? encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, k_cache, dims4, strides4, box4, "k_cache")
                  : encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, k_cache, dims5, strides5, box5, "k_cache");
    };
    pkv_status s = encode(&p.kmap, (uint32_t)seg);
    if (s == PKV_OK && p.big_ok) s = encode(&p.kmap_big, kWTile);
    if (s != PKV_OK) return s;
  }
  p.k_scale = k_scale;
  p.num_blocks = num_blocks;
  p.s_stride_blk = scale_stride_blk, p.s_stride_tok = scale_stride_tok;
  p.block_table = block_table, p.bt_stride = bt_stride, p.max_blocks = max_blocks;
  p.seq_lens = seq_lens, p.q_valid = q_valid;
  p.num_reqs = num_reqs, p.T = T, p.group = group, p.num_q_heads = num_q_heads, p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.part_lse = part_lse, p.split_tokens = split_tokens, p.max_splits = max_splits;
  p.prev = prev, p.prev_lens = prev_lens;
  p.weights = weights, p.w_stride_req = w_stride_req, p.w_stride_head = w_stride_head, p.max_ctx = max_ctx;
  p.lse2 = static_cast<float*>(workspace);
  p.stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + lse);
  p.dev_err = dev_err;
  p.wait_limit_ns = take_wait_limit_ns();
  const int64_t room = (workspace_bytes - (int64_t)lse) / (int64_t)kStatBytes;
  const int ctas = (int)(room < num_sms() ? room : num_sms());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // more query columns than one pass takes: tokens in passes, each on top of the one before
  const int most = kWMaxCols / group;
  for (int t = 0; t < T; t += most) {
    p.t_base = t;
    p.tpc = T - t < most ? T - t : most;
    const uint64_t dims[3] = {(uint64_t)kWD, (uint64_t)num_q_heads, (uint64_t)num_reqs * (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)kWD * 2, (uint64_t)num_q_heads * kWD * 2};
    const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)p.tpc};
    pkv_status s = encode_tiled(&p.qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box, "q");
    if (s != PKV_OK) return s;
    // a CTA a KV head and range of tiles; more heads than CTAs: in turns
    for (int h = 0; h < num_kv_heads; h += ctas) {
      p.h_base = h;
      p.heads = num_kv_heads - h < ctas ? num_kv_heads - h : ctas;
      const int grid = ctas / p.heads * p.heads;
      s = kv_dtype == PKV_KV_BF16 ? run_attn_weights_bf16(p, grid, st)
          : kv_dtype == PKV_KV_INT8 ? run_attn_weights_int8(p, grid, st) : run_attn_weights_fp8(p, grid, st);
      if (s != PKV_OK) return s;
    }
    p.prev = weights;
    p.prev_lens = nullptr;
  }
  return PKV_OK;
}
