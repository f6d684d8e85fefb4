// kv_evict_select.cu - pkv_kv_evict_select: the positions of a cache that stay.
//
// Of each (request, KV head) longer than the budget: the first `sinks`, the last `recent`, and of the positions in
// between the budget - sinks - recent with the highest scores, the lowest position first among equals; ascending.
//
// One cluster of CTAs a (request, KV head). Each CTA reads its slice of the scores once, as integers that order as the
// scores do, into shared memory (slices past its size are read again from L2). The score of the last one that stays is
// found digit by digit (11 + 11 + 10 bits): a histogram a CTA, summed over the cluster through distributed shared
// memory. Then each warp counts what stays in its stretch of the slice and writes it behind what stays before it.
#include <cooperative_groups.h>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kBins = 2048;
constexpr int kMaxCached = 49152;  // scores of a slice that shared memory holds (192 KB)

struct SelectParams {
  const float* scores;
  int64_t stride_req, stride_head;
  const int32_t* seq_lens;
  int32_t num_kv_heads, sinks, recent, budget;
  int64_t max_ctx;
  int32_t* keep;
  int32_t* new_lens;
  int cached;  // scores that shared memory holds
  int* dev_err;
};

// Integers that order as the scores do; NaN below everything, the two zeros alike.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Shared {
  uint32_t hist[3][kBins];
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t gt, eq;       // of this CTA's slice
  uint32_t scan[kWarps];
  int digit;
  uint32_t above;
};

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int unit = blockIdx.x / kCluster;
  const int r = unit / p.num_kv_heads, h = unit - r * p.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = __ldg(p.seq_lens + r);
  const int n = (int)max((int64_t)0, min((int64_t)len, p.max_ctx));
  int32_t* keep = p.keep + (int64_t)unit * p.budget;
  if (rank == 0 && tid == 0) {
    if (len < 0 || len > p.max_ctx) record_error(p.dev_err, kErrDeviceBounds);
    if (h == 0) p.new_lens[r] = min(n, p.budget);
  }
  if (n <= p.budget) {  // uniform over the cluster
    for (int i = rank * kThreads + tid; i < n; i += kCluster * kThreads) keep[i] = i;
    return;
  }
  const float* sc = p.scores + (int64_t)r * p.stride_req + (int64_t)h * p.stride_head;
  const int first = p.sinks, last = n - p.recent;  // what is chosen from: [first, last)
  const uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent);

  // slices: a multiple of 32 positions each
  const int slice = ((n + kCluster - 1) / kCluster + 31) & ~31;
  const int lo = min(rank * slice, n), hi = min(lo + slice, n);
  const int held = min(hi - lo, p.cached);
  auto key_at = [&](int i) { return i - lo < held ? s_key[i - lo] : ordered(__ldg(sc + i)); };

  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  for (int i = lo + tid; i < hi; i += kThreads) {
    const uint32_t k = ordered(__ldg(sc + i));
    if (i - lo < held) s_key[i - lo] = k;
    if (i >= first && i < last) atomicAdd(&sh.hist[0][k >> 21], 1u);
  }

  uint32_t prefix = 0, rest = want;  // the digits found, and how many are still wanted among the scores that have them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    if (pass) {
      const int shift = pass == 1 ? 21 : 10;
      for (int i = max(lo, first) + tid; i < min(hi, last); i += kThreads) {
        const uint32_t k = key_at(i);
        if (k >> shift == prefix) atomicAdd(&sh.hist[pass][pass == 1 ? (k >> 10) & 2047u : k & 1023u], 1u);
      }
    }
    cluster.sync();
    // bins from the highest down: thread t has bins 2047 - 4t .. 2044 - 4t
    uint32_t c[4] = {0, 0, 0, 0};
    for (int k = 0; k < kCluster; ++k) {
      const uint4 x = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&sh.hist[pass][kBins - 4 - 4 * tid], k));
      c[0] += x.w, c[1] += x.z, c[2] += x.y, c[3] += x.x;
    }
    const uint32_t own = c[0] + c[1] + c[2] + c[3];
    uint32_t run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) sh.scan[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += sh.scan[w];
    uint32_t above = run - own;  // scores in higher bins than this thread's
    if (above < rest && run >= rest) {
      int d = kBins - 1 - 4 * tid;
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (above + c[e] < rest && d == kBins - 1 - 4 * tid - e) {
          above += c[e];
          --d;
        }
      sh.digit = d;
      sh.above = above;
    }
    __syncthreads();
    if (rest) {
      prefix = pass == 0 ? (uint32_t)sh.digit : pass == 1 ? (prefix << 11) | (uint32_t)sh.digit : (prefix << 10) | (uint32_t)sh.digit;
      rest -= sh.above;
    }
  }
  // prefix: the last score that stays, `rest` of its equals stay (none is wanted: nothing is above)
  const uint32_t limit = want ? prefix : 0xffffffffu;

  // a warp's stretch of the slice
  const int stretch = ((hi - lo + kWarps - 1) / kWarps + 31) & ~31;
  const int w_lo = min(lo + warp * stretch, hi), w_hi = min(w_lo + stretch, hi);
  uint32_t gt = 0, eq = 0;
  for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
    const int i = i0 + lane;
    bool is_gt = false, is_eq = false;
    if (i < w_hi) {
      const bool fixed = i < first || i >= last;
      const uint32_t k = fixed ? 0 : key_at(i);
      is_gt = fixed || k > limit;
      is_eq = !fixed && k == limit;
    }
    gt += __popc(__ballot_sync(0xffffffffu, is_gt));
    eq += __popc(__ballot_sync(0xffffffffu, is_eq));
  }
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, b = 0;
    for (int w = 0; w < kWarps; ++w) a += sh.warp_gt[w], b += sh.warp_eq[w];
    sh.gt = a;
    sh.eq = b;
  }
  cluster.sync();
  uint32_t gt_before = 0, eq_before = 0;
  for (int k = 0; k < rank; ++k) {
    gt_before += *cluster.map_shared_rank(&sh.gt, k);
    eq_before += *cluster.map_shared_rank(&sh.eq, k);
  }
  for (int w = 0; w < warp; ++w) gt_before += sh.warp_gt[w], eq_before += sh.warp_eq[w];
  for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
    const int i = i0 + lane;
    bool is_gt = false, is_eq = false;
    if (i < w_hi) {
      const bool fixed = i < first || i >= last;
      const uint32_t k = fixed ? 0 : key_at(i);
      is_gt = fixed || k > limit;
      is_eq = !fixed && k == limit;
    }
    const uint32_t m_gt = __ballot_sync(0xffffffffu, is_gt), m_eq = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t e = eq_before + __popc(m_eq & below);
    if (is_gt || (is_eq && e < rest)) keep[gt_before + __popc(m_gt & below) + min(e, rest)] = i;
    gt_before += __popc(m_gt);
    eq_before += __popc(m_eq);
  }
  cluster.sync();  // shared memory that other CTAs read stays until they have
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_evict_select(const float* scores, int64_t stride_req, int64_t stride_head, int64_t max_ctx,
                                          const int32_t* seq_lens, int32_t num_reqs, int32_t num_kv_heads, int32_t sinks,
                                          int32_t recent, int32_t budget, int32_t* keep, int32_t* new_lens,
                                          int32_t* dev_err, void* stream) {
  using namespace pkv;
  clear_error();
  const char* name = "kv_evict_select";
  PKV_ARG(num_reqs >= 0 && num_kv_heads > 0 && max_ctx > 0 && budget > 0 && sinks >= 0 && recent >= 0,
          "%s: bad size argument", name);
  PKV_ARG((int64_t)sinks + recent <= budget, "%s: sinks + recent must be at most budget", name);
  PKV_UNSUP(max_ctx <= INT32_MAX - 4096, "%s: max_ctx too large", name);
  PKV_UNSUP((int64_t)num_reqs * num_kv_heads <= INT32_MAX / kCluster, "%s: too many requests", name);
  PKV_ARG(stride_req >= 0 && stride_head >= 0, "%s: strides must not be negative", name);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(scores && seq_lens && keep && new_lens, "%s: null pointer argument", name);
  PKV_ARG((reinterpret_cast<uintptr_t>(scores) & 3) == 0, "%s: scores must be 4-byte aligned", name);
  SelectParams p{scores, stride_req, stride_head, seq_lens, num_kv_heads, sinks, recent, budget, max_ctx, keep, new_lens, 0, dev_err};
  const int64_t slice = ((max_ctx + kCluster - 1) / kCluster + 31) & ~(int64_t)31;
  p.cached = (int)(slice < kMaxCached ? slice : kMaxCached);
  const size_t smem = (size_t)p.cached * 4;
  static std::atomic<uint64_t> attr_done{0};
  once_per_device(attr_done, [] {
    cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_reqs * num_kv_heads * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, select_kernel, p);
  return check_launch(name);
}
