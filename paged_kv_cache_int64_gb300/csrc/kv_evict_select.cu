// kv_evict_select.cu - pkv_kv_evict_select: the positions of a cache that stay.
//
// Of each (request, KV head) longer than the budget: the first `sinks`, the last `recent`, and of the positions in
// between the budget - sinks - recent with the highest scores, the lowest position first among equals; ascending.
//
// A (request, KV head) is one CTA's, or a cluster's, a slice of the positions each. The scores are read once, as integers
// that order as they do, into shared memory (slices past its size are read again from L2). The last one that stays is
// found by histograms of 2,048 bins over the range that the scores take (not over their leading bits: those are the same
// few exponents for most scores, and the additions to one bin would wait for one another), until the bin that holds it
// has few enough scores to rank them against each other. Then each warp counts what stays in its stretch of the slice and
// writes it behind what stays before it.
#include <cooperative_groups.h>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
static_assert(kBins == 4 * kThreads && kWarps <= 32, "bins and warps a thread");
constexpr int kListMax = kThreads;     // scores that are ranked against each other
constexpr int kMaxCluster = 8;
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

struct alignas(16) Shared {
  uint32_t hist[3][kBins];
  uint2 list[kListMax];  // (key, position) of this slice's scores in the last bin
  uint2 all[kListMax];   // of every slice's
  uint32_t list_n;
  uint32_t lo[kWarps], hi[kWarps];  // the warps' smallest and largest keys; then of the slice in [0]
  uint32_t slice_lo, slice_hi;
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t gt, eq;  // of this slice
  uint32_t scan[kWarps];
  uint32_t digit, above, in_bin;
  uint32_t limit, equal;
};

template <int kCluster>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCluster > 1 ? (int)cluster.block_rank() : 0;
  auto sync = [&]() {
    if (kCluster > 1) cluster.sync(); else __syncthreads();
  };
  auto at_rank = [&](auto* x, int k) { return kCluster > 1 ? cluster.map_shared_rank(x, k) : x; };
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
  const int first = p.sinks, last = n - p.recent;  // what is chosen from: [first, last), more than `want`
  const uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent);

  // slices: a multiple of 32 positions each
  const int slice = ((n + kCluster - 1) / kCluster + 31) & ~31;
  const int lo = min(rank * slice, n), hi = min(lo + slice, n);
  const int held = min(hi - lo, p.cached);
  const int c_lo = max(lo, first), c_hi = min(hi, last);  // the slice's part of what is chosen from
  auto key_at = [&](int i) { return i - lo < held ? s_key[i - lo] : ordered(__ldg(sc + i)); };

  // a warp's stretch of the slice
  const int stretch = ((hi - lo + kWarps - 1) / kWarps + 31) & ~31;
  const int w_lo = min(lo + warp * stretch, hi), w_hi = min(w_lo + stretch, hi);
  const int w_held = min(w_hi, lo + held);  // up to here in shared memory
  // f(position, key) for every position of the warp's stretch that is chosen from, four at a time from shared memory
  auto each_key = [&](auto&& f) {
    const int a = max(w_lo, c_lo), b = min(w_held, c_hi);
    for (int i = w_lo + 4 * lane; i < b; i += 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(s_key + (i - lo));
      if (i >= a && i + 4 <= b) {
        f(i, x.x), f(i + 1, x.y), f(i + 2, x.z), f(i + 3, x.w);
      } else {
        if (i >= a) f(i, x.x);
        if (i + 1 >= a && i + 1 < b) f(i + 1, x.y);
        if (i + 2 >= a && i + 2 < b) f(i + 2, x.z);
        if (i + 3 >= a && i + 3 < b) f(i + 3, x.w);
      }
    }
    for (int i = max(a, w_held) + lane; i < min(w_hi, c_hi); i += 32) f(i, ordered(__ldg(sc + i)));
  };

  for (int i = tid; i < 3 * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.list_n = 0;
  if (tid < kWarps) sh.warp_gt[tid] = sh.warp_eq[tid] = 0;
  // each warp's stretch into shared memory, all of it on its way at once
  if ((reinterpret_cast<uintptr_t>(sc) & 15) == 0) {
    for (int i = w_lo + 4 * lane; i < w_held; i += 128) {
      const uint32_t to = smem_u32(s_key + (i - lo));
      if (i + 4 <= n) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(sc + i) : "memory");
      } else {
        for (int e = 0; i + e < n; ++e) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * e), "l"(sc + i + e) : "memory");
      }
    }
  } else {
    for (int i = w_lo + lane; i < w_held; i += 32)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(s_key + (i - lo))), "l"(sc + i) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  for (int i = w_lo + 4 * lane; i < w_held; i += 128) {  // (a last vector may pass the stretch: the slice's room is a multiple)
    uint4* at = reinterpret_cast<uint4*>(s_key + (i - lo));
    const uint4 x = *at;
    *at = make_uint4(ordered(__uint_as_float(x.x)), ordered(__uint_as_float(x.y)), ordered(__uint_as_float(x.z)), ordered(__uint_as_float(x.w)));
  }
  __syncwarp();
  uint32_t mn = 0xffffffffu, mx = 0;
  each_key([&](int, uint32_t k) { mn = min(mn, k), mx = max(mx, k); });
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) sh.lo[warp] = mn, sh.hi[warp] = mx;
  __syncthreads();
  if (kCluster > 1) {
    if (warp == 0) {
      mn = __reduce_min_sync(0xffffffffu, sh.lo[lane & (kWarps - 1)]);
      mx = __reduce_max_sync(0xffffffffu, sh.hi[lane & (kWarps - 1)]);
      if (lane == 0) sh.slice_lo = mn, sh.slice_hi = mx;
    }
    sync();
    mn = lane < kCluster ? *at_rank(&sh.slice_lo, lane < kCluster ? lane : 0) : 0xffffffffu;
    mx = lane < kCluster ? *at_rank(&sh.slice_hi, lane < kCluster ? lane : 0) : 0u;
  } else {
    mn = sh.lo[lane & (kWarps - 1)];
    mx = sh.hi[lane & (kWarps - 1)];
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);

  // [base, base + (2048 << shift)): the keys that are still looked among, `rest` of them wanted
  uint32_t base = mn, rest = want, limit = 0xffffffffu;
  uint32_t n_gt = 0, n_eq = 0;  // this lane's, of the warp's stretch
  bool counted = false;
  int shift = max(0, 21 - __clz(mx - mn));
  if (want)
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      uint32_t* hist = sh.hist[pass];
      each_key([&](int, uint32_t k) {
        const uint32_t d = (k - base) >> shift;
        if (d < kBins) atomicAdd(&hist[d], 1u);
      });
      sync();
      // bins from the highest down: thread t has 2047 - 4t .. 2044 - 4t
      uint32_t c[4] = {0, 0, 0, 0};
      for (int k = 0; k < kCluster; ++k) {
        const uint4 x = *reinterpret_cast<const uint4*>(at_rank(&hist[kBins - 4 - 4 * tid], k));
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
      run += __reduce_add_sync(0xffffffffu, lane < warp ? sh.scan[lane] : 0u);
      uint32_t above = run - own;  // scores in higher bins than this thread's
      if (above < rest && run >= rest) {
        int e = 0;
        while (e < 3 && above + c[e] < rest) above += c[e], ++e;
        sh.digit = kBins - 1 - 4 * tid - e;
        sh.above = above;
        sh.in_bin = e == 0 ? c[0] : e == 1 ? c[1] : e == 2 ? c[2] : c[3];
      }
      __syncthreads();
      rest -= sh.above;
      base += sh.digit << shift;
      if (shift == 0) {  // one key: `rest` of those that have it
        limit = base;
        break;
      }
      if (sh.in_bin <= kListMax) {
        // few enough: ranked against each other, everywhere alike
        const uint32_t top = base + ((1u << shift) - 1u);
        each_key([&](int i, uint32_t k) {
          n_gt += k > top;
          if (k >= base && k <= top) sh.list[atomicAdd(&sh.list_n, 1u)] = make_uint2(k, (uint32_t)i);
        });
        counted = true;
        sync();
        uint32_t m = 0;
        for (int k = 0; k < kCluster; ++k) {
          const uint32_t cnt = *at_rank(&sh.list_n, k);
          const uint2* from = at_rank(sh.list, k);
          if ((uint32_t)tid < cnt) sh.all[m + tid] = from[tid];
          m += cnt;
        }
        __syncthreads();
        if ((uint32_t)tid < m) {
          const uint2 x = sh.all[tid];
          uint32_t ahead = 0, same = 0;
          for (uint32_t j = 0; j < m; ++j) {
            const uint2 y = sh.all[j];
            ahead += y.x > x.x;
            same += y.x == x.x && y.y < x.y;
          }
          if (ahead + same == rest - 1) {  // the last one that stays
            sh.limit = x.x;
            sh.equal = same + 1;
          }
        }
        __syncthreads();
        limit = sh.limit;
        rest = sh.equal;
        if ((uint32_t)tid < sh.list_n) {  // what of the slice's own list stays, to its warp's count
          const uint2 x = sh.list[tid];
          if (x.x > limit) atomicAdd(&sh.warp_gt[((int)x.y - lo) / stretch], 1u);
          if (x.x == limit) atomicAdd(&sh.warp_eq[((int)x.y - lo) / stretch], 1u);
        }
        break;
      }
      shift = max(0, shift - 11);
    }

  // what is above `limit` stays, and the first `rest` of its equals
  auto kind = [&](int i, bool& gt, bool& eq) {
    gt = eq = false;
    if (i < hi) {
      const bool fixed = i < first || i >= last;
      const uint32_t k = fixed ? 0u : key_at(i);
      gt = fixed || k > limit;
      eq = !fixed && k == limit;
    }
  };
  if (!counted) each_key([&](int, uint32_t k) { n_gt += k > limit, n_eq += k == limit; });
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) {
    // the fixed positions of the stretch: before `first`, from `last` on
    const int fixed = max(0, min(w_hi, first) - w_lo) + max(0, w_hi - max(w_lo, last));
    atomicAdd(&sh.warp_gt[warp], n_gt + (uint32_t)fixed);
    atomicAdd(&sh.warp_eq[warp], n_eq);
  }
  __syncthreads();
  uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_gt[lane] : 0u);
  uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_eq[lane] : 0u);
  if (kCluster > 1) {
    if (tid == kThreads - 1) sh.gt = gt_before + sh.warp_gt[warp], sh.eq = eq_before + sh.warp_eq[warp];  // (the last warp's: the slice's)
    sync();
    const bool mine = lane < rank;
    gt_before += __reduce_add_sync(0xffffffffu, mine ? *at_rank(&sh.gt, mine ? lane : 0) : 0u);
    eq_before += __reduce_add_sync(0xffffffffu, mine ? *at_rank(&sh.eq, mine ? lane : 0) : 0u);
  }
  const uint32_t below = (1u << lane) - 1u;
  if (sh.warp_eq[warp] == 0 && w_lo >= c_lo && w_hi <= c_hi && w_hi - lo <= held) {
    int32_t* to = keep + gt_before + min(eq_before, rest);
#pragma unroll 4
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const bool gt = i0 + lane < w_hi && s_key[i0 - lo + lane] > limit;
      const uint32_t m = __ballot_sync(0xffffffffu, gt);
      if (gt) to[__popc(m & below)] = i0 + lane;
      to += __popc(m);
    }
  } else {
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      bool gt, eq;
      kind(i0 + lane, gt, eq);
      const uint32_t m_gt = __ballot_sync(0xffffffffu, gt), m_eq = __ballot_sync(0xffffffffu, eq);
      const uint32_t e = eq_before + __popc(m_eq & below);
      if (gt || (eq && e < rest)) keep[gt_before + __popc(m_gt & below) + min(e, rest)] = i0 + lane;
      gt_before += __popc(m_gt);
      eq_before += __popc(m_eq);
    }
  }
  if (kCluster > 1) sync();  // shared memory that other CTAs read stays until they have
}

template <int kCluster>
pkv_status launch(SelectParams p, int units, cudaStream_t stream) {
  const int64_t slice = ((p.max_ctx + kCluster - 1) / kCluster + 31) & ~(int64_t)31;
  p.cached = (int)(slice < kMaxCached ? slice : kMaxCached);
  static std::atomic<uint64_t> attr_done{0};
  once_per_device(attr_done, [] {
    cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.cached * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, select_kernel<kCluster>, p);
  return check_launch("kv_evict_select");
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
  PKV_UNSUP((int64_t)num_reqs * num_kv_heads <= INT32_MAX / kMaxCluster, "%s: too many requests", name);
  PKV_ARG(stride_req >= 0 && stride_head >= 0, "%s: strides must not be negative", name);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(scores && seq_lens && keep && new_lens, "%s: null pointer argument", name);
  PKV_ARG((reinterpret_cast<uintptr_t>(scores) & 3) == 0, "%s: scores must be 4-byte aligned", name);
  SelectParams p{scores, stride_req, stride_head, seq_lens, num_kv_heads, sinks, recent, budget, max_ctx, keep, new_lens, 0, dev_err};
  const int units = num_reqs * num_kv_heads;
  // Slices: as many CTAs a unit as the device holds of them at once (two an SM), of 4,096 positions at least.
  int ctas = 1;
  while (ctas < kMaxCluster && (int64_t)units * ctas * 2 <= 2 * num_sms() && max_ctx > (int64_t)ctas * 4096) ctas *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (ctas) {
    case 1: return launch<1>(p, units, st);
    case 2: return launch<2>(p, units, st);
    case 4: return launch<4>(p, units, st);
    default: return launch<8>(p, units, st);
  }
}
