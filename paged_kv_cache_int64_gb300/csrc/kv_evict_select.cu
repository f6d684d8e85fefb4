// kv_evict_select.cu - pkv_kv_evict_select: the positions of a cache that stay.
//
// Of each (request, KV head) longer than the budget: the first `sinks`, the last `recent`, and of the positions in
// between the budget - sinks - recent with the highest scores, the lowest position first among equals; ascending.
//
// A (request, KV head) is one CTA's, or a cluster's, a slice of the positions each. The scores are read once, as integers
// that order as they do, into shared memory (slices past its size are read again from L2). The last one that stays is
// found by histograms of 2,048 bins over the range that the scores take (not over their leading bits: those are the same
// few exponents for most scores, and the additions to one bin would wait for one another), at first of the 16 octaves below
// the largest, which is where it lies as a rule. Once the bin that holds it has few enough scores, they are listed and the
// last one is found among them. Then each warp counts what stays in its stretch of the slice and writes it behind what
// stays before it.
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
constexpr int kListMax = 2 * kThreads;  // scores that are listed
constexpr int kRankMax = 256;           // of these: ranked against each other
constexpr int kMaxCluster = 16;
constexpr int kMaxCached = 47104;  // scores of a slice that shared memory holds (184 KB)

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

// Integers that order as the scores do, 0xff800000 (infinity) at most; NaN below everything, the two zeros alike.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr uint32_t kFixed = 0xffffffffu;  // the key of a position that stays whatever its score

template <int kCluster>
struct alignas(16) Shared {
  uint32_t hist[3][kBins];
  alignas(16) uint32_t sums[kCluster >= 4 ? kBins : 4];  // of every slice's histogram
  uint32_t list[kListMax];     // this slice's keys in the last bin
  uint8_t list_warp[kListMax];  // the warps whose stretches have them
  uint32_t list_n;
  uint32_t lo[kWarps], hi[kWarps];  // the warps' smallest and largest keys
  uint32_t slice_lo, slice_hi;
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t gt, eq;  // of this slice
  uint32_t scan[kWarps];
  uint32_t digit, above, in_bin, total;
};

template <int kCluster>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ Shared<kCluster> sh;
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
    uint4 y = make_uint4(ordered(__uint_as_float(x.x)), ordered(__uint_as_float(x.y)), ordered(__uint_as_float(x.z)), ordered(__uint_as_float(x.w)));
    if (i < first || i + 4 > last) {
      if (i < first || i >= last) y.x = kFixed;
      if (i + 1 < first || i + 1 >= last) y.y = kFixed;
      if (i + 2 < first || i + 2 >= last) y.z = kFixed;
      if (i + 3 < first || i + 3 >= last) y.w = kFixed;
    }
    *at = y;
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

  // [base, base + width): the keys that are still looked among, `rest` of them wanted, in bins of 2^shift
  constexpr uint32_t kOctaves = 16u << 23;
  uint32_t base = mx - mn > kOctaves ? mx - kOctaves : mn, width = mx - base + 1, rest = want, limit = kFixed - 1;
  auto bins_of = [&](uint32_t w) { return max(0, 21 - __clz(w - 1)); };  // (w = 1: 21 - 32)
  int shift = bins_of(width);
  uint32_t n_gt = 0, n_eq = 0;  // this lane's, of the warp's stretch
  bool counted = false;
  if (want)
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      uint32_t* hist = sh.hist[pass % 3];
      if (pass == 2)  // (read by everyone before the last barrier; a fourth pass, of the lower range, uses it again)
        for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
      each_key([&](int, uint32_t k) {
        const uint32_t d = k - base;
        if (d < width) atomicAdd(&hist[d >> shift], 1u);
      });
      sync();
      // bins from the highest down: thread t has 2047 - 4t .. 2044 - 4t
      uint32_t c[4] = {0, 0, 0, 0};
      if constexpr (kCluster >= 4) {
        // each CTA adds up its part of the bins over the cluster and gives the sums to every CTA (every CTA reading every
        // histogram whole takes 9 us of 27 for one context of 262,144)
        constexpr int kPart = kBins / kCluster;
        if (tid < kPart / 4) {
          const int at = rank * kPart + 4 * tid;
          uint4 x[kCluster];
#pragma unroll
          for (int k = 0; k < kCluster; ++k) x[k] = *reinterpret_cast<const uint4*>(at_rank(&hist[at], k));
          uint4 t = x[0];
#pragma unroll
          for (int k = 1; k < kCluster; ++k) t.x += x[k].x, t.y += x[k].y, t.z += x[k].z, t.w += x[k].w;
#pragma unroll
          for (int k = 0; k < kCluster; ++k) *reinterpret_cast<uint4*>(at_rank(&sh.sums[at], k)) = t;
        }
        sync();
        const uint4 x = *reinterpret_cast<const uint4*>(&sh.sums[kBins - 4 - 4 * tid]);
        c[0] = x.w, c[1] = x.z, c[2] = x.y, c[3] = x.x;
      } else {
#pragma unroll
        for (int k = 0; k < kCluster; ++k) {
          const uint4 x = *reinterpret_cast<const uint4*>(at_rank(&hist[kBins - 4 - 4 * tid], k));
          c[0] += x.w, c[1] += x.z, c[2] += x.y, c[3] += x.x;
        }
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
      if (tid == kThreads - 1) sh.total = run;
      if (above < rest && run >= rest) {
        int e = 0;
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (e == t && above + c[t] < rest) above += c[t], ++e;
        sh.digit = kBins - 1 - 4 * tid - e;
        sh.above = above;
        sh.in_bin = e == 0 ? c[0] : e == 1 ? c[1] : e == 2 ? c[2] : c[3];
      }
      __syncthreads();
      if (sh.total < rest) {  // it lies below the 16 octaves
        rest -= sh.total;
        width = base - mn;
        base = mn;
        shift = bins_of(width);
        continue;
      }
      rest -= sh.above;
      base += sh.digit << shift;
      width = min(width - (sh.digit << shift), 1u << shift);
      if (shift == 0) {  // one key: `rest` of those that have it
        limit = base;
        break;
      }
      const uint32_t in_bin = sh.in_bin;
      if (in_bin <= kListMax) {
        const uint32_t top = base + (width - 1);
        each_key([&](int, uint32_t k) {
          n_gt += k > top;
          if (k >= base && k <= top) {
            const uint32_t at = atomicAdd(&sh.list_n, 1u);
            sh.list[at] = k;
            sh.list_warp[at] = (uint8_t)warp;
          }
        });
        counted = true;
        sync();
        // every slice's, to every CTA: in the histogram that is read by nobody any more
        uint32_t* all = sh.hist[(pass + 2) % 3];
        const uint32_t m = in_bin;
        if (kCluster == 1) {
          all = sh.list;
        } else {  // a warp a slice
          const uint32_t cnt = lane < kCluster ? *at_rank(&sh.list_n, lane < kCluster ? lane : 0) : 0u;
          for (int k = warp; k < kCluster; k += kWarps) {
            const uint32_t n_k = __shfl_sync(0xffffffffu, cnt, k), from_k = __reduce_add_sync(0xffffffffu, lane < k ? cnt : 0u);
            const uint32_t* from = at_rank(sh.list, k);
            for (uint32_t j = lane; j < n_k; j += 32) all[from_k + j] = from[j];
          }
          __syncthreads();
        }
        if (m <= kRankMax) {  // few: each against all others
          if ((uint32_t)tid < m) {
            const uint32_t x = all[tid];
            uint32_t n_above = 0, same = 0;
            for (uint32_t j = 0; j < m; ++j) n_above += all[j] > x, same += all[j] == x;
            if (n_above < rest && n_above + same >= rest) {  // (its equals write the same)
              sh.digit = x;
              sh.above = n_above;
            }
          }
          __syncthreads();
          limit = sh.digit;
          rest -= sh.above;
        } else {  // the largest key that `rest` of them reach, bit by bit
          const uint32_t k0 = (uint32_t)tid < m ? all[tid] : 0u, k1 = (uint32_t)tid + kThreads < m ? all[tid + kThreads] : 0u;
          limit = base;
          for (int bit = shift - 1; bit >= 0; --bit) {
            const uint32_t x = limit + (1u << bit);
            int n_at = __syncthreads_count(k0 >= x);
            if (m > kThreads) n_at += __syncthreads_count(k1 >= x);
            if ((uint32_t)n_at >= rest) limit = x;
          }
          int n_above = __syncthreads_count(k0 > limit);
          if (m > kThreads) n_above += __syncthreads_count(k1 > limit);
          rest -= (uint32_t)n_above;
        }
        for (uint32_t j = tid; j < sh.list_n; j += kThreads) {  // what of the slice's own list stays, to its warp's count
          const uint32_t x = sh.list[j], w = sh.list_warp[j];
          if (x > limit) atomicAdd(&sh.warp_gt[w], 1u);
          if (x == limit) atomicAdd(&sh.warp_eq[w], 1u);
        }
        break;
      }
      shift = max(0, shift - 11);
    }

  // what is above `limit` stays, and the first `rest` of its equals
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
  const uint32_t eq_here = sh.warp_eq[warp];
  const bool all_eq = eq_before + eq_here <= rest, no_eq = eq_here == 0 || eq_before >= rest;
  if (w_held == w_hi && (all_eq || no_eq)) {
    const uint32_t least = no_eq ? limit + 1 : limit;
    int32_t* to = keep + gt_before + min(eq_before, rest);
#pragma unroll 4
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const bool stays = i0 + lane < w_hi && s_key[i0 - lo + lane] >= least;
      const uint32_t m = __ballot_sync(0xffffffffu, stays);
      if (stays) to[__popc(m & below)] = i0 + lane;
      to += __popc(m);
    }
  } else {
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const int i = i0 + lane;
      uint32_t k = 0;
      if (i < w_hi) k = i < w_held ? s_key[i - lo] : i < first || i >= last ? kFixed : ordered(__ldg(sc + i));
      const bool gt = i < w_hi && k > limit, eq = i < w_hi && k == limit;
      const uint32_t m_gt = __ballot_sync(0xffffffffu, gt), m_eq = __ballot_sync(0xffffffffu, eq);
      const uint32_t e = eq_before + __popc(m_eq & below);
      if (gt || (eq && e < rest)) keep[gt_before + __popc(m_gt & below) + min(e, rest)] = i;
      gt_before += __popc(m_gt);
      eq_before += __popc(m_eq);
    }
  }
  if (kCluster > 1) sync();  // shared memory that other CTAs read stays until they have
}

static_assert(kMaxCached * 4 + sizeof(Shared<kMaxCluster>) + 1024 <= 227 * 1024, "shared memory of one CTA");

template <int kCluster>
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int units, size_t smem, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  once_per_device(attr_done, [] {
    cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (kCluster > 8) cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  cfg = {};
  cfg.gridDim = dim3((unsigned)units * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

// Whether the device holds a cluster of 16 CTAs with all of their shared memory (above the portable 8).
bool sixteen_fit() {
  static std::atomic<uint64_t> known{0}, fits{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (!(known.load() & bit)) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    configure<16>(cfg, attr, 1, (size_t)kMaxCached * 4, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, select_kernel<16>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    if (n > 0) fits.fetch_or(bit);
    known.fetch_or(bit);
    if (!bit) return n > 0;
  }
  return (fits.load() & bit) != 0;
}

template <int kCluster>
pkv_status launch(SelectParams p, int units, cudaStream_t stream) {
  const int64_t slice = ((p.max_ctx + kCluster - 1) / kCluster + 31) & ~(int64_t)31;
  p.cached = (int)(slice < kMaxCached ? slice : kMaxCached);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  configure<kCluster>(cfg, attr, units, (size_t)p.cached * 4, stream);
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
  // every CTA of a request reads its length, at its own time: nothing may be written there (lengths updated in place would
  // make the later ones take the cache for one within the budget)
  const uint64_t lens_bytes = (uint64_t)num_reqs * 4, keep_bytes = (uint64_t)num_reqs * num_kv_heads * (uint64_t)budget * 4;
  PKV_ARG(!overlaps(seq_lens, lens_bytes, new_lens, lens_bytes) && !overlaps(seq_lens, lens_bytes, keep, keep_bytes) &&
              !overlaps(new_lens, lens_bytes, keep, keep_bytes),
          "%s: seq_lens, keep and new_lens must not overlap", name);
  SelectParams p{scores, stride_req, stride_head, seq_lens, num_kv_heads, sinks, recent, budget, max_ctx, keep, new_lens, 0, dev_err};
  const int units = num_reqs * num_kv_heads;
  // Slices: as many CTAs a unit as the device holds of them at once (two an SM), of 4,096 positions at least; more where
  // shared memory would not hold the slices.
  const int most = max_ctx > 8 * 4096 && sixteen_fit() ? kMaxCluster : 8;
  int ctas = 1;
  while (ctas < most && (max_ctx > (int64_t)ctas * kMaxCached ||
                         ((int64_t)units * ctas * 2 <= 2 * num_sms() && max_ctx > (int64_t)ctas * 4096)))
    ctas *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (ctas) {
    case 1: return launch<1>(p, units, st);
    case 2: return launch<2>(p, units, st);
    case 4: return launch<4>(p, units, st);
    case 8: return launch<8>(p, units, st);
    default: return launch<16>(p, units, st);
  }
}
