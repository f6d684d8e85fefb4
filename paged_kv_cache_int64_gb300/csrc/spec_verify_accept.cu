// spec_verify_accept.cu - pkv_spec_verify_accept: which drafted tokens stay, and the token after them.
//
// Draft t of a request stays when u_t q_t(x_t) < p_t(x_t) and every draft before it stayed (the product in fp64,
// where it is exact). At the first that does not, the next token is drawn from max(p_t - q_t, 0); after the last
// draft, from p itself: the smallest i whose running sum passes u times the total.
//
// The sums are integers: each probability as a multiple of 2^-58 (exact from 2^-34 up), so they do not depend on
// the order in which they are added, and the token is the one that exact arithmetic gives.
//
// One cluster of CTAs a request, one pass over one row of p (and one of q). Each warp sums a contiguous segment of
// the row; the segment sums meet in the first CTA's shared memory; its first warps find the segment that holds the
// target and read that one again (it is in L2) to find the token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <utility>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct AcceptParams {
  const void* target;
  const void* draft;  // null: a draft's own probability is one
  int64_t t_stride_req, t_stride_tok, d_stride_req, d_stride_tok;
  const int32_t* ids;
  const float* u_accept;
  const float* u_sample;
  const int32_t* num_drafts;
  int32_t T, vocab;
  int32_t* out_tokens;
  int32_t* num_out;
  int* dev_err;
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// A probability as a multiple of 2^-58: values outside [0, 1] are clamped, NaN counts as 0.
__device__ __forceinline__ uint64_t fixed58(float p) {
  p = fminf(fmaxf(p, 0.0f), 1.0f);  // fmaxf(NaN, 0) = 0
  return __float2ull_rn(p * 0x1p58f);
}

// 16 bytes of a row as values.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / (int)sizeof(T);
  T v[kN];
};

// kN values of row `row` from index i on (i a multiple of kN); 0 past the vocabulary.
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int i, int vocab, bool wide) {
  constexpr int kN = Vec<T>::kN;
  Vec<T> o;
  if (wide && i + kN <= vocab) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + i));
    memcpy(&o, &x, 16);
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e) o.v[e] = i + e < vocab ? row[i + e] : T(0.0f);
  }
  return o;
}

// What the token is drawn from: p, max(p - q, 0), or p without the draft's own token.
template <typename T>
struct Source {
  const T* p;
  const T* q;   // null: none
  int skip;     // index left out, or -1
  int vocab;
  bool wide;    // both rows 16-byte aligned

  static constexpr int kN = Vec<T>::kN;
  __device__ __forceinline__ void load(int i, Vec<T>& a, Vec<T>& b) const {
    a = load_vec(p, i, vocab, wide);
    if (q) b = load_vec(q, i, vocab, wide);
  }
  __device__ __forceinline__ uint64_t weight(int i, int e, const Vec<T>& a, const Vec<T>& b) const {
    const uint64_t x = fixed58(as_float(a.v[e]));
    if (q) {
      const uint64_t y = fixed58(as_float(b.v[e]));
      return x > y ? x - y : 0;
    }
    return i + e == skip ? 0 : x;
  }
  __device__ __forceinline__ uint64_t sum(int i, const Vec<T>& a, const Vec<T>& b) const {
    uint64_t s = 0;
#pragma unroll
    for (int e = 0; e < kN; ++e) s += weight(i, e, a, b);
    return s;
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

constexpr int kBatch = 4;  // loads in flight a lane and table

// The warp's sum over [lo, hi), both multiples of a warp's load.
template <typename T>
__device__ uint64_t segment_sum(const Source<T>& s, int lo, int hi, int lane) {
  constexpr int kStep = 32 * Vec<T>::kN;
  uint64_t acc = 0;
  for (int i0 = lo; i0 < hi; i0 += kBatch * kStep) {
    Vec<T> a[kBatch], b[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) s.load(i0 + k * kStep < hi ? i0 + k * kStep + lane * Vec<T>::kN : s.vocab, a[k], b[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) acc += s.sum(i0 + k * kStep + lane * Vec<T>::kN, a[k], b[k]);
  }
  return warp_sum(acc);
}

// The smallest index of [lo, hi) whose running sum within the segment passes `target`; -1 if none does.
template <typename T>
__device__ int segment_find(const Source<T>& s, int lo, int hi, uint64_t target, int lane) {
  constexpr int kN = Vec<T>::kN, kStep = 32 * kN;
  uint64_t before = 0;
  for (int i0 = lo; i0 < hi; i0 += kBatch * kStep) {
    Vec<T> a[kBatch], b[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) s.load(i0 + k * kStep < hi ? i0 + k * kStep + lane * kN : s.vocab, a[k], b[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kStep + lane * kN;
      const uint64_t mine = s.sum(i, a[k], b[k]);
      uint64_t run = before + warp_inclusive(mine, lane);
      const uint32_t past = __ballot_sync(0xffffffffu, run > target);
      if (past) {
        const int l = __ffs(past) - 1;
        int at = -1;
        uint64_t c = run - mine;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          c += s.weight(i, e, a[k], b[k]);
          if (at < 0 && c > target) at = i + e;
        }
        return __shfl_sync(0xffffffffu, at, l);
      }
      before = __shfl_sync(0xffffffffu, run, 31);
    }
  }
  return -1;
}

// floor(u * total), u in [0, 1) taken exactly.
__device__ uint64_t scaled(float u, uint64_t total) {
  u = fminf(fmaxf(u, 0.0f), 0x1.fffffep-1f);
  const uint32_t bits = __float_as_uint(u);
  const int e = (int)(bits >> 23);
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int shift = 150 - (e ? e : 1);  // u = m 2^-shift, 24 <= shift <= 149
  const uint64_t hi = __umul64hi(m, total), lo = m * total;
  if (shift >= 128) return 0;
  if (shift >= 64) return hi >> (shift - 64);
  return (hi << (64 - shift)) | (lo >> shift);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto started = cluster.barrier_arrive();  // waited for before the first CTA's shared memory is written
  __shared__ uint64_t s_sum[kMaxCluster * kWarps];  // the first CTA's: every segment's sum
  __shared__ int s_accepted;

  const T* P = static_cast<const T*>(p.target) + (int64_t)r * p.t_stride_req;
  const T* Q = p.draft ? static_cast<const T*>(p.draft) + (int64_t)r * p.d_stride_req : nullptr;
  const int32_t* ids = p.ids + (int64_t)r * (p.T - 1);
  int nd = p.num_drafts ? __ldg(p.num_drafts + r) : p.T - 1;
  const bool bad_count = nd < 0 || nd > p.T - 1;
  nd = max(0, min(nd, p.T - 1));

  if (warp == 0) {  // how many drafts stay: 32 at a time
    int n = 0;
    for (int t0 = 0; t0 < nd; t0 += 32) {
      const int t = t0 + lane;
      bool ok = false;
      if (t < nd) {
        const int x = __ldg(ids + t);
        if (x >= 0 && x < p.vocab) {
          const float pt = as_float(P[(int64_t)t * p.t_stride_tok + x]);
          const float qt = Q ? as_float(Q[(int64_t)t * p.d_stride_tok + x]) : 1.0f;
          ok = (double)p.u_accept[(int64_t)r * (p.T - 1) + t] * (double)qt < (double)pt;
        } else if (rank == 0) {
          record_error(p.dev_err, kErrDeviceBounds);
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, t < nd && !ok);
      if (no) {
        n = t0 + __ffs(no) - 1;
        break;
      }
      n = min(t0 + 32, nd);
    }
    if (lane == 0) {
      s_accepted = n;
      if (rank == 0 && bad_count) record_error(p.dev_err, kErrDeviceBounds);
    }
  }
  __syncthreads();
  const int n = s_accepted;

  Source<T> src;
  src.p = P + (int64_t)n * p.t_stride_tok;
  src.q = (n < nd && Q) ? Q + (int64_t)n * p.d_stride_tok : nullptr;
  src.skip = (n < nd && !Q) ? __ldg(ids + n) : -1;
  src.vocab = p.vocab;
  src.wide = ((reinterpret_cast<uintptr_t>(src.p) | reinterpret_cast<uintptr_t>(src.q)) & 15) == 0;

  // segments: one a warp of the cluster, whole warp loads each
  constexpr int kStep = 32 * Vec<T>::kN;
  const int segs = ranks * kWarps;
  const int steps = (p.vocab + kStep - 1) / kStep;
  const int seg_len = (steps + segs - 1) / segs * kStep;
  // (64-bit: a segment's start may pass 2^31 for the largest vocabularies)
  auto lo_of = [&](int s) { return (int)min((int64_t)s * seg_len, (int64_t)steps * kStep); };
  const int mine = rank * kWarps + warp;
  const uint64_t sum = segment_sum(src, lo_of(mine), lo_of(mine + 1), lane);
  cluster.barrier_wait(std::move(started));
  if (lane == 0) cluster.map_shared_rank(s_sum, 0)[mine] = sum;
  cluster.sync();
  if (rank) return;

  for (int pass = 0; pass < 2; ++pass) {
    uint64_t total = 0;
    for (int s = lane; s < segs; s += 32) total += s_sum[s];
    total = warp_sum(total);
    if (total == 0 && pass == 0 && (src.q || src.skip >= 0)) {
      // nothing of p is left over (p = q up to rounding): draw from p
      src.q = nullptr;
      src.skip = -1;
      __syncthreads();
      for (int s = warp; s < segs; s += kWarps) {
        const uint64_t x = segment_sum(src, lo_of(s), lo_of(s + 1), lane);
        if (lane == 0) s_sum[s] = x;
      }
      __syncthreads();
      continue;
    }
    if (warp) return;
    int token = 0;
    if (total == 0) {
      if (lane == 0) record_error(p.dev_err, kErrDeviceBounds);
    } else {
      uint64_t target = scaled(p.u_sample[r], total), before = 0;
      token = p.vocab - 1;  // unless the sums wrapped around, one segment holds it
      for (int s0 = 0; s0 < segs; s0 += 32) {
        const uint64_t x = s0 + lane < segs ? s_sum[s0 + lane] : 0;
        const uint64_t run = before + warp_inclusive(x, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, run > target);
        if (past) {
          const int l = __ffs(past) - 1;
          const uint64_t start = __shfl_sync(0xffffffffu, run - x, l);
          const int at = segment_find(src, lo_of(s0 + l), lo_of(s0 + l + 1), target - start, lane);
          if (at >= 0) token = at;
          break;
        }
        before = __shfl_sync(0xffffffffu, run, 31);
      }
    }
    for (int t = lane; t < p.T; t += 32)
      p.out_tokens[(int64_t)r * p.T + t] = t < n ? __ldg(ids + t) : t == n ? token : -1;
    if (lane == 0) p.num_out[r] = n + 1;
    return;
  }
}

template <typename T>
pkv_status launch(const AcceptParams& p, int num_reqs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_reqs * kMaxCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, accept_kernel<T>, p) != cudaSuccess) return check_launch("spec_verify_accept");
  return check_launch("spec_verify_accept");
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_spec_verify_accept(const void* target_probs, int64_t target_stride_req,
                                             int64_t target_stride_tok, const void* draft_probs,
                                             int64_t draft_stride_req, int64_t draft_stride_tok, int32_t prob_dtype,
                                             const int32_t* draft_ids, const float* u_accept, const float* u_sample,
                                             const int32_t* num_drafts, int32_t num_reqs, int32_t T, int32_t vocab,
                                             int32_t* out_tokens, int32_t* num_out, int32_t* dev_err, void* stream) {
  using namespace pkv;
  clear_error();
  const char* name = "spec_verify_accept";
  PKV_ARG(num_reqs >= 0 && T > 0 && vocab > 0, "%s: bad size argument", name);
  PKV_UNSUP(vocab <= (1 << 30), "%s: vocab must be at most 2^30 (got %d)", name, vocab);
  PKV_UNSUP(num_reqs <= INT32_MAX / kMaxCluster, "%s: too many requests", name);
  PKV_ARG(prob_dtype >= PKV_PROB_F32 && prob_dtype <= PKV_PROB_F16, "%s: prob_dtype must be one of pkv_prob_dtype (got %d)", name, prob_dtype);
  if (num_reqs == 0) return PKV_OK;
  PKV_ARG(target_probs && u_sample && out_tokens && num_out && (T == 1 || (draft_ids && u_accept)),
          "%s: null pointer argument", name);
  const uintptr_t size = prob_dtype == PKV_PROB_F32 ? 4 : 2;
  PKV_ARG(reinterpret_cast<uintptr_t>(target_probs) % size == 0 && reinterpret_cast<uintptr_t>(draft_probs) % size == 0,
          "%s: probabilities must be aligned to their type", name);
  PKV_ARG(target_stride_tok >= 0 && target_stride_req >= 0 && draft_stride_tok >= 0 && draft_stride_req >= 0,
          "%s: strides must not be negative", name);
  AcceptParams p{target_probs, T > 1 ? draft_probs : nullptr, target_stride_req, target_stride_tok, draft_stride_req,
                 draft_stride_tok, draft_ids, u_accept, u_sample, num_drafts, T, vocab, out_tokens, num_out, dev_err};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prob_dtype == PKV_PROB_F32) return launch<float>(p, num_reqs, st);
  if (prob_dtype == PKV_PROB_BF16) return launch<__nv_bfloat16>(p, num_reqs, st);
  return launch<__half>(p, num_reqs, st);
}
