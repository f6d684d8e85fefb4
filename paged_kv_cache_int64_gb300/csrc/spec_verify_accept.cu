// spec_verify_accept.cu - pkv_spec_verify_accept: which drafted tokens stay, and the token after them.
//
// Draft t of a request stays when u_t q_t(x_t) < p_t(x_t) and every draft before it stayed (the product in fp64,
// where it is exact). At the first that does not, the next token is drawn from max(p_t - q_t, 0); after the last
// draft, from p itself: the smallest i whose running sum passes u times the total.
//
// The sums are integers: each probability as the nearest multiple of 2^-46 (exact from 2^-22 up), so they do not depend on
// the order in which they are added, and the token is the one that exact arithmetic gives for these multiples. What the
// rounding does: a value moves by 2^-47 at most (one below that becomes 0 and is not drawn), a running sum over V tokens by
// V 2^-47, that of a difference by V 2^-46: 2^-30 and 2^-29 over 131,072 tokens, where u itself comes in steps of
// 2^-24. Where little is left of p (q close to it), that is more beside what is left, but then a draft goes as rarely. Multiples
// of 2^-58 would take sums of 64-bit integers in the loop: 31 us where the parts below took 25 (64 requests over 131,072
// tokens, fp32; 19 since).
//
// One cluster of CTAs a request, one pass over one row of p (and one of q). Each warp sums a contiguous segment of
// the row and gives the sum to every CTA; the warp whose segment holds the target reads it again, from its own SM's
// cache, to find the token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <limits.h>

#include <type_traits>
#include <utility>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxThreads = 512;  // of a CTA; two of them an SM, or four of half the size (64 registers a thread)
constexpr int kMaxWarps = kMaxThreads / 32;
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

// A probability in [0, 1] as the nearest multiple of 2^-46, in two parts: hi 2^23 + lo. Four fp32 operations: adding 1 (or
// 1.5) to x rounds it to a multiple of 2^-23 and leaves that multiple in the sum's low bits. (The conversion to 64-bit
// integers runs at a small part of their rate; 64-bit shifts of the mantissa take twice the instructions.)
struct Fixed {
  int hi, lo;
};
__device__ __forceinline__ Fixed fixed46(float p) {
  const float t = __fadd_rn(p, 1.0f);
  const float rest = __fsub_rn(p, __fsub_rn(t, 1.0f));  // exact, at most 2^-24
  return {__float_as_int(t) - 0x3f800000, __float_as_int(__fmaf_rn(rest, 0x1p23f, 1.5f)) - 0x3fc00000};
}
// To [0, 1], NaN to 0.
__device__ __forceinline__ float saturated(float x) {
  float y;
  asm("add.rn.sat.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// Elements [i, i + kN) of a row of `vocab` values, 0 outside of it. row + i is 16-byte aligned; elements before the row and
// behind it are not read.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int i, int vocab) {
  constexpr int kN = 16 / (int)sizeof(T);
  if (i >= 0 && i + kN <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + i));
  T v[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) v[e] = i + e >= 0 && i + e < vocab ? row[i + e] : T(0.0f);
  uint4 x;
  memcpy(&x, v, 16);
  return x;
}

// The rows that are read: p alone; p and q, aligned alike; p and q, not so.
enum { kOne, kAlike, kShifted };

// What the token is drawn from: p, max(p - q, 0), or p without the draft's own token. Indices run in vectors of 16 bytes
// that are aligned in p's row, so the first may begin before the row; q's row is read in its own aligned vectors, two
// for one of p's where the rows are not aligned alike, and shifted.
template <typename T>
struct Source {
  static constexpr int kN = 16 / (int)sizeof(T);
  const T* p;
  const T* q;   // null: none
  int skip;     // index left out, or below every index
  int vocab;
  int begin;    // index of the first vector, -(kN - 1) .. 0
  int shift;    // elements by which p's vectors begin behind q's, 0 .. kN - 1

  __device__ __forceinline__ void align() {
    begin = -(int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
    const int q_begin = -(int)(reinterpret_cast<uintptr_t>(q) % 16 / sizeof(T));
    shift = q ? (begin - q_begin + kN) % kN : 0;
  }
  // x with element e set to 0
  static __device__ __forceinline__ uint4 without(const uint4& x, int e) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const int word = e * (int)sizeof(T) / 4;
    const uint32_t left = sizeof(T) == 4 ? 0u : e & 1 ? 0xffffu : 0xffff0000u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j == word) w[j] &= left;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // The lane's vectors of the step that begins at index i0 (begin + a multiple of a warp's load); a: p's, b: q's (kOne: none).
  // Steps from `end` on are 0. inside: the step is before `end`, and no vector that it reads passes the row's ends.
  template <int kMode>
  __device__ __forceinline__ void load(int i0, int end, int lane, bool inside, uint4& a, uint4& b) const {
    const int i = i0 + lane * kN;
    a = b = make_uint4(0, 0, 0, 0);
    if (!inside && i0 >= end) return;
    a = inside ? __ldg(reinterpret_cast<const uint4*>(p + i)) : load_vec(p, i, vocab);
    if constexpr (kMode == kOne) {
      if ((unsigned)skip - (unsigned)i < (unsigned)kN) a = without(a, skip - i);
    } else {
      const T* at = q + (i - shift);
      b = inside ? __ldg(reinterpret_cast<const uint4*>(at)) : load_vec(q, i - shift, vocab);
      if constexpr (kMode == kShifted) {
        const uint4 c = inside ? __ldg(reinterpret_cast<const uint4*>(at + kN)) : load_vec(q, i - shift + kN, vocab);
        uint32_t w[8] = {b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        const int bytes = shift * (int)sizeof(T);
        if (bytes & 8) {
#pragma unroll
          for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
        }
        if (bytes & 4) {
#pragma unroll
          for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
        }
        if (bytes & 2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
        }
        b = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  static __device__ __forceinline__ float value(const uint4& x, int e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (sizeof(T) == 4) return __uint_as_float(w[e]);
    if (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)(w[e / 2] >> (e & 1 ? 16 : 0))));
    return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  template <int kMode>
  static __device__ __forceinline__ Fixed weight(int e, const uint4& a, const uint4& b) {
    const float x = saturated(value(a, e));
    const Fixed f = fixed46(x);
    if constexpr (kMode != kOne) {
      const Fixed g = fixed46(fminf(saturated(value(b, e)), x));  // q, p at most: the difference is 0 where q is above
      return {f.hi - g.hi, f.lo - g.lo};
    }
    return f;
  }
};
// (2^23 hi is 2^46 at most for a vector or two: the parts are added up in 32 bits, a batch at a time)
__device__ __forceinline__ uint64_t joined(const Fixed& f) { return (uint64_t)((int64_t)f.hi * (1 << 23) + f.lo); }

__device__ __forceinline__ uint64_t warp_inclusive(uint64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Steps (a vector a lane and table) whose loads go out together: no more than 64 registers hold without spilling, as 32
// warps an SM stream better than 16 (64 requests over 131,072 tokens: 26 us). The next batch is not loaded ahead: with
// it the registers spill (21 us; 19.2 without).
template <int kMode>
constexpr int kBatchOf = kMode == kOne ? 4 : 2;
// steps (a vector a lane) that are reduced together: 256 values of 2^23 at most each, 2^31 together
template <typename T>
constexpr int kGroupOf = (int)sizeof(T) / 2;

// The sum of kSteps steps: two 32-bit reductions (unsigned).
template <int kMode, typename T, int kSteps>
__device__ __forceinline__ uint64_t steps_sum(const uint4* a, const uint4* b, Fixed& mine) {
  static_assert(kSteps * 32 * Source<T>::kN <= 256, "32 bits");
  mine = {0, 0};
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
#pragma unroll
    for (int e = 0; e < Source<T>::kN; ++e) {
      const Fixed f = Source<T>::template weight<kMode>(e, a[k], b[k]);
      mine.hi += f.hi, mine.lo += f.lo;
    }
  // the low parts of 256 differences may add up to 2^31 (each p half a multiple of 2^-23 above one, each q half below):
  // a lane's go into its high part first, so that both sums are of what is not negative
  mine.hi += mine.lo >> 23, mine.lo &= (1 << 23) - 1;
  return ((uint64_t)__reduce_add_sync(0xffffffffu, (unsigned)mine.hi) << 23) +
         __reduce_add_sync(0xffffffffu, (unsigned)mine.lo);
}

// The warp's sum over [lo, hi), whole groups of steps; lane l gets in `part` that of its l-th part of `per` groups.
template <int kMode, typename T>
__device__ __forceinline__ uint64_t segment_sum(const Source<T>& s, int lo, int hi, int per, int lane, uint64_t& part) {
  constexpr int kStep = 32 * Source<T>::kN, kBatch = kBatchOf<kMode>, kGroup = kGroupOf<T>;
  uint64_t acc = 0;
  int groups = 0, parts = 0;
  part = 0;
#pragma unroll 1
  for (int i0 = lo; i0 < hi; i0 += kBatch * kStep) {
    uint4 a[kBatch], b[kBatch];
    constexpr int kAll = kBatch * kStep;
    if (i0 - Source<T>::kN >= 0 && i0 + kAll <= hi && i0 + kAll + Source<T>::kN <= s.vocab) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) s.template load<kMode>(i0 + k * kStep, hi, lane, true, a[k], b[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) s.template load<kMode>(i0 + k * kStep, hi, lane, false, a[k], b[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; k += kGroup) {
      Fixed mine;
      const uint64_t x = steps_sum<kMode, T, kGroup>(a + k, b + k, mine);  // (groups behind the last one add 0)
      if (lane == parts) part += x;
      acc += x;
      if (++groups == per) groups = 0, ++parts;
    }
  }
  return acc;
}

// The smallest index of [lo, hi), whole steps, whose running sum from lo passes `target`; -1 if none does.
template <int kMode, typename T>
__device__ __forceinline__ int find(const Source<T>& s, int lo, int hi, uint64_t target, int lane) {
  constexpr int kN = Source<T>::kN, kStep = 32 * kN;
  uint64_t before = 0;
#pragma unroll 1
  for (int i0 = lo; i0 < hi; i0 += kStep) {
    const int i = i0 + lane * kN;
    uint4 a, b;
    s.template load<kMode>(i0, hi, lane, false, a, b);
    Fixed sum;
    const uint64_t step = steps_sum<kMode, T, 1>(&a, &b, sum);
    if (before + step > target) {
      const uint64_t mine = joined(sum), run = before + warp_inclusive(mine, lane);
      int at = -1;
      uint64_t c = run - mine;
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        c += joined(Source<T>::template weight<kMode>(e, a, b));
        if (at < 0 && c > target) at = i + e;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run > target);
      return __shfl_sync(0xffffffffu, at, past ? __ffs(past) - 1 : 31);
    }
    before += step;
  }
  return -1;
}

// A uniform number, to [0, 1 - 2^-24], NaN to 0.
__device__ __forceinline__ float in_range(float u) { return fminf(fmaxf(u, 0.0f), 0x1.fffffep-1f); }

// floor(u * total), u in [0, 1) taken exactly.
__device__ uint64_t scaled(float u, uint64_t total) {
  u = in_range(u);
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
__global__ void __launch_bounds__(kMaxThreads, 2) accept_kernel(const AcceptParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto started = cluster.barrier_arrive();  // waited for before another CTA's shared memory is written
  __shared__ uint64_t s_sum[2][kMaxCluster * kMaxWarps];  // every segment's sum, of the first and of a second pass
  __shared__ int s_accepted;

  const T* P = static_cast<const T*>(p.target) + (int64_t)r * p.t_stride_req;
  const T* Q = p.draft ? static_cast<const T*>(p.draft) + (int64_t)r * p.d_stride_req : nullptr;
  const int32_t* ids = p.ids + (int64_t)r * (p.T - 1);
  int nd = p.num_drafts ? __ldg(p.num_drafts + r) : p.T - 1;
  const bool bad_count = nd < 0 || nd > p.T - 1;
  nd = max(0, min(nd, p.T - 1));

  if (warp == 0) {  // how many drafts stay: 32 at a time
    int n = 0;
    for (int t0 = 0; t0 < p.T - 1; t0 += 32) {
      const int t = t0 + lane;
      bool ok = false;
      if (t < p.T - 1) {
        const int x = __ldg(ids + t);  // (drafts behind the request's own too, while num_drafts is on its way)
        const float u = in_range(p.u_accept[(int64_t)r * (p.T - 1) + t]);
        if (t < nd) {
          if (x >= 0 && x < p.vocab) {
            const float pt = as_float(P[(int64_t)t * p.t_stride_tok + x]);
            const float qt = Q ? as_float(Q[(int64_t)t * p.d_stride_tok + x]) : 1.0f;
            ok = (double)u * (double)qt < (double)pt;
          } else if (rank == 0) {
            record_error(p.dev_err, kErrDeviceBounds);
          }
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        n = t0 + __ffs(no) - 1;  // the first that goes, or the first behind the last
        break;
      }
      n = t0 + 32;
    }
    if (lane == 0) {
      s_accepted = min(n, nd);
      if (rank == 0 && bad_count) record_error(p.dev_err, kErrDeviceBounds);
    }
  }
  __syncthreads();
  const int n = s_accepted;

  Source<T> src;
  src.p = P + (int64_t)n * p.t_stride_tok;
  src.q = (n < nd && Q) ? Q + (int64_t)n * p.d_stride_tok : nullptr;
  src.skip = (n < nd && !Q) ? __ldg(ids + n) : INT_MIN;
  if (src.skip < 0) src.skip = INT_MIN;  // (a draft id out of range leaves p whole; beside q it changes nothing)
  src.vocab = p.vocab;
  src.align();

  // segments: one a warp of the cluster, whole warp loads each
  constexpr int kStep = 32 * Source<T>::kN;
  const int warps = blockDim.x >> 5;
  const int segs = ranks * warps;
  const int steps = (p.vocab - src.begin + kStep - 1) / kStep;
  constexpr int kGroup = kGroupOf<T>;
  const int seg_groups = (steps + segs * kGroup - 1) / (segs * kGroup), seg_len = seg_groups * kGroup * kStep;
  const int per = (seg_groups + 31) / 32;  // groups of a lane's part of the segment
  const int mine = rank * warps + warp;
  // (64-bit: a segment's start may pass 2^31 for the largest vocabularies)
  const int lo = src.begin + (int)min((int64_t)mine * seg_len, (int64_t)steps * kStep);
  const int hi = src.begin + (int)min((int64_t)(mine + 1) * seg_len, (int64_t)steps * kStep);

#pragma unroll 1
  for (int pass = 0;; ++pass) {
    uint64_t part;
    const uint64_t sum = !src.q ? segment_sum<kOne>(src, lo, hi, per, lane, part)
                         : src.shift ? segment_sum<kShifted>(src, lo, hi, per, lane, part)
                                     : segment_sum<kAlike>(src, lo, hi, per, lane, part);
    if (pass == 0) cluster.barrier_wait(std::move(started));
    // every CTA gets every segment's sum: the warp whose segment holds the target goes on, from its own SM's cache
    if (lane < ranks) cluster.map_shared_rank(&s_sum[pass][0], lane)[mine] = sum;
    cluster.sync();
    // the running sums: each lane has kMaxCluster * kMaxWarps / 32 segments in a row
    constexpr int kPer = kMaxCluster * kMaxWarps / 32;
    uint64_t x[kPer], own = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int sg = lane * kPer + j;
      x[j] = sg < segs ? s_sum[pass][sg] : 0;
      own += x[j];
    }
    const uint64_t run = warp_inclusive(own, lane), total = __shfl_sync(0xffffffffu, run, 31);
    int token = 0;
    if (total == 0) {
      if (pass == 0 && (src.q || src.skip != INT_MIN)) {
        // nothing of p is left over (p = q up to rounding): from p. Uniform over the cluster.
        src.q = nullptr;
        src.skip = INT_MIN;
        src.shift = 0;
        continue;
      }
      if (mine) return;
      if (lane == 0) record_error(p.dev_err, kErrDeviceBounds);
    } else {
      // the segment that holds the target; every warp finds the same one (the last, where sums wrapped around and
      // none does)
      const uint64_t target = scaled(p.u_sample[r], total);
      const uint32_t past = __ballot_sync(0xffffffffu, run > target);
      int chosen = segs - 1;
      uint64_t start = run - own;
      if (past) {
        int j = 0;
#pragma unroll
        for (int t = 0; t < kPer - 1; ++t)
          if (j == t && start + x[t] <= target) start += x[t], ++j;
        chosen = __shfl_sync(0xffffffffu, lane * kPer + j, __ffs(past) - 1);
        start = __shfl_sync(0xffffffffu, start, __ffs(past) - 1);
      }
      if (chosen != mine) return;
      // the part of the segment that holds it, then its steps
      const uint64_t left = past ? target - start : 0, upto = warp_inclusive(part, lane);
      const uint32_t in = __ballot_sync(0xffffffffu, upto > left);
      const int l = in ? __ffs(in) - 1 : 31;
      const int from = min(lo + l * per * kGroup * kStep, hi);
      const int to = min(from + per * kGroup * kStep, hi);
      const uint64_t behind = left - __shfl_sync(0xffffffffu, upto - part, l);
      token = !src.q ? find<kOne>(src, from, to, behind, lane)
              : src.shift ? find<kShifted>(src, from, to, behind, lane) : find<kAlike>(src, from, to, behind, lane);
      if (token < 0) token = p.vocab - 1;
    }
    for (int t = lane; t < p.T; t += 32)
      p.out_tokens[(int64_t)r * p.T + t] = t < n ? __ldg(ids + t) : t == n ? token : -1;
    if (lane == 0) p.num_out[r] = n + 1;
    return;
  }
}

template <typename T>
pkv_status launch(const AcceptParams& p, int num_reqs, cudaStream_t stream) {
  // Every request's CTAs on the device at once, as many threads a request as that leaves: a cluster of eight CTAs of 512
  // (two an SM) or 256 threads (four), or a smaller one.
  const int room = num_sms() * 4;  // CTAs of 256 threads
  int ctas = kMaxCluster;
  while (ctas > 1 && (int64_t)num_reqs * ctas > room) ctas /= 2;
  const int threads = (int64_t)num_reqs * ctas * 2 <= room ? kMaxThreads : kMaxThreads / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_reqs * ctas));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, accept_kernel<T>, p);
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
  // a request's CTAs read its drafts while another's write their tokens (num_out over num_drafts: each after it has been read)
  const uint64_t reqs = (uint64_t)num_reqs * 4, tokens = reqs * (uint64_t)T, ids = reqs * (uint64_t)(T - 1);
  PKV_ARG((T == 1 || (!overlaps(out_tokens, tokens, draft_ids, ids) && !overlaps(num_out, reqs, draft_ids, ids))) &&
              !overlaps(out_tokens, tokens, num_out, reqs) &&
              (!num_drafts || (!overlaps(out_tokens, tokens, num_drafts, reqs) &&
                               (num_out == num_drafts || !overlaps(num_out, reqs, num_drafts, reqs)))),
          "%s: out_tokens and num_out must not overlap draft_ids, num_drafts or each other", name);
  AcceptParams p{target_probs, T > 1 ? draft_probs : nullptr, target_stride_req, target_stride_tok, draft_stride_req,
                 draft_stride_tok, draft_ids, u_accept, u_sample, num_drafts, T, vocab, out_tokens, num_out, dev_err};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prob_dtype == PKV_PROB_F32) return launch<float>(p, num_reqs, st);
  if (prob_dtype == PKV_PROB_BF16) return launch<__nv_bfloat16>(p, num_reqs, st);
  return launch<__half>(p, num_reqs, st);
}
