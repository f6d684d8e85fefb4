// kv_attn_weights.cuh - the kernel of pkv_kv_attn_weights: scores of a step's queries against every cached key on the
// tensor cores, reduced either to each query row's log-sum-exp (kStats) or to each key's collected weight.
//
// S^T = K Q^T with the 128 keys of a tile on the MMA's M axis and the query columns (tokens x query heads of the KV
// head, kN at most) on N, fp32 in tensor memory: a key is a TMEM lane, so a thread has one key's scores and adds its
// exponentials up by itself; no sum crosses threads. The weights need one log-sum-exp a column, from the verify's
// partials or from a first launch of the same kernel, where a thread keeps one sum a column and the references are per
// warp (moved only when a score passes its reference by 2^64, so that a tile has no exchange between threads).
//
// The K cache is what is read: bf16 tiles go to the tensor core as TMA leaves them (128-byte swizzle); int8 and e4m3
// rows are widened to fp16 in registers (every code is an fp16 value) and stored to tensor memory as the A operand. Both
// operands have one type, so the queries of a (request, KV head) then become fp16 too, times the power of two that takes
// the largest of them to [2^14, 2^15): elements down to 2^-28 of the largest keep all of their bits, smaller ones are
// taken to 2^-39 of it (a score moves by that times the key's sum of magnitudes at most). (Widening to bf16 instead, which
// needs no change to the queries, takes twice the instructions, and these are what bounds the kernel: int8 137 us, e4m3 131
// for eight tokens over 32 requests of up to 40,960 keys.)
//
// The tiles of all (request, 128 keys) are one list, cut into equal ranges from the lengths on the device. A range has a
// CTA a KV head, side by side, so that the heads' parts of a token's row are read together (a head's tiles of all
// requests after another's: the same bytes, scattered, take longer). Roles: warp 0 K producer, warp 1 MMA issuer, warp 2
// tensor memory, warp 3 Q producer, warps 4-11 two reducing warpgroups (tiles in turn; with kN above 32 the log-sum-exps' take
// half of the columns each), warps 12 on the widening ones (tiles in turn where there are two).
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "host_common.h"
#include "sm103.cuh"

namespace pkv {

constexpr int kWD = 256;
constexpr int kWTile = 128;     // keys of a tile
constexpr int kWMaxCols = 128;  // query columns of a pass
constexpr int kWBadRing = 16;   // tiles whose bad segments are remembered: more than are ever under way

struct WeightParams {
  CUtensorMap qmap;   // bf16 [R*T][Hq][256]: dims {256, Hq, R*T}, box {64, group, tpc}
  // bf16: dims {256, Hkv, bs, nb}, box {64, 1, seg, 1}. int8, e4m3: dims {128, bs, 2, Hkv, nb} (a row's halves are the third),
  // box {128, seg, 2, 1, 1}, one copy a segment.
  CUtensorMap kmap;
  CUtensorMap kmap_big;  // the same with 128 rows: a whole tile inside one block
  int32_t big_ok, seg;
  const float* k_scale;
  int64_t num_blocks, s_stride_blk, s_stride_tok;
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  const int32_t* q_valid;
  int32_t num_reqs, T, group, num_q_heads, num_kv_heads, block_size;
  int32_t t_base, tpc;  // tokens of this pass: t_base .. t_base + tpc - 1
  int32_t h_base, heads;  // KV heads of this launch: h_base .. h_base + heads - 1
  float scale_log2;
  const float* part_lse;
  int32_t split_tokens, max_splits;
  const float* prev;
  const int32_t* prev_lens;
  float* weights;
  int64_t w_stride_req, w_stride_head, max_ctx;
  float2* stat;   // workspace: [CTAs][2][kWMaxCols] (reference, sum) of the requests that a CTA has a part of
  float* lse2;    // workspace: [R*T*Hq], base 2, of the requests that one CTA has whole
  int* dev_err;
  uint64_t wait_limit_ns;
};

template <int kFmt, int kN>
struct WGeo {
  static constexpr bool kWide = kFmt == PKV_KV_BF16;   // no widening
  static constexpr int kConv = kWide ? 0 : kN == 128 ? 1 : 2;  // widening warpgroups
  static constexpr int kThreads = 384 + 128 * kConv;
  static constexpr int kRowBytes = kWide ? 512 : 256;
  static constexpr int kChunks = kRowBytes / 128;      // 128-byte columns of a K tile
  static constexpr int kChunk = kWTile * 128;
  static constexpr int kStage = kChunks * kChunk;      // 64 or 32 KB
  static constexpr int kStages = kWide ? (kN == 32 ? 3 : 2) : 4;
  static constexpr int kQChunk = kN * 128;             // bf16 [kN rows][64]
  static constexpr int kQBytes = 4 * kQChunk;
  static constexpr int kQBufs = kWide ? (kN == 64 ? 2 : 1) : (kN == 128 ? 1 : 2);
  static constexpr int kOffK = kQBufs * kQBytes;
  static constexpr int kTiles = kOffK + kStages * kStage;
  static constexpr int kHalf = kN == 32 ? 32 : kN / 2; // columns of a warp's sums
  // widened K: three buffers of 128 columns, so that a tile's MMAs need not be done before the group that widened it goes on
  // (32 requests of up to 40,960 keys in int8: 163 us with two); two beside 2 x 128 columns of scores
  static constexpr int kABufs = kWide ? 1 : kN == 128 ? 2 : 3;
  static constexpr uint32_t kColA = 0;
  static constexpr uint32_t kColS = kWide ? 0 : 128 * kABufs;  // 2 x kN columns
  static_assert(kColS + 2 * kN <= 512, "tensor memory");
  static constexpr uint32_t kTmemCols = kWide ? (uint32_t)(2 * kN) : 512;
};

// The list's ranges, [c total / count, (c + 1) total / count): the longer ones spread evenly, so that requests of one length
// begin with a range where their number divides that of the ranges.
struct WRanges {
  int total, count;
  // (divisions of 32 bits where the products fit: 0.2 us less a launch, of 8)
  __device__ __forceinline__ int first(int c) const {
    return total < 1 << 24 && count <= 256 ? (int)((unsigned)total * c / (unsigned)count) : (int)((long long)total * c / count);
  }
  __device__ __forceinline__ int owner(int x) const {
    return total < 1 << 24 && count <= 256 ? (int)((((unsigned)x + 1) * count - 1) / (unsigned)total)
                                           : (int)((((long long)x + 1) * count - 1) / total);
  }
};

template <int kFmt, int kN>
struct alignas(16) WShared {
  using G = WGeo<kFmt, kN>;
  uint64_t q_full[2], q_ready[2], q_free[2];  // q_ready: as fp16
  uint64_t k_full[G::kStages], k_free[G::kStages];
  uint64_t a_ready[G::kABufs], a_free[G::kABufs];
  uint64_t s_full[2], s_free[2];
  uint64_t drain;
  uint32_t armed_k[G::kStages], armed_q[2];
  uint32_t bad[kWBadRing];
  int rows_log2[kWBadRing];  // rows of a tile's segments
  uint32_t tmem_base;
  int abort;
  int start_r, start_tile;
  int first, last;  // this CTA's tiles in the list
  WRanges ranges;
  alignas(16) float col[2][kN];              // per reducing group: minus the column's log-sum-exp (weights)
  alignas(16) int token[kN];                 // a column's token of the pass
  float q_unscale[8];                        // of the last requests' queries: the power of two back
  uint32_t q_max[2][4];                      // per widening group and warp
  alignas(16) float ref[8][G::kHalf];        // per reducing warp: the columns' references (log-sum-exps)
  alignas(16) float2 part[2][8][G::kHalf];   // per unit parity and warp: (reference, sum)
};

// A place in the list of tiles.
struct WWalk {
  int r, tile, tiles, n;
  __device__ __forceinline__ void length(const WeightParams& p) {
    const int64_t most = (int64_t)p.max_blocks * p.block_size;
    n = (int)max((int64_t)0, min((int64_t)__ldg(p.seq_lens + r), most));
    tiles = (n + kWTile - 1) / kWTile;
  }
  __device__ __forceinline__ void start(const WeightParams& p, int r0, int t0) {
    r = r0, tile = t0;
    if (r < p.num_reqs) length(p);
  }
  // to the next tile; r = num_reqs past the last
  __device__ __forceinline__ void next(const WeightParams& p) {
    if (++tile < tiles) return;
    tile = 0;
    for (++r; r < p.num_reqs; ++r) {
      length(p);
      if (tiles) return;
    }
  }
};

__device__ __forceinline__ bool w_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// The wait for a request's queries: with a bound below the time that a suspended wait may sleep (a test of the give-up
// path) it polls. (The same in every wait: 2 to 4 % of the kernel's time.)
static __device__ __noinline__ bool w_wait_brief(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if (*abort || globaltimer_ns() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool w_wait_q(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return limit_ns < kSuspendHintNs ? w_wait_brief(bar, parity, abort, limit_ns) : mbar_wait_suspend(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ void w_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// 4 int8 codes -> 4 fp16 integers, exact: fp16 bits 0x6400 | u are 1024 + u, u = code + 128.
__device__ __forceinline__ void widen4_int8(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x5140);
  hi = __byte_perm(u, 0x64646464u, 0x7362);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));  // 1152
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}
// 4 e4m3 codes -> 4 fp16 values, exact: the hardware's conversion.
__device__ __forceinline__ void widen4_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2((uint16_t)w);
  hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
}

// Sums over the warp's lanes of kC (16 or 32 at a time) columns: lane l gets column l's (kC = 16: l & 15's).
template <int kC>
__device__ __forceinline__ float w_reduce(float (&v)[kC], int lane) {
#pragma unroll
  for (int o = kC / 2; o >= 1; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int q = 0; q < o; ++q) {
      const float keep = upper ? v[q + o] : v[q];
      const float send = upper ? v[q] : v[q + o];
      v[q] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float x = v[0];
#pragma unroll
  for (int o = kC; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Maxima over the warp's lanes of 16 columns: lane l gets column l & 15's. The input is kept.
__device__ __forceinline__ float w_max16(const float (&t)[16], int lane) {
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float keep = lane & 8 ? t[q + 8] : t[q], send = lane & 8 ? t[q] : t[q + 8];
    v[q] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
  }
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) {
#pragma unroll
    for (int q = 0; q < o; ++q) {
      const float keep = lane & o ? v[q + o] : v[q], send = lane & o ? v[q] : v[q + o];
      v[q] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// The log-sum-exp, base 2, of column c of request r of n keys and KV head h, whose tiles are u0 .. u0 + tiles - 1 of the list; infinite for a
// query that sees nothing.
static __device__ __noinline__ float column_lse(const WeightParams& p, int r, int h, int n, int tiles, int u0, WRanges ranges, int c) {
  const int64_t row = ((int64_t)r * p.T + p.t_base + c / p.group) * p.num_q_heads + (int64_t)h * p.group + c % p.group;
  float m = -INFINITY, sum = 0.0f;
  if (p.part_lse) {
    const int64_t rows = (int64_t)p.num_reqs * p.T * p.num_q_heads;
    const int splits = min((n - 1) / p.split_tokens + 1, p.max_splits);
    for (int s0 = 0; s0 < splits; s0 += 8) {  // eight loads at a time
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s0 + j < splits ? __ldg(p.part_lse + (s0 + j) * rows + row) : -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (x[j] > m) {
          sum = sum * expf(m - x[j]) + 1.0f;
          m = x[j];
        } else if (x[j] != -INFINITY) {
          sum += x[j] == m ? 1.0f : expf(x[j] - m);  // (NaN comes in here)
        }
      }
    }
    // m log2(e) in two parts, so that only the last addition rounds
    const float hi = m * 1.4426950408889634f, lo = fmaf(m, 1.4426950408889634f, -hi) + m * 1.925963033500412e-8f;
    return sum != 0.0f && m < INFINITY ? hi + (lo + log2f(sum)) : INFINITY;
  }
  // the ranges that have the request's tiles: only the first can have begun with another request's
  const int c0 = ranges.owner(u0), c1 = ranges.owner(u0 + tiles - 1);
  if (c0 == c1) return __ldcg(p.lse2 + row);
  const int which = u0 > ranges.first(c0);
  for (int o0 = c0; o0 <= c1; o0 += 8) {
    float2 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = o0 + j <= c1 ? __ldcg(p.stat + (((int64_t)(o0 + j) * p.heads + h - p.h_base) * 2 + (o0 + j == c0 ? which : 0)) * kWMaxCols + c) : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (x[j].y == 0.0f) continue;
      if (x[j].x > m) {
        sum = sum * exp2f(m - x[j].x) + x[j].y;
        m = x[j].x;
      } else {
        sum += x[j].y * exp2f(x[j].x - m);
      }
    }
  }
  return sum != 0.0f ? m + log2f(sum) : INFINITY;
}

template <int kFmt, int kN, bool kStats>
__global__ void __launch_bounds__(WGeo<kFmt, kN>::kThreads, 1) kv_attn_weights_kernel(const __grid_constant__ WeightParams p) {
  using G = WGeo<kFmt, kN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WShared<kFmt, kN>& sh = *reinterpret_cast<WShared<kFmt, kN>*>(smem + G::kTiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int range = (int)blockIdx.x / p.heads, h = p.h_base + (int)blockIdx.x - range * p.heads;
  const uint64_t wl = p.wait_limit_ns;
  // every tile's scores are read by one reducing group, or by both where each has half of the columns
  constexpr bool kBoth = kStats && kN > 32;

  if (warp == 0) {
    // the list's length and this CTA's range of it (32 bits: the host has checked)
    const int64_t most = (int64_t)p.max_blocks * p.block_size;
    const int64_t reach = !kStats && p.part_lse ? (int64_t)p.max_splits * p.split_tokens : most;  // of the log-sum-exps given
    int total = 0, tiles0 = 0;  // tiles0: of request `lane`
    bool odd = false;
    for (int r = lane; r < p.num_reqs; r += 32) {
      const int len = __ldg(p.seq_lens + r);
      const int n = (int)max((int64_t)0, min((int64_t)len, most)), tiles = (n + kWTile - 1) / kWTile;
      odd |= len < 0 || len > most || n > reach || (!kStats && len > p.max_ctx);
      if (r == lane) tiles0 = tiles;
      total += tiles;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    odd = __any_sync(0xffffffffu, odd);
    // a tile each, where there are fewer tiles than ranges (so that none between a request's ranges is without a part)
    const int ranges = min((int)gridDim.x / p.heads, max(total, 1));
    const WRanges cut{total, ranges};
    const bool idle = range >= ranges;
    const int first = idle ? total : cut.first(range), last = idle ? total : cut.first(range + 1);
    int at_r = p.num_reqs, at_t = 0, before = 0;  // before: tiles of the requests before
    if (first < last)
      for (int r0 = 0; r0 < p.num_reqs; r0 += 32) {
        const int r = r0 + lane;
        int mine = r0 ? 0 : tiles0;
        if (r0 && r < p.num_reqs) {
          const int n = (int)max((int64_t)0, min((int64_t)__ldg(p.seq_lens + r), most));
          mine = (n + kWTile - 1) / kWTile;
        }
        int run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += y;
        }
        run += before;
        const uint32_t past = __ballot_sync(0xffffffffu, run > first);
        if (past) {
          const int l = __ffs(past) - 1;
          at_t = __shfl_sync(0xffffffffu, first - (run - mine), l);
          at_r = r0 + l;
          break;
        }
        before = __shfl_sync(0xffffffffu, run, 31);
      }
    if (lane == 0) {
      sh.first = first, sh.last = last, sh.ranges = cut;
      sh.start_r = at_r, sh.start_tile = at_t;
      if (odd && blockIdx.x == 0) record_error(p.dev_err, kErrDeviceBounds);
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_ready[i], 128);
      mbar_init(&sh.q_free[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kBoth ? 256 : 128);
      sh.armed_q[i] = 0;
    }
    for (int i = 0; i < G::kABufs; ++i) {
      mbar_init(&sh.a_ready[i], 128);
      mbar_init(&sh.a_free[i], 1);
    }
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_free[i], G::kWide ? 1 : 128);
      sh.armed_k[i] = 0;
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
  } else if (warp == 2) {
    tmem_alloc(&sh.tmem_base, G::kTmemCols);
    tmem_relinquish();
  } else if (warp == 3 && lane == 0) {
    prefetch_tensormap(&p.qmap);
    prefetch_tensormap(&p.kmap);
    if (p.big_ok) prefetch_tensormap(&p.kmap_big);
  }
  if (warp >= 4 && threadIdx.x - 128 < kN) {
    const int c = threadIdx.x - 128;
    sh.token[c] = c < p.tpc * p.group ? c / p.group : INT_MIN;  // (padding: sees nothing)
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  if (kStats) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  volatile int* abort = &sh.abort;
  const int count = sh.last - sh.first;
  WWalk at;
  at.start(p, sh.start_r, sh.start_tile);

  if (warp == 0) {
    // ------------------------------------------------------------------------------------ K producer
    // the table entries of a tile's segments, a lane each, are looked up a tile ahead
    const int nseg = kWTile / p.seg, seg_log2 = 31 - __clz(p.seg);
    auto look_up = [&](const WWalk& w, int& slot) -> int {
      const int pos = w.tile * kWTile + lane * p.seg;
      slot = 0;
      if (lane >= nseg || pos >= w.n) return -1;
      const int col = pos / p.block_size;
      slot = pos - col * p.block_size;
      const int blk = __ldg(p.block_table + (int64_t)w.r * p.bt_stride + col);
      return blk < 0 || (int64_t)blk >= p.num_blocks ? -2 : blk;
    };
    int slot = 0, blk = -1, st = 0, round = 0;
    if (count) blk = look_up(at, slot);
    for (int i = 0; i < count; ++i) {
      uint8_t* stage = smem + G::kOffK + st * G::kStage;
      const int my_blk = blk, my_slot = slot;
      at.next(p);
      if (i + 1 < count) blk = look_up(at, slot);
      bool ok = true;
      if (lane == 0 && round) ok = mbar_wait_suspend(&sh.k_free[st], (round - 1) & 1, abort, wl);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const uint32_t bad = __ballot_sync(0xffffffffu, my_blk == -2);
      const uint32_t loaded = __popc(__ballot_sync(0xffffffffu, my_blk >= 0));
      const int blk0 = __shfl_sync(0xffffffffu, my_blk, 0), slot0 = __shfl_sync(0xffffffffu, my_slot, 0);
      const bool big = p.big_ok && blk0 >= 0 && slot0 + kWTile <= p.block_size;  // the tile lies in one block
      if (lane == 0) {
        if (bad) record_error(p.dev_err, kErrDeviceBounds);
        sh.bad[i & (kWBadRing - 1)] = bad;
        sh.rows_log2[i & (kWBadRing - 1)] = big ? 7 : seg_log2;
        mbar_arm_tx(&sh.k_full[st], (big ? (uint32_t)kWTile : loaded * (uint32_t)p.seg) * (uint32_t)G::kRowBytes, &sh.armed_k[st]);
      }
      __syncwarp();
      if constexpr (G::kWide) {
        if (big) {
          if (w_elect()) {
#pragma unroll
            for (int c = 0; c < G::kChunks; ++c)
              tma_load_4d(stage + c * G::kChunk, &p.kmap_big, &sh.k_full[st], c * 64, h, slot0, blk0);
          }
        } else if (my_blk >= 0) {
#pragma unroll
          for (int c = 0; c < G::kChunks; ++c)
            tma_load_4d(stage + c * G::kChunk + lane * p.seg * 128, &p.kmap, &sh.k_full[st], c * 64, h, my_slot, my_blk);
        }
      } else {
        // [segment][half][rows][128 bytes]
        if (big) {
          if (w_elect()) tma_load_5d(stage, &p.kmap_big, &sh.k_full[st], 0, slot0, 0, h, blk0);
        } else if (my_blk >= 0) {
          tma_load_5d(stage + lane * p.seg * 256, &p.kmap, &sh.k_full[st], 0, my_slot, 0, h, my_blk);
        }
      }
      __syncwarp();
      if (++st == G::kStages) st = 0, ++round;
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------------------------ Q producer
    int units = 0;
    for (int i = 0; i < count; ++i, at.next(p)) {
      if (i && at.tile) continue;
      const int b = units % G::kQBufs, round = units / G::kQBufs;
      bool ok = true;
      if (lane == 0) {
        if (round) ok = mbar_wait_suspend(&sh.q_free[b], (round - 1) & 1, abort, wl);
        if (ok) {
          mbar_arm_tx(&sh.q_full[b], 512u * (uint32_t)(p.tpc * p.group), &sh.armed_q[b]);
          for (int c = 0; c < 4; ++c)
            tma_load_3d(smem + b * G::kQBytes + c * G::kQChunk, &p.qmap, &sh.q_full[b], c * 64, h * p.group, at.r * p.T + p.t_base);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      ++units;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------------ MMA issuer
    constexpr uint32_t id = idesc_f16(128, kN, G::kWide, false, false);
    int st = 0, round = 0, units = -1;
    for (int i = 0; i < count; ++i) {
      const bool first = i == 0 || at.tile == 0;
      if (first) ++units;
      const int b = units % G::kQBufs, ab = i % G::kABufs;
      const bool last = i + 1 == count || at.tile + 1 == at.tiles;
      at.next(p);
      bool ok = true;
      if (first) ok = w_wait_q(G::kWide ? &sh.q_full[b] : &sh.q_ready[b], (units / G::kQBufs) & 1, abort, wl);
      if (ok && i >= 2) ok = mbar_wait_suspend(&sh.s_free[i & 1], ((i >> 1) - 1) & 1, abort, wl);
      if (ok) ok = G::kWide ? mbar_wait_suspend(&sh.k_full[st], round & 1, abort, wl)
                            : mbar_wait_suspend(&sh.a_ready[ab], (i / G::kABufs) & 1, abort, wl);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t q_base = smem_u32(smem) + b * G::kQBytes, k_base = smem_u32(smem) + G::kOffK + st * G::kStage;
      const uint32_t d = tmem + G::kColS + (i & 1) * kN;
      if (w_elect()) {
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
          const uint64_t qd = smem_desc(q_base + (ks >> 2) * G::kQChunk + (ks & 3) * 32, 16, 1024);
          if constexpr (G::kWide)
            umma_f16_ss(d, smem_desc(k_base + (ks >> 2) * G::kChunk + (ks & 3) * 32, 16, 1024), qd, id, ks > 0);
          else
            umma_f16_ts(d, tmem + G::kColA + ab * 128 + ks * 8, qd, id, ks > 0);
        }
        umma_commit(&sh.s_full[i & 1]);
        umma_commit(G::kWide ? &sh.k_free[st] : &sh.a_free[ab]);
        if (last) umma_commit(&sh.q_free[b]);
      }
      __syncwarp();
      if (++st == G::kStages) st = 0, ++round;
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------------------------ widening
    // thread k has key row k: 256 codes -> 128 tensor-memory columns of its lane. Rows that are not loaded hold what the
    // stage had before; a row meets its own lane's scores only, and those are masked.
    if constexpr (!G::kWide) {
      const int grp = (warp - 12) >> 2;
      const int k = (warp & 3) * 32 + lane;
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      int units = -1;
      bool dead = false;  // (the groups' own barrier is reached as often by every warp)
      for (int i = 0; i < count; ++i, at.next(p)) {
        const bool first = i == 0 || at.tile == 0;
        units += first;
        if (first && (i + 1) % G::kConv == grp % G::kConv) {
          // the request's queries, by the group that does not have its first tile
          const int b = units % G::kQBufs;
          uint8_t* q = smem + b * G::kQBytes;
          const int pieces = 4 * kN * 8;  // of 16 bytes; the columns behind the pass's tokens are nobody's
          if (!dead) dead = !__all_sync(0xffffffffu, w_wait_q(&sh.q_full[b], (units / G::kQBufs) & 1, abort, wl));
          const int cols = p.tpc * p.group;
          uint32_t big = 0;  // the largest finite magnitude's bits, in the upper half
#pragma unroll 2
          for (int j = k; j < pieces; j += 128) {
            if ((j >> 3 & (kN - 1)) >= cols) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(q + j * 16);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = x[e] << 16 & 0x7fff0000u, hi = x[e] & 0x7fff0000u;
              big = max(big, max(lo < 0x7f800000u ? lo : 0u, hi < 0x7f800000u ? hi : 0u));
            }
          }
          big = __reduce_max_sync(0xffffffffu, big);
          if (lane == 0) sh.q_max[grp][warp & 3] = big;
          w_bar(4 + grp, 128);
          big = max(max(sh.q_max[grp][0], sh.q_max[grp][1]), max(sh.q_max[grp][2], sh.q_max[grp][3]));
          // 2^(14 - e) for a largest of exponent e, in two factors that stay finite
          const int up = max(-126, min(14 - ((int)(big >> 23) - 127), 141));
          const int up1 = up / 2;
          const float s0 = __int_as_float((127 + up1) << 23), s1 = __int_as_float((127 + up - up1) << 23);
#pragma unroll 2
          for (int j = k; j < pieces; j += 128) {
            if ((j >> 3 & (kN - 1)) >= cols) continue;
            uint4* ptr = reinterpret_cast<uint4*>(q + j * 16);
            const uint4 v = *ptr;
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack_f16x2(__uint_as_float(x[e] << 16) * s0 * s1, __uint_as_float(x[e] & 0xffff0000u) * s0 * s1);
            *ptr = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if (k == 0) sh.q_unscale[units & 7] = __int_as_float((127 - up1) << 23) * __int_as_float((127 - (up - up1)) << 23);
          fence_proxy_async_smem();
          w_bar(4 + grp, 128);  // (q_max may be written again)
          if (!dead) mbar_arrive(&sh.q_ready[b]);
        }
        if (i % G::kConv != grp) continue;
        const int st = i % G::kStages;
        bool ok = !dead && mbar_wait_suspend(&sh.k_full[st], (i / G::kStages) & 1, abort, wl);
        const int ab = i % G::kABufs;
        if (ok && i >= G::kABufs) ok = mbar_wait_suspend(&sh.a_free[ab], (i / G::kABufs - 1) & 1, abort, wl);
        dead = !__all_sync(0xffffffffu, ok);
        if (dead) continue;
        tc_fence_after();
        const uint32_t a = tmem + lane_off + G::kColA + ab * 128;
        const int rows_log2 = sh.rows_log2[i & (kWBadRing - 1)], half = 128 << rows_log2;  // of the key's segment
        const uint8_t* row = smem + G::kOffK + st * G::kStage + (k >> rows_log2) * 2 * half + (k & ((1 << rows_log2) - 1)) * 128;
        // (rolled, as every loop of a role: together they have to fit the instruction cache)
#pragma unroll 4
        for (int w8 = 0; w8 < 8; ++w8) {  // 32 codes, 16 columns a step
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int piece = 2 * (w8 & 3) + j;
            const uint4 v = *reinterpret_cast<const uint4*>(row + (w8 >> 2) * half + ((piece ^ (k & 7)) * 16));
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (kFmt == PKV_KV_INT8)
                widen4_int8(x[e], o[8 * j + 2 * e], o[8 * j + 2 * e + 1]);
              else
                widen4_e4m3(x[e], o[8 * j + 2 * e], o[8 * j + 2 * e + 1]);
            }
          }
          tmem_st_32x32b_x16(a + 16 * w8, o);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.a_ready[ab]);
        mbar_arrive(&sh.k_free[st]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------------------------ reducing
    const int grp = (warp - 4) >> 2, quarter = warp & 3;
    const int k = quarter * 32 + lane;  // this thread's key of a tile
    const int kseg = k / p.seg;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int c_first = kBoth ? grp * G::kHalf : 0;  // the group's first column
    const float per_tensor = kFmt == PKV_KV_FP8 ? __ldg(p.k_scale) : 1.0f;
    constexpr int kStride = kBoth ? 1 : 2;  // tiles from one of this group's to the next
    bool dead = false;
    int units = 0;

    // what a tile needs from memory is loaded a tile of this group's ahead (the block id of an int8 scale two)
    WWalk far = at, near = at;
    int far_i = kBoth ? 0 : grp, near_i = far_i;
    if (far_i && count) far.next(p), near.next(p);
    auto step = [&](WWalk& w, int& i) {
#pragma unroll
      for (int n = 0; n < kStride; ++n, ++i)
        if (i < count) w.next(p);
    };
    int blk = -1, slot = 0, near_r = -1, near_len = 0;
    auto load_block = [&]() {
      blk = -1;
      if (far_i < count) {
        const int pos = far.tile * kWTile + k;
        if (pos < far.n) {
          const int col = pos / p.block_size;
          slot = pos - col * p.block_size;
          blk = __ldg(p.block_table + (int64_t)far.r * p.bt_stride + col);
        }
      }
      step(far, far_i);
    };
    auto load_scale = [&]() {
      return blk >= 0 && (int64_t)blk < p.num_blocks
                 ? __ldg(p.k_scale + (int64_t)blk * p.s_stride_blk + (int64_t)slot * p.s_stride_tok + h) : 0.0f;
    };
    auto load_prev = [&]() {
      float x = 0.0f;
      if (near_i < count && p.prev) {
        const int key = near.tile * kWTile + k;
        if (near.r != near_r) {
          near_r = near.r;
          near_len = (int)min((int64_t)(p.prev_lens ? min(__ldg(p.prev_lens + near_r), near.n) : near.n), p.max_ctx);
        }
        if (key < near_len) x = p.prev[(int64_t)near.r * p.w_stride_req + (int64_t)h * p.w_stride_head + key];
      }
      step(near, near_i);
      return x;
    };
    float scale_next = 0.0f, prev_next = 0.0f;
    if (kFmt == PKV_KV_INT8) {
      load_block();
      scale_next = load_scale();
      load_block();
    }
    if (!kStats) prev_next = load_prev();

    // the weights' launch begins before the log-sum-exps' has ended: these are waited for, the keys are not
    if (!kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
    float l[kStats ? G::kHalf : 1];  // a thread's part of the columns' sums
    int prefix = 0, nq = kStats ? p.tpc * p.group : 0, seen = -1;  // seen: requests so far
    for (int i = 0; i < count; ++i) {
      const bool first = i == 0 || at.tile == 0, last = i + 1 == count || at.tile + 1 == at.tiles;
      seen += first;
      if (first) {
        prefix = __ldg(p.seq_lens + at.r) - p.T + p.t_base;  // the pass's token t sits at position prefix + t
        if constexpr (kStats) {
#pragma unroll
          for (int c = 0; c < G::kHalf; ++c) l[c] = 0.0f;
          for (int c = lane; c < G::kHalf; c += 32) sh.ref[warp - 4][c] = -3.4028235e38f;  // below every finite score
          __syncwarp();
        } else {
          const int valid = p.q_valid ? min(__ldg(p.q_valid + at.r), p.T) : p.T;
          nq = max(0, min(valid - p.t_base, p.tpc)) * p.group;
          w_bar(1 + grp, 128);  // the group has read the last unit's columns
          if (k < kN) sh.col[grp][k] = k < nq ? -column_lse(p, at.r, h, at.n, at.tiles, sh.first + i - at.tile, sh.ranges, k) : -INFINITY;
          w_bar(1 + grp, 128);
        }
      }
      if (kBoth || (i & 1) == grp) {
        const int key = at.tile * kWTile + k;
        float f = p.scale_log2 * per_tensor;
        const float before = prev_next;
        if (kFmt == PKV_KV_INT8) {
          f *= scale_next;
          scale_next = load_scale();
          load_block();
        }
        if (!kStats) prev_next = load_prev();
        if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait_suspend(&sh.s_full[i & 1], (i >> 1) & 1, abort, wl));
        if (!dead) {
          tc_fence_after();
          const uint32_t s_addr = tmem + lane_off + G::kColS + (i & 1) * kN + c_first;
          const bool bad_key = (sh.bad[i & (kWBadRing - 1)] >> kseg) & 1u;
          if (!G::kWide) f *= sh.q_unscale[seen & 7];
          if (bad_key) f = 0.0f;
          // columns of tokens before this do not see the key; every column does where it is not above 0
          const int behind = key < at.n ? key - prefix : INT_MAX;
          const bool open = __all_sync(0xffffffffu, behind <= 0);
          if constexpr (kStats) {
#pragma unroll
            for (int cc = 0; cc < G::kHalf / 16; ++cc) {
              const int c0 = c_first + cc * 16;
              if (c0 < nq) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(s_addr + cc * 16, v);
                tmem_wait_ld();
                float t[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) t[q] = (bad_key ? 0.0f : __uint_as_float(v[q])) * f;
                if (!open || c0 + 16 > nq) {
                  const int4* tok = reinterpret_cast<const int4*>(sh.token + c0);
#pragma unroll
                  for (int q = 0; q < 16; ++q) t[q] = behind <= reinterpret_cast<const int*>(tok)[q] ? t[q] : -INFINITY;
                }
                float* ref = sh.ref[warp - 4] + cc * 16;
                float rv[16], m = -INFINITY;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                  rv[q] = ref[q];
                  m = fmaxf(m, t[q] - rv[q]);
                }
                if (__any_sync(0xffffffffu, m > 64.0f)) {  // a reference moves
                  const float x = w_max16(t, lane);          // lane l: column l & 15's maximum
                  const float old = ref[lane & 15], now = fmaxf(old, x), a = ex2_approx(old - now);
                  __syncwarp();
                  if (lane < 16) ref[lane] = now;
                  __syncwarp();
#pragma unroll
                  for (int q = 0; q < 16; ++q) {
                    l[cc * 16 + q] *= __shfl_sync(0xffffffffu, a, q);
                    rv[q] = ref[q];
                  }
                }
#pragma unroll
                for (int q = 0; q < 16; ++q) l[cc * 16 + q] += ex2_approx(t[q] - rv[q]);
              }
            }
            tc_fence_before();
            mbar_arrive(&sh.s_free[i & 1]);
          } else {
            float sum = 0.0f;
#pragma unroll 1
            for (int c0 = 0; c0 < nq; c0 += 16) {
              uint32_t v[16];
              tmem_ld_32x32b_x16(s_addr + c0, v);
              float cv[16];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 x = *reinterpret_cast<const float4*>(sh.col[grp] + c0 + 4 * q);
                cv[4 * q] = x.x, cv[4 * q + 1] = x.y, cv[4 * q + 2] = x.z, cv[4 * q + 3] = x.w;
              }
              tmem_wait_ld();
              float e[16];
#pragma unroll
              for (int q = 0; q < 16; ++q)  // (the product rounded as for the log-sum-exp: else a score of 2^30 and its own maximum differ by 2^6)
                e[q] = ex2_approx(__fadd_rn(__fmul_rn(bad_key ? 0.0f : __uint_as_float(v[q]), f), cv[q]));
              if (!open || c0 + 16 > nq) {
                const int* tok = sh.token + c0;
#pragma unroll
                for (int q = 0; q < 16; ++q) e[q] = behind <= tok[q] && c0 + q < nq ? e[q] : 0.0f;
              }
#pragma unroll
              for (int q = 0; q < 16; q += 4) sum += (e[q] + e[q + 1]) + (e[q + 2] + e[q + 3]);
            }
            tc_fence_before();
            mbar_arrive(&sh.s_free[i & 1]);
            if (key < at.n && key < p.max_ctx)
              p.weights[(int64_t)at.r * p.w_stride_req + (int64_t)h * p.w_stride_head + key] = before + sum;
          }
        }
      }
      if constexpr (kStats) {
        if (last) {  // the warps' sums of this unit meet; both groups come here for every unit
          float2* mine = sh.part[units & 1][warp - 4];
#pragma unroll
          for (int c0 = 0; c0 < G::kHalf; c0 += 32) {
            float x[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) x[q] = l[c0 + q];
            const float y = w_reduce<32>(x, lane);
            mine[c0 + lane] = make_float2(sh.ref[warp - 4][c0 + lane], y);
          }
          w_bar(3, 256);
          const int c = (warp - 4) * 32 + lane;
          if (c < nq && !dead) {
            const int w0 = kBoth ? c / G::kHalf * 4 : 0, w1 = kBoth ? w0 + 4 : 8;
            const int cl = c % G::kHalf;
            float m = -INFINITY, sum = 0.0f;
            for (int w = w0; w < w1; ++w) {
              const float2 x = sh.part[units & 1][w][cl];
              if (x.y != 0.0f) m = fmaxf(m, x.x);
            }
            for (int w = w0; w < w1; ++w) {
              const float2 x = sh.part[units & 1][w][cl];
              if (x.y != 0.0f) sum += x.y * exp2f(x.x - m);
            }
            const int u0 = sh.first + i - at.tile;
            if (u0 >= sh.first && u0 + at.tiles <= sh.last) {
              const int64_t row = ((int64_t)at.r * p.T + p.t_base + c / p.group) * p.num_q_heads + (int64_t)h * p.group + c % p.group;
              p.lse2[row] = sum != 0.0f ? m + log2f(sum) : INFINITY;
            } else {
              p.stat[((int64_t)blockIdx.x * 2 + (u0 > sh.first)) * kWMaxCols + c] = make_float2(m, sum);
            }
          }
          ++units;
        }
      }
      at.next(p);
    }
  }

  tc_fence_before();
  // every role has left its loop; the flag's final value, the same for every thread
  const bool gave_up = __syncthreads_or(*abort != 0);
  if (gave_up) {
    // what this CTA still has in flight ends before its tensor memory is freed: the copies armed, the MMAs issued
    if (warp == 0 && lane == 0)
      for (int s = 0; s < G::kStages; ++s) drain_armed(&sh.k_full[s], sh.armed_k[s]);
    if (warp == 3 && lane == 0)
      for (int b = 0; b < G::kQBufs; ++b) drain_armed(&sh.q_full[b], sh.armed_q[b]);
    if (warp == 1) {
      if (w_elect()) {
        umma_commit(&sh.drain);
        mbar_wait_drain(&sh.drain, 0);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmemCols);
  }
  if (threadIdx.x == 0 && gave_up) record_error(p.dev_err, kErrTimeout);
  if (!kStats) asm volatile("griddepcontrol.wait;" ::: "memory");  // (no thread ends before the launch it follows)
}

template <int kFmt, int kN, bool kStats>
inline pkv_status launch_attn_weights(const WeightParams& p, int ctas, cudaStream_t stream) {
  using G = WGeo<kFmt, kN>;
  constexpr int kSmem = 1024 + G::kTiles + (int)sizeof(WShared<kFmt, kN>);
  static_assert(kSmem <= 227 * 1024, "dynamic shared memory of one CTA");
  static std::atomic<uint64_t> attr_done{0};
  once_per_device(attr_done, [] {
    cudaFuncSetAttribute(kv_attn_weights_kernel<kFmt, kN, kStats>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = !kStats && !p.part_lse ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kv_attn_weights_kernel<kFmt, kN, kStats>, p);
  return check_launch("kv_attn_weights");
}

// One pass over the columns of p: the log-sum-exps first where they are not given, then the weights.
template <int kFmt>
inline pkv_status run_attn_weights(const WeightParams& p, int ctas, cudaStream_t stream) {
  // 33 to 64 columns as 64: four bf16 prompts of 24,576 and 16 tokens of 4 heads 89 us as 128 columns, 72 as 64; eight tokens of
  // 6 heads over 8 requests of 20,008 e4m3 keys 90 and 75. Up to 32 as 32: eight tokens of 4 heads over 32 requests of up to
  // 16,384 bf16 keys 84 us as 64 columns, 76 as 32.
  const int cols = p.tpc * p.group;
  auto launch = [&](auto stats) {
    constexpr bool kStats = decltype(stats)::value;
    return cols <= 32   ? launch_attn_weights<kFmt, 32, kStats>(p, ctas, stream)
           : cols <= 64 ? launch_attn_weights<kFmt, 64, kStats>(p, ctas, stream)
                        : launch_attn_weights<kFmt, 128, kStats>(p, ctas, stream);
  };
  const pkv_status s = p.part_lse ? PKV_OK : launch(std::true_type{});
  return s != PKV_OK ? s : launch(std::false_type{});
}

pkv_status run_attn_weights_bf16(const WeightParams& p, int ctas, cudaStream_t stream);
pkv_status run_attn_weights_int8(const WeightParams& p, int ctas, cudaStream_t stream);
pkv_status run_attn_weights_fp8(const WeightParams& p, int ctas, cudaStream_t stream);

}  // namespace pkv
