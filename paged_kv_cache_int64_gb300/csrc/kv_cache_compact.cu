// kv_cache_compact.cu - pkv_kv_cache_compact: the rows that stay move to the front of their cache.
//
// Row j of (request r, KV head h) becomes row keep[r][h][j], in K, in V, in the scale caches and in the weights; in
// place, or into other blocks. keep ascends strictly, so keep[j] >= j: a row moves down or stays.
//
// A chunk is kRows rows of a (request, KV head): a CTA reads them all into shared memory and then writes them. In place, a
// chunk's destinations are sources of earlier chunks only (of chunks whose j is below: keep[j'] = j has j' <= j), so it
// writes once those have been read: each chunk raises a flag when it has its rows, and waits, before it
// writes, for the flags of the at most two chunks whose sources can lie in its destinations. The flags depend on
// nothing but a chunk's own loads, and a CTA takes its chunks in ascending order, all CTAs resident (cooperative
// launch): every wait ends. The waits are bounded all the same; a chunk whose wait runs out does not write. Its own flag is up by
// then (raised after the wait, flags would hang on each other in a row, a chunk's time each, where rows move by a little), so
// its rows may be written over: after such a status the rows of its (request, KV head) are undefined.
//
// Those two chunks are searched for, which takes a keep that ascends. Whether it does the CTAs look at together, each at some
// parts of it while its first chunk's rows are on their way, and a word a unit counts the parts that do. Where one does not,
// a chunk waits for all lower chunks: an entry that is not valid moves nothing, and one that is valid, from >= j, is read by
// a lower chunk or the chunk itself. (16 requests of up to 32,768 in int8 / e4m3 / 4 bits, six, eight and six CTAs an SM:
// 120 / 106 / 101 us, 116 / 105 / 101 for an order taken on trust, 121 / 109 / 105 with a launch of its own that looks at it.)
#include "host_common.h"
#include "sm103.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32;  // rows of a chunk
static_assert(kRows * 8 % kThreads == 0 && 2 * kRows <= kThreads, "pieces and scales a thread");
constexpr int kPartRows = 1024;  // of keep, whose order one CTA looks at (4 a thread, on their way at once)
constexpr uint32_t kUnordered = 1u << 31;

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
  int32_t num_kv_heads, budget, block_size, chunks;
  int64_t total;  // chunks of all units
  float* weights;
  int64_t w_stride_req, w_stride_head, max_ctx;
  int32_t parts;    // of a unit's keep
  int64_t all_parts;
  uint32_t* flags;  // workspace: [units][chunks], the chunk has its rows
  uint32_t* order;  // workspace: [units], the parts that ascend; kUnordered: one does not
  int* dev_err;
  uint64_t wait_limit_ns;
};

// A row of a chunk: where it comes from and goes to.
struct Move {
  int src_blk, src_slot, dst_blk, dst_slot;  // src_blk < 0: it does not move
  int from;  // its position; -1: the weight does not move
};

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t x;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t load_relaxed(const uint32_t* p) {
  uint32_t x;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t x) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

// Row j of the unit (r, h) with n rows.
__device__ __forceinline__ Move find_move(const CompactParams& p, int unit, int r, int j, int n) {
  Move m{-1, 0, -1, 0, -1};
  if (j >= n) return m;
  const int32_t* keep = p.keep + (int64_t)unit * p.budget;
  const int from = __ldg(keep + j), above = j ? __ldg(keep + j - 1) : -1;
  const int col = from / p.block_size, dcol = j / p.block_size;
  bool ok = from >= j && from > above && col < p.src_blocks && dcol < p.dst_blocks && (!p.weights || from < p.max_ctx);
  if (ok) {
    m.src_blk = __ldg(p.src_table + (int64_t)r * p.src_stride + col);
    m.dst_blk = __ldg(p.dst_table + (int64_t)r * p.dst_stride + dcol);
    m.src_slot = from - col * p.block_size;
    m.dst_slot = j - dcol * p.block_size;
    ok = m.src_blk >= 0 && m.src_blk < p.num_blocks && m.dst_blk >= 0 && m.dst_blk < p.num_blocks;
  }
  if (!ok) {
    record_error(p.dev_err, kErrDeviceBounds);
    m.src_blk = -1;
    return m;
  }
  if (from != j) m.from = from;
  if (m.src_blk == m.dst_blk && m.src_slot == m.dst_slot) m.src_blk = -1;
  return m;
}

// The first j of [0, n) with keep[j] >= x (n if there is none), by the whole warp, 32 places a step.
__device__ int first_at_least(const int32_t* keep, int n, int x, int lane) {
  int lo = 0, len = n;
  while (len > 0) {
    const int step = (len + 31) / 32;
    const int i = lo + min(lane * step + step - 1, len - 1);  // the last of the lane's part
    const uint32_t yes = __ballot_sync(0xffffffffu, lane * step < len && __ldg(keep + i) >= x);
    if (!yes) return lo + len;
    const int l = __ffs(yes) - 1;
    const int part = min(step, len - l * step);
    lo += l * step;
    if (part == 1) return lo;
    len = part - 1;  // its last is known to pass
    if (step == 1) return lo;
  }
  return lo;
}

// Whether each of the CTA's parts of keep ascends.
__device__ __forceinline__ void look_at_order(const CompactParams& p) {
#pragma unroll 1
  for (int64_t at = blockIdx.x; at < p.all_parts; at += gridDim.x) {
    const int64_t unit = at / p.parts;
    const int part = (int)(at - unit * p.parts);
    const int len = __ldg(p.new_lens + unit / p.num_kv_heads);
    const int32_t* keep = p.keep + unit * p.budget;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPartRows / kThreads; ++i) {
      const int64_t j = (int64_t)part * kPartRows + i * kThreads + threadIdx.x;
      if (j > 0 && j < p.budget) bad |= __ldg(keep + j) <= __ldg(keep + j - 1) && j < len;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      if (bad) atomicOr(p.order + unit, kUnordered);
      else atomicAdd(p.order + unit, 1u);
    }
  }
}

// kPieces: 16-byte pieces of a row; kScale: bytes of a row's scales (0, 4 or 16).
// (CTAs an SM: as many as shared memory holds of bf16's; the others eight, a few registers spilled: int8 112 us, 4 bits 94, with
// six 120 and 101)
template <int kPieces, int kScale>
__global__ void __launch_bounds__(kThreads, kPieces == 32 ? 6 : 8) compact_kernel(const CompactParams p) {
  constexpr int kPer = kRows * kPieces / kThreads;  // pieces a thread, of K and of V
  extern __shared__ __align__(16) uint8_t s_rows[];  // [K, V][kRows][row]
  __shared__ Move s_move[kRows];
  __shared__ int s_go;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // chunks in the order (request, rows, KV head): the heads of the same rows run side by side, so that the pieces of a
  // token's row are written (and mostly read) together (16 requests of up to 32,768 keys, before later steps: 215 us with a
  // head after the other, 179 so)
  auto chunk_of = [&](int64_t c, int& unit, int& j0, int& n) {
    const int per = p.chunks * p.num_kv_heads;
    const int r = (int)(c / per), in = (int)(c - (int64_t)r * per), at = in / p.num_kv_heads;
    unit = r * p.num_kv_heads + in - at * p.num_kv_heads;
    j0 = at * kRows;
    const int len = __ldg(p.new_lens + r);
    n = max(0, min(len, p.budget));
    if (j0 == 0 && tid == 0 && n != len) record_error(p.dev_err, kErrDeviceBounds);
  };
  // the places of a chunk's rows are looked up a chunk ahead, by the first kRows threads
  int unit = 0, j0 = 0, n = 0;
  Move next{-1, 0, -1, 0, -1};
  if (blockIdx.x < p.total) {
    chunk_of(blockIdx.x, unit, j0, n);
    if (tid < kRows) next = find_move(p, unit, unit / p.num_kv_heads, j0 + tid, n);
  }
  for (int64_t c = blockIdx.x; c < p.total; c += gridDim.x) {
    const int r = unit / p.num_kv_heads, h = unit - r * p.num_kv_heads;
    const int my_unit = unit, my_j0 = j0;
    if (tid < kRows) s_move[tid] = next;
    if (tid == 0) s_go = 1;
    // (a chunk all of whose rows stay has nothing to do but its flag)
    const bool moves = __syncthreads_or(tid < kRows && (next.src_blk >= 0 || next.from >= 0));
    const bool last_chunk = my_j0 + kRows >= n;
    float* w = p.weights + (int64_t)r * p.w_stride_req + (int64_t)h * p.w_stride_head;
    const int srow = tid & (kRows - 1);
    uint8_t* spool = tid < kRows ? p.ks : p.vs;
    uint4 sx = make_uint4(0, 0, 0, 0);
    float wv = 0.0f;
    bool scales = false;
    if (moves) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = i * kThreads + tid, row = piece / kPieces;
        const Move& m = s_move[row];
        if (m.src_blk >= 0) {
          const int64_t at = m.src_blk * p.stride_blk + m.src_slot * p.stride_tok + h * p.stride_head + piece % kPieces * 16;
          const uint32_t to = smem_u32(s_rows + piece * 16);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p.k + at) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kRows * kPieces * 16), "l"(p.v + at) : "memory");
        }
      }
      scales = kScale && tid < 2 * kRows && s_move[srow].src_blk >= 0;
      if (scales) {
        const Move& m = s_move[srow];
        const uint8_t* at = spool + m.src_blk * p.s_stride_blk + m.src_slot * p.s_stride_tok + h * p.s_stride_head;
        if (kScale == 4) sx.x = *reinterpret_cast<const uint32_t*>(at);
        if (kScale == 16) sx = *reinterpret_cast<const uint4*>(at);
      }
      if (p.weights && tid < kRows && s_move[tid].from >= 0) wv = w[s_move[tid].from];
    }
    if (c == blockIdx.x && p.chunks > 1) look_at_order(p);  // (while the first chunk's rows are on their way)
    // the next chunk's places
    if (c + gridDim.x < p.total) {
      chunk_of(c + gridDim.x, unit, j0, n);
      if (tid < kRows) next = find_move(p, unit, unit / p.num_kv_heads, j0 + tid, n);
    }
    const int ci = my_j0 / kRows;
    uint32_t* flags = p.flags + (int64_t)my_unit * p.chunks;
    if (moves) {
      int dep = 0, dep_last = -1;
      uint32_t seen = 0;
      if (warp == kWarps - 1 && ci) {
        seen = load_relaxed(p.order + my_unit);
        // rows whose source lies in this chunk's destinations: at most kRows in a row from the first
        const int j = first_at_least(p.keep + (int64_t)my_unit * p.budget, my_j0, my_j0, lane);
        if (j < my_j0) {
          dep = j / kRows;
          dep_last = min(j + kRows - 1, my_j0 - 1) / kRows;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();  // every thread has its part of the rows
      if (warp == kWarps - 1) {
        if (lane == 0 && !last_chunk) store_release(flags + ci, 1u);
        if (ci) {
          const uint64_t t0 = globaltimer_ns();
          const bool brief = p.wait_limit_ns < kSuspendHintNs;  // (a test's bound: it counts as run out at once)
          bool ok = true;
          while (seen < (uint32_t)p.parts && ok) {  // (kUnordered is above)
            ok = !brief && globaltimer_ns() - t0 <= p.wait_limit_ns;
            seen = load_relaxed(p.order + my_unit);
          }
          if (seen & kUnordered) dep = 0, dep_last = ci - 1;
          for (int i = dep + lane; ok && i <= dep_last;) {
            if (!brief && load_acquire(flags + i))
              i += 32;
            else
              ok = !brief && globaltimer_ns() - t0 <= p.wait_limit_ns;
          }
          if (!ok) {
            record_error(p.dev_err, kErrTimeout);
            s_go = 0;
          }
        }
      }
      __syncthreads();
      if (s_go) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int piece = i * kThreads + tid, row = piece / kPieces;
          const Move& m = s_move[row];
          if (m.src_blk >= 0) {
            const int64_t at = m.dst_blk * p.stride_blk + m.dst_slot * p.stride_tok + h * p.stride_head + piece % kPieces * 16;
            *reinterpret_cast<uint4*>(p.k + at) = *reinterpret_cast<const uint4*>(s_rows + piece * 16);
            *reinterpret_cast<uint4*>(p.v + at) = *reinterpret_cast<const uint4*>(s_rows + (kRows * kPieces + piece) * 16);
          }
        }
        if (scales) {
          const Move& m = s_move[srow];
          uint8_t* at = spool + m.dst_blk * p.s_stride_blk + m.dst_slot * p.s_stride_tok + h * p.s_stride_head;
          if (kScale == 4) *reinterpret_cast<uint32_t*>(at) = sx.x;
          if (kScale == 16) *reinterpret_cast<uint4*>(at) = sx;
        }
        if (p.weights && tid < kRows && s_move[tid].from >= 0) w[my_j0 + tid] = wv;
      }
    } else if (tid == 0 && !last_chunk) {
      store_release(flags + ci, 1u);
    }
    __syncthreads();
  }
}

template <int kPieces, int kScale>
pkv_status launch(const CompactParams& p, cudaStream_t st) {
  static std::atomic<int> known[64];
  constexpr int kSmem = 2 * kRows * kPieces * 16;
  const int per_sm = per_device(known, [] {
    int n = 0;
    const bool ok = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, compact_kernel<kPieces, kScale>, kThreads, kSmem) == cudaSuccess;
    return ok && n > 0 ? n : 1;
  });
  const int64_t most = (int64_t)per_sm * num_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.total < most ? p.total : most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.chunks > 1 && cudaMemsetAsync(p.flags, 0, (size_t)(p.total + p.total / p.chunks) * 4, st) != cudaSuccess)
    return check_launch("kv_cache_compact");
  cudaLaunchKernelEx(&cfg, compact_kernel<kPieces, kScale>, p);
  return check_launch("kv_cache_compact");
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_kv_cache_compact_workspace_bytes(int32_t num_reqs, int32_t num_kv_heads, int32_t budget) {
  if (num_reqs <= 0 || num_kv_heads <= 0 || budget <= 0) return 0;
  const size_t chunks = ((size_t)budget + pkv::kRows - 1) / pkv::kRows;
  return ((size_t)num_reqs * (size_t)num_kv_heads * (chunks + 1) * 4 + 255) & ~(size_t)255;
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
  PKV_UNSUP((int64_t)num_reqs * num_kv_heads <= INT32_MAX && ((int64_t)budget + kRows) * num_kv_heads <= INT32_MAX, "%s: too many rows", name);
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
  PKV_ARG(!weights || rows_apart(num_reqs, w_stride_req, num_kv_heads, w_stride_head, max_ctx),
          "%s: rows of weights must not overlap", name);
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
  p.chunks = (budget + kRows - 1) / kRows;
  p.total = (int64_t)num_reqs * num_kv_heads * p.chunks;
  p.parts = (budget + kPartRows - 1) / kPartRows;
  p.all_parts = (int64_t)num_reqs * num_kv_heads * p.parts;
  p.flags = static_cast<uint32_t*>(workspace);
  p.order = p.flags + p.total;
  p.wait_limit_ns = take_wait_limit_ns();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (kv_dtype) {
    case PKV_KV_BF16: return launch<32, 0>(p, st);
    case PKV_KV_INT8: return launch<16, 4>(p, st);
    case PKV_KV_FP8: return launch<16, 0>(p, st);
    default: return launch<8, 16>(p, st);
  }
}
