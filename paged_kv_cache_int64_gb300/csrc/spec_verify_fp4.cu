// spec_verify_fp4.cu - pkv_spec_verify_attn_fp4: decode / speculative-verify attention over the paged
// 4-bit cache.
//
// For a KV head, the columns are the query rows that share it (tokens x group, kCols of them) and the
// MMAs are swapped, so the 128 keys of a tile are the M dimension:
//   S^T = K Q^T (M 128 keys, N kCols, K 256),  P = 2^(S f - m),  O^T += V^T P^T (M 2 x 128, K 128 keys),
// out = O / sum P * v_scale, f = softmax_scale log2(e) k_scale.
//
// A tile of 128 keys is 36 KB, 0.83 us (1,590 clocks) of an SM's share of the measured copy rate, and holds
// 65,536 codes. What the design follows from:
//   - K needs no widening: QK runs on the stored codes and scales (kind::mxf4nvf4), with a query row as a
//     sum of six e2m1 rows under block scales (kTerms). Widening K to fp16 in registers as well took the
//     issue slots that V needs (eight tokens over up to 40,960 keys, with four terms: 235 us against 210).
//   - V has to be transposed (M is head_dim) and its scales vary along both axes, so it is widened, to fp16,
//     which holds e2m1 * e4m3 exactly (6 significant bits). ldmatrix.m16n16.trans.b8 hands a thread one
//     byte column of four keys, the conversion of a byte gives the (even, odd) elements of one key, and
//     they go to tensor memory as a column of the A operand: written back to shared memory, 64 KB a tile
//     would be stored and read again. A column then mixes two rows of head_dim, so P^T has two rows a
//     key, one that meets the even elements and one that meets the odd ones, and O^T two column blocks.
//   - The scales of V are laid out once by one warp as fp16, transposed.
//   - The weights may grow to 2^15 before a column's maximum moves (they start at 2^8); a vote of the
//     column group's warps finds the tiles where one has to, so that most tiles have no reduction over
//     the keys, and the sums stay in registers until the end. P is fp16 (2^-11 a weight, random over the
//     keys; 11 bits where bf16 has 8), its sum takes the fp32 weights.
//
// The keys are divided evenly: the tiles of a "line" (one KV head's, for all requests one after the
// other) are cut into equal ranges, one a CTA, and the CTAs of the lines (heads) work side by side on
// the same pages. Request pieces that a cut divides are merged by a second, small kernel; a CTA has
// at most one piece that began before it and one that ends after it, so two slots of workspace. The
// pipeline runs on from one request to the next.
//
// Roles: warps 0 and 6 TMA producers of K and V; 1 QK issuer; 2 PV issuer; 3 V scales; 4-5 Q; 7 K scales;
// 8-15 V columns; 16-23 softmax, a warpgroup for half the columns.
//
// Measured (4 KV heads, 16 query heads): one token, 32 requests of up to 16,384 keys 67 us (3.9
// TB/s of cache); one token, one request of 262,144 keys 63 us (4.8 TB/s); eight tokens, 32 requests of
// up to 40,960 keys 209 us (3.6 TB/s); one token, one request of 1,024 keys 15.0 us. No unit is above a
// half (issue slots 46 %, tensor pipe 23 %): a tile passes through scores, exponentials, vote, weights and
// back in about 1,800 (kCols 16) or 2,500 clocks (32) of latencies, of which the double buffers overlap
// two tiles. With 32 columns the 80 registers that 24 warps leave spill (172 bytes stored, 292 loaded). About 14 us
// of every call are none of its tiles': 3 until the range is known, 2 to 3 until the first tile has
// come, 2 through it, then the launch of the merge and its two or three turns of loads.
#include <cuda_bf16.h>

#include <numeric>

#include "host_common.h"
#include "kv_fp4.cuh"

namespace pkv {

namespace {

constexpr int kBN = 128;                  // keys of a tile
constexpr int kCodeTile = kBN * kFp4RowBytes;  // 16 KB
constexpr int kScaleTile = kBN * kFp4Groups;   // 2 KB
constexpr int kStage = kCodeTile + kScaleTile;
constexpr int kMaxCols = 32;
constexpr uint32_t kTmemCols = 512;
// Q as a sum of six e2m1 rows, digits of base 8: a block of 16 elements whose largest magnitude lies in
// [2^E, 2^(E+1)) has the scales 2^E, 2^(E-3), ... 2^(E-15), each term the last one's remainder rounded to
// halves (which are e2m1 values up to 2). What is kept are multiples of 2^(E-16): a bf16 element has 8
// bits, so all of them down to 2^-9 of the block's largest, and 2^-17 of the largest is the most that a smaller
// one is off by. (Four terms keep 8 bits down to 2^-3: with one channel of 16 a hundred times the others,
// and K's small there, outputs were off by 5 % and more. They took 195 us where six take 208, eight tokens over
// up to 40,960 keys; one token measured the same.) Rows are brought to [2^8, 2^9) first; e4m3 ends at 2^-9, so that
// no block keeps less than 2^-10 there, 2^-18 of the row's power of two. Terms stand side by side as
// columns of one product (kSide; the instruction takes 40 clocks for 16 or 32 columns and 49 for 64), and
// the softmax adds their scores.
constexpr int kTerms = 6;
constexpr float kUnset = -3e38f;          // running maximum of a column that has seen no key
constexpr float kStart = 8.0f;            // a new maximum's weight is 2^8; the maximum moves when a thread's
constexpr float kMove = 32768.0f;         // weights of one key add up to more than this (fp16 ends at 65,504)

// Workspace of n CTAs: their notes for the merge, [n]; the sums and maxima (log2) of two slots of each (0: the
// piece that began before it, 1: the piece that goes on after it), [n][2][kMaxCols]; the slots' O, [n][2][live
// columns][256]. Close together: with a CTA's whole share in one place the merge's loads met a page each.
struct Note {
  int32_t pieces, r, unit, pad;  // pieces: CTAs of the line that hold the unit (0: none begins here and goes on)
};
constexpr size_t kWorkspaceOfCta = sizeof(Note) + 2 * kMaxCols * (sizeof(float2) + kFp4D * sizeof(float));
static_assert(sizeof(Note) == 16 && kWorkspaceOfCta % 16 == 0, "workspace of a CTA");
struct Workspace {
  Note* notes;
  float2* lm;
  float* o;
  __host__ __device__ Workspace(void* base, int n) {
    notes = static_cast<Note*>(base);
    lm = reinterpret_cast<float2*>(notes + n);
    o = reinterpret_cast<float*>(lm + (size_t)n * 2 * kMaxCols);
  }
};

template <int kCols>
struct Geo {
  static constexpr int kGC = kCols == 16 ? 8 : 16;  // columns of a softmax warpgroup
  static constexpr int kGroups = kCols / kGC;
  static constexpr int kThreads = 512 + 128 * kGroups;
  // K codes are held until QK has read them, V codes until they are converted, which waits for the PV two
  // tiles back
  static constexpr int kKStages = kCols == 16 ? 4 : 3;
  static constexpr int kVStages = kCols == 16 ? 4 : 3;
  static constexpr int kSide = kCols == 16 ? 3 : 2;  // terms side by side
  static constexpr int kTurns = kTerms / kSide;      // products of a step of K
  static constexpr int kQTerm = kCols * 128;     // codes of one term of Q: [kCols rows][128 B], 128-byte swizzle
  static constexpr int kQsTurn = 4 * 512;        // scales of kSide terms: [4 steps of 64 elements][32 lanes][16 B]
  static constexpr int kQBuf = kTerms * kQTerm + kTurns * kQsTurn;
  static constexpr int kPRow = kCols * 4;        // bytes of a row of P^T: 2 kCols columns
  static constexpr uint32_t kPLayout = kCols == 16 ? kLayoutSW64 : kLayoutSW128;
  static constexpr int kPBuf = 2 * kBN * kPRow;
  static constexpr int kPBufs = kCols == 16 ? 2 : 1;
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kOffQ + 2 * kQBuf;
  static constexpr int kOffSf = kOffP + kPBufs * kPBuf;     // V scales, fp16 [4 quarters][32 key quads][4 groups][4 keys]
  static constexpr int kSfBuf = kBN * kFp4Groups * 2;
  static constexpr int kOffKs = kOffSf + 2 * kSfBuf;        // K scales: [4 steps][32 lanes][4 keys lane + 32 x][4 groups]
  static constexpr int kOffK = kOffKs + 2 * kScaleTile;     // stages: codes, then scales
  static constexpr int kOffV = kOffK + kKStages * kStage;
  static constexpr int kTiles = kOffV + kVStages * kStage;
  // tensor memory; the scale factors in blocks of 4 columns (one step of 64 elements)
  static constexpr uint32_t kColV = 0;                      // two V tiles: a column a key
  static constexpr uint32_t kColS = 256;                    // two S^T, the sums of kSide terms side by side
  static constexpr uint32_t kSBuf = 64;
  static constexpr uint32_t kColO = kColS + 2 * kSBuf;      // O^T of the even elements, then of the odd ones
  static constexpr uint32_t kColKs = kColO + 2 * kCols;     // a tile's K scales
  static constexpr uint32_t kColQs = kColKs + 16;           // Q scales of the turns
  static_assert(kTerms % kSide == 0 && kSide * kCols <= (int)kSBuf, "terms side by side");
  static_assert(kColQs + 16 * kTurns <= kTmemCols && kColKs % 4 == 0, "tensor memory");
  static_assert(kOffQ == 0 && kQBuf % 1024 == 0 && kOffP % 1024 == 0 && kOffK % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");
};

template <int kCols>
struct alignas(16) Shared {
  static constexpr int kKStages = Geo<kCols>::kKStages, kVStages = Geo<kCols>::kVStages;
  uint64_t k_full[kKStages], k_empty[kKStages];  // codes and scales of a tile's K
  uint64_t v_full[kVStages], v_empty[kVStages];  // ... of its V
  uint64_t q_first;                              // every warp's share of the first run's Q
  uint64_t q_ready[4], q_free[2];                // Q of run s (buffer s % 2; barrier s % 4: Q may be 3 runs ahead of the softmax)
  uint64_t ks_ready[2];                          // K scales of a tile laid out
  uint64_t s_full[2], s_free[2];                 // S^T; s_free also means that the K scales are read
  uint64_t sf_ready[2], sf_free[2];              // transposed V scales
  uint64_t vt_ready[2];                          // V tile in tensor memory
  uint64_t p_full[2], pv_done[2];                // P^T written; PV of the tile complete (frees V tile and P^T)
  uint64_t drain;
  uint32_t k_armed[kKStages], v_armed[kVStages];
  uint32_t k_bad[kKStages], v_bad[kVStages];     // key segments in a bad block
  uint32_t tmem_base;
  int abort;
  int v_nan;                                     // a NaN V scale was left out for a key that some columns do not see
  int r0, u0, t00;                               // first tile of the CTA's range
  long long wsum[Geo<kCols>::kThreads / 32];
  int32_t row_off[kCols];                        // column -> token * Hq + head in group
  int32_t tok[kCols];                            // column -> token
  alignas(16) float f[8][kCols];                 // column factors of the segment (ring: the softmax may be 4 behind)
  alignas(16) float m[kCols];                    // running maxima, log2, negated
  float red[Geo<kCols>::kGroups][4][Geo<kCols>::kGC];
  float fin[kCols];                              // 1 / sum, 0 for a column without a key
};

struct Params {
  // K then V, each: codes [nb][bs][hkv][128 B] and scales [nb][bs][hkv][16 B] in boxes of seg keys, then
  // both in boxes of 128 keys (block_size >= 128)
  CUtensorMap map[8];
  const __nv_bfloat16* q;
  const uint8_t* v_bscale;
  int64_t scale_stride_blk, scale_stride_tok, scale_stride_head;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  int64_t bt_stride, num_blocks;
  int32_t max_blocks, big_ok, block_size, seg;
  const int32_t* seq_lens;
  int32_t num_reqs, T, group, num_q_heads;
  int32_t tpc, n_tg;               // tokens of a CTA's columns; column groups of a KV head
  int32_t lines, units, ctas;      // lines; units of a request in a line; CTAs of a line
  float scale_log2;
  __nv_bfloat16* out;
  void* ws;
  int* dev_err;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ int64_t line_begin(int64_t total, int c, int ctas) {
  const uint64_t x = (uint64_t)total * (uint32_t)c;  // (a 32-bit division where it does)
  return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)ctas) : (int64_t)(x / (uint32_t)ctas);
}

// The tiles of a CTA, as runs of consecutive tiles of one (request, unit). Every role walks the same runs.
struct Cursor {
  int r, u, t;
  int64_t left;
};
struct Run {
  int r, u, t0, n, len, tiles;
};
__device__ __forceinline__ bool next_run(const Params& p, Cursor& c, Run& s) {
  if (c.left <= 0) return false;
  int len = 0;
  while (true) {
    if (c.r >= p.num_reqs) return false;
    len = __ldg(p.seq_lens + c.r);
    if (len > 0) break;
    ++c.r;
  }
  s.r = c.r;
  s.u = c.u;
  s.t0 = c.t;
  s.len = len;
  s.tiles = (int)(((int64_t)len + kBN - 1) / kBN);
  s.n = (int)min((int64_t)(s.tiles - s.t0), c.left);
  if (s.n <= 0) return false;
  c.left -= s.n;
  c.t += s.n;
  if (c.t == s.tiles) {
    c.t = 0;
    if (++c.u == p.units) {
      c.u = 0;
      ++c.r;
    }
  }
  return true;
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// kind::mxf4nvf4: e2m1 operands with an e4m3 scale per 16 elements (K = 64), fp32 accumulator, A and B in
// shared memory, the scales in tensor memory (blocks of 4 columns: row r's four scales in lane r % 32,
// column r / 32). Instruction descriptor: bits 7-9 and 10-12 the operand types (1: e2m1), 17-22 N >> 3,
// 23 the scale type (0: e4m3), 27-28 M >> 7.
constexpr uint32_t idesc_fp4(int N) { return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 27); }
__device__ __forceinline__ void umma_fp4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// A block of scales, 32 lanes x 16 bytes, from shared memory to the four quarters of tensor memory; runs
// in order with the MMAs that the same lane issues after it.
__device__ __forceinline__ void tmem_cp_scales(uint32_t t, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(t), "l"(desc) : "memory");
}
// One arrival for the warp, after every lane's preceding accesses.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// A warp waits for a barrier's phase: false when limit_ns has passed, or when another warp of the CTA has
// given up. A satisfied wait is one test (56 clocks; 86 with a sleep's bound); the rest is out of line
// and sleeps in the test, or with a bound below the sleep (a test of this path) polls.
__device__ __noinline__ bool warp_wait_long(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  bool got = true;
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, s;\n\t"
        "setp.ge.u64 s, %4, %3;\n\t"
        "@s mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@!s mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "n"(kSuspendHintNs), "l"(limit_ns)
        : "memory");
    if (done) break;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (*abort || t - t0 > limit_ns) {
      *abort = 1;
      got = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, got);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t wl) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (__all_sync(0xffffffffu, done)) return true;
  return warp_wait_long(smem_u32(bar), parity, abort, wl);
}
// Stage and parity of the tile ring.
template <int kStages>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      ph ^= 1;
    }
  }
};

template <int kGC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t a, uint32_t (&r)[kGC]) {
  if constexpr (kGC == 8) tmem_ld_32x32b_x8(a, r);
  else tmem_ld_32x32b_x16(a, r);
}
template <int kGC>
__device__ __forceinline__ void tmem_st_cols(uint32_t a, const uint32_t (&r)[kGC]) {
  if constexpr (kGC == 8) tmem_st_32x32b_x8(a, r);
  else tmem_st_32x32b_x16(a, r);
}

// kGC columns over the warp's lanes: lane l ends with column l % kGC's maximum or sum.
template <int kGC, bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[kGC], int lane) {
#pragma unroll
  for (int o = kGC / 2; o >= 1; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int q = 0; q < o; ++q) {
      const float keep = up ? v[q + o] : v[q], send = up ? v[q] : v[q + o];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      v[q] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  float x = v[0];
#pragma unroll
  for (int o = kGC; o < 32; o <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, x, o);
    x = kMax ? fmaxf(x, got) : x + got;
  }
  return x;
}

__device__ __forceinline__ void ldmatrix_t8_x2(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes x 16 columns (two groups of 8): thread t holds lane t / 4 (registers 0, 1 of a group of four)
// and t / 4 + 8 (registers 2, 3), columns 2 (t % 4) and the next.
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// What the scores of all rows share of their factor, softmax_scale log2(e) k_scale = m 2^e: with the exponents
// apart no part of the product leaves fp32's range where the whole (2^-shift of the row joins it) does not.
struct Factor {
  float m;
  int e;
  __device__ __forceinline__ Factor(float scale_log2, float kg) {
    int a, b;
    m = frexpf(scale_log2, &a) * frexpf(kg, &b);
    e = a + b;
  }
  // m 2^(e - shift) in two steps: the first stays normal (m is at least 1/4)
  __device__ __forceinline__ float row(int shift) const {
    const int t = min(max(e - shift, -240), 240), h = t >> 1;
    return m * __int_as_float((127 + h) << 23) * __int_as_float((127 + t - h) << 23);
  }
};
// A query row's terms and their scales into a Q buffer, and its factor: by one warp, a lane 8 elements (two
// lanes share a block of 16).
template <int kCols>
__device__ __noinline__ void quantize_q_row(uint4 raw, int row, uint8_t* buf, float* f, Factor shared) {
  using Gm = Geo<kCols>;
  const int lane = threadIdx.x & 31;
  const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t mx = 0;
#pragma unroll
  for (int x = 0; x < 4; ++x) mx = __vmaxu2(mx, rw[x] & 0x7fff7fffu);
  mx = max(mx & 0xffffu, mx >> 16);
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));  // of the block
  const uint32_t mr = __reduce_max_sync(0xffffffffu, mx);
  const int shift = min(135 - (int)(mr >> 7), 126);  // the row's largest to [2^8, 2^9)
  const float up = __int_as_float((127 + shift) << 23);
  int e = max((int)(__float_as_uint(__uint_as_float(mx << 16) * up) >> 23) - 127, -9);
  const float inv = __int_as_float((127 - e) << 23);
  float y[8];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    y[2 * x] = __uint_as_float(rw[x] << 16) * up * inv;
    y[2 * x + 1] = __uint_as_float(rw[x] & 0xffff0000u) * up * inv;
  }
  uint8_t* dst = buf + row * 128 + (((lane >> 2) ^ (row & 7)) * 16) + (lane & 3) * 4;
  // row n = row + kCols (t % kSide) of the turn t / kSide: lane n % 32, word n / 32 of the step's block
  uint8_t* sdst = buf + kTerms * Gm::kQTerm + (lane >> 3) * 512 + row * 16 + ((lane >> 1) & 3);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    *reinterpret_cast<uint32_t*>(dst + t * Gm::kQTerm) = e2m1x8_rn(y);
    const int n0 = t % Gm::kSide * kCols;
    if ((lane & 1) == 0)
      sdst[t / Gm::kSide * Gm::kQsTurn + n0 % 32 * 16 + n0 / 32 * 4] = (uint8_t)(e >= -6 ? (e + 7) << 3 : 1 << (e + 9));
    if (t == kTerms - 1) break;
    const int down = min(3, e + 9);
    const float next = __int_as_float((127 + down) << 23);
    e -= down;
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      constexpr float kHalves = 6291456.0f;  // 1.5 * 2^22: adding it leaves a multiple of one half
      float v0, v1;
      add2(v0, v1, y[x], y[x + 1], kHalves, kHalves);
      add2(v0, v1, v0, v1, -kHalves, -kHalves);
      add2(y[x], y[x + 1], y[x], y[x + 1], -v0, -v1);
      mul2(y[x], y[x + 1], y[x], y[x + 1], next, next);
    }
  }
  // rows with an infinity or NaN: a NaN factor makes their scores, and so the row, NaN
  if (lane == 0)
    f[row] = mr >= 0x7f80u ? __int_as_float(0x7fc00000) : shared.row(shift);
}

template <int kCols>
__global__ void __launch_bounds__(Geo<kCols>::kThreads, 1) spec_verify_fp4_kernel(const __grid_constant__ Params p) {
  using Gm = Geo<kCols>;
  constexpr int kGC = Gm::kGC, kThreads = Gm::kThreads, kKStages = Gm::kKStages, kVStages = Gm::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared<kCols>& sh = *reinterpret_cast<Shared<kCols>*>(smem + Gm::kTiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int line = blockIdx.x % p.lines, cta = blockIdx.x / p.lines;
  const int nq_max = p.tpc * p.group;
  const Workspace ws(p.ws, (int)gridDim.x);

  // ------------------------------------------------------------------ barriers, tensor memory, range
  if (warp == 2) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  const int live_groups = (nq_max + kGC - 1) / kGC;  // softmax warpgroups with a live column
  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 2);  // QK, K scales
      sh.k_armed[s] = 0;
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 9);  // V columns, V scales
      sh.v_armed[s] = 0;
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.q_ready[b], 2);
      mbar_init(&sh.q_ready[2 + b], 2);
      mbar_init(&sh.q_free[b], 1);
      mbar_init(&sh.ks_ready[b], 1);
      mbar_init(&sh.s_full[b], 1);
      mbar_init(&sh.s_free[b], 4 * live_groups);
      mbar_init(&sh.sf_ready[b], 1);
      mbar_init(&sh.sf_free[b], 8);
      mbar_init(&sh.vt_ready[b], 8);
      mbar_init(&sh.pv_done[b], 1);
      mbar_init(&sh.p_full[b], 4 * live_groups);
    }
    mbar_init(&sh.drain, 2);
    mbar_init(&sh.q_first, kThreads / 32 - 2);
    sh.abort = 0;
    sh.v_nan = 0;
    sh.r0 = -1;
    fence_mbar_init();
  }
  if (tid < kCols) {
    const int t = tid / p.group;
    sh.tok[tid] = t;
    sh.row_off[tid] = t * p.num_q_heads + (tid - t * p.group);
  }
  // Q: rows past the live ones count for nothing, but have to be numbers; P^T: its zero half stays zero
  for (int x = tid; x < Gm::kOffSf / 16; x += kThreads) reinterpret_cast<uint4*>(smem)[x] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  // The CTA's range of the line's tiles. A thread holds a request (kThreads of them at a time).
  auto tiles_of = [&](int r) -> int {
    const int len = r < p.num_reqs ? __ldg(p.seq_lens + r) : 0;
    return len > 0 ? (int)(((int64_t)len + kBN - 1) / kBN) : 0;
  };
  auto scan = [&](long long x, long long& sum) -> long long {  // inclusive over the CTA; two barriers
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh.wsum[warp] = x;
    __syncthreads();
    sum = 0;
#pragma unroll 8
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long y = sh.wsum[w];
      if (w < warp) x += y;
      sum += y;
    }
    return x;
  };
  tc_fence_before();
  int t_req = tiles_of(tid);
  long long sum, inc = scan(t_req, sum), total = sum;
  for (int base = kThreads; base < p.num_reqs; base += kThreads) {
    scan(tiles_of(base + tid), sum);
    total += sum;
  }
  tc_fence_after();
  // zeros for the rows of empty requests, each CTA its share of the requests
  for (int base = 0; base < p.num_reqs; base += kThreads) {
    const int r = base + tid;
    const bool empty = r < p.num_reqs && r % (int)gridDim.x == (int)blockIdx.x && (base ? tiles_of(r) : t_req) == 0;
    if (!__syncthreads_or(empty)) continue;
    for (int x = base; x < min(base + kThreads, p.num_reqs); ++x) {
      if (x % (int)gridDim.x != (int)blockIdx.x || tiles_of(x) != 0) continue;
      uint4* o = reinterpret_cast<uint4*>(p.out + (int64_t)x * p.T * p.num_q_heads * kFp4D);
      const int64_t n = (int64_t)p.T * p.num_q_heads * (kFp4D / 8);
      for (int64_t i = tid; i < n; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    }
  }
  const int64_t line_total = total * p.units;
  const int64_t begin = line_begin(line_total, cta, p.ctas), end = line_begin(line_total, cta + 1, p.ctas);
  if (begin < end) {  // the requests that hold the range's first and last tile
    long long before = 0;
    for (int base = 0;; base += kThreads) {
      if (base) {
        t_req = tiles_of(base + tid);
        inc = scan(t_req, sum);
      } else if (p.num_reqs > kThreads) {
        inc = scan(t_req, sum);
      }
      const long long at = (before + inc - t_req) * p.units, next = at + (long long)t_req * p.units;
      if (at <= begin && begin < next) {
        const int64_t x = begin - at;
        sh.r0 = base + tid;
        sh.u0 = p.units == 1 ? 0 : (int)(x / t_req);
        sh.t00 = (int)(x - (int64_t)sh.u0 * t_req);
      }
      if (at < end && end <= next) {
        // for the merge: does the unit of the last tile begin in this range and go on past it?
        const int64_t u = p.units == 1 ? 0 : (end - 1 - at) / t_req, unit_begin = at + u * t_req, unit_end = unit_begin + t_req;
        Note& note = ws.notes[blockIdx.x];
        note.r = base + tid;
        note.unit = p.lines > 1 ? line : (int)u;
        // its last CTA: the first whose range ends at or after the unit's end
        note.pieces = unit_begin >= begin && unit_end > end ? (int)((unit_end * p.ctas + line_total - 1) / line_total) - cta : 0;
      }
      before += sum;
      if (before * p.units >= end || base + kThreads >= p.num_reqs) break;  // CTA-uniform
    }
  } else {  // nothing to do (fewer tiles than CTAs): the merge may still pass by
    if (tid == 0) ws.notes[blockIdx.x].pieces = 0;
    if (tid < kMaxCols) ws.lm[(size_t)blockIdx.x * 2 * kMaxCols + tid].x = 0.0f;
  }
  __syncthreads();
  const Cursor start{sh.r0, sh.u0, sh.t00, sh.r0 >= 0 ? end - begin : 0};
  const uint32_t tmem = sh.tmem_base;
  volatile int* const abort = &sh.abort;
  const uint64_t wl = p.wait_limit_ns;
  const int G = p.seg;

  auto q_rows = [&](const Run& run, int unit) {  // the unit's first query row
    return reinterpret_cast<const uint4*>(p.q) +
           (((int64_t)run.r * p.T + (unit % p.n_tg) * p.tpc) * p.num_q_heads + (int64_t)(unit / p.n_tg) * p.group) * (kFp4D / 8);
  };
  if (warp != 0 && warp != 6) {
    Cursor cur = start;
    Run run;
    if (next_run(p, cur, run)) {
      const int unit = p.lines > 1 ? line : run.u;
      const int nq = min(p.tpc, p.T - (unit % p.n_tg) * p.tpc) * p.group;
      const uint4* base = q_rows(run, unit);
      const Factor factor(p.scale_log2, __ldg(p.k_scale));
      const int at = warp - (warp > 6 ? 2 : 1);  // 0 .. kThreads / 32 - 3
      if (at == 0 && lane >= nq && lane < kCols) sh.f[0][lane] = 0.0f;
#pragma unroll 1
      for (int row = at; row < nq; row += kThreads / 32 - 2)
        quantize_q_row<kCols>(__ldg(base + (int64_t)sh.row_off[row] * (kFp4D / 8) + lane), row, smem + Gm::kOffQ, sh.f[0], factor);
      fence_proxy_async_smem();
      warp_arrive(&sh.q_first, lane);
    }
  }

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------------------------ producers
    // Warp 0 K, warp 6 V, each through its own ring. Lane = key segment (G keys, inside one block). Each lane
    // walks its segment's place in the table a tile ahead of the copies, without divisions inside a run; one
    // elected lane issues the tile's copies. Few instructions a tile: this code runs once in a tile, so it
    // is fetched anew each time.
    const int nseg = kBN / G;
    const int q128 = kBN / p.block_size, r128 = kBN % p.block_size;
    Cursor cur = start;
    Run run;
    run.n = 0;
    int j = 0, key = 0, col = 0, slot = 0, kvh = 0;  // of the tile that is looked up
    const int32_t* table = nullptr;
    bool more = true;
    bool need = false;  // the segment has a key of the request
    // moves on to the next tile and reads its table entry (-1 past the table, as for any bad block)
    auto look_up = [&]() -> int {
      if (++j < run.n) {
        key += kBN;
        col += q128;
        slot += r128;
        if (slot >= p.block_size) {
          slot -= p.block_size;
          ++col;
        }
      } else {
        more = next_run(p, cur, run);
        if (!more) {
          need = false;
          return -1;
        }
        j = 0;
        kvh = (p.lines > 1 ? line : run.u) / p.n_tg;
        key = run.t0 * kBN + lane * G;
        col = key / p.block_size;
        slot = key - col * p.block_size;
        table = p.block_table + (int64_t)run.r * p.bt_stride;
      }
      need = lane < nseg && key < run.len;
      return need && col < p.max_blocks ? __ldg(table + col) : -1;
    };
    const bool is_k = warp == 0;
    uint64_t* const fulls = is_k ? sh.k_full : sh.v_full;
    uint64_t* const empties = is_k ? sh.k_empty : sh.v_empty;
    uint32_t* const bads = is_k ? sh.k_bad : sh.v_bad;
    uint32_t* const armed = is_k ? sh.k_armed : sh.v_armed;
    const int stages = is_k ? kKStages : kVStages;
    uint8_t* const base = smem + (is_k ? Gm::kOffK : Gm::kOffV);
    const CUtensorMap* const maps = &p.map[is_k ? 0 : 4];
    int blk = look_up();
    int st = 0;
    uint32_t ph = 1;  // parity of the stage's last release (none before its first use)
    bool first = true;
    while (more) {
      const int c_slot = slot, c_kvh = kvh;
      const bool c_need = need;
      int c_blk = blk;
      blk = look_up();
      uint64_t* full = &fulls[st];
      if (!first && !warp_wait(&empties[st], ph, abort, wl)) break;
      if ((int64_t)c_blk >= p.num_blocks) c_blk = -1;
      const uint32_t bad = __ballot_sync(0xffffffffu, c_need && c_blk < 0);
      const uint32_t live = __ballot_sync(0xffffffffu, c_blk >= 0);
      // one block holds the tile (segment 0 is live then, or bad)
      const bool big = p.big_ok && __shfl_sync(0xffffffffu, c_blk >= 0 && c_slot + kBN <= p.block_size, 0);
      uint8_t* stage = base + st * kStage;
      if (bad && lane == 0) record_error(p.dev_err, kErrDeviceBounds);
      if (lane == 0) {
        bads[st] = bad;
        const uint32_t rows = big ? (uint32_t)kBN : (uint32_t)(__popc(live) * G);
        mbar_arm_tx(full, rows * (uint32_t)(kFp4RowBytes + kFp4Groups), &armed[st]);
      }
      __syncwarp();
      if (big) {
        const int b0 = __shfl_sync(0xffffffffu, c_blk, 0), s0 = __shfl_sync(0xffffffffu, c_slot, 0);
        if (elect_one()) {
          tma_load_4d(stage, maps + 2, full, 0, c_kvh, s0, b0);
          tma_load_4d(stage + kCodeTile, maps + 3, full, 0, c_kvh, s0, b0);
        }
      } else {
        // segments in batches: their places by shuffles first, then one lane issues the batch's copies, 65
        // clocks each (a segment at a time: 136; one token, 32 requests of up to 16,384 keys in pages of 16: 67 us
        // against 79)
        constexpr int kBatch = 8;
#pragma unroll 1
        for (int g0 = 0; g0 < nseg; g0 += kBatch) {
          int sb[kBatch], ss[kBatch];
#pragma unroll
          for (int g = 0; g < kBatch; ++g) {
            sb[g] = __shfl_sync(0xffffffffu, c_blk, g0 + g);
            ss[g] = __shfl_sync(0xffffffffu, c_slot, g0 + g);
          }
          uint8_t* const codes = stage + g0 * G * kFp4RowBytes;
          uint8_t* const scales = stage + kCodeTile + g0 * G * kFp4Groups;
          if (elect_one()) {
#pragma unroll
            for (int g = 0; g < kBatch; ++g)
              if (sb[g] >= 0) {  // (negative past the tile's segments, and for a bad block)
                tma_load_4d(codes + g * G * kFp4RowBytes, maps, full, 0, c_kvh, ss[g], sb[g]);
                tma_load_4d(scales + g * G * kFp4Groups, maps + 1, full, 0, c_kvh, ss[g], sb[g]);
              }
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (++st == stages) {
        st = 0;
        ph ^= 1;
        first = false;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------ QK issuer
    // S^T = sum over the terms of K Q_term^T, kSide terms' columns side by side. The whole warp walks the
    // tiles and one elected lane issues: with a warp-uniform address stream the MMAs follow one another
    // at the tensor core's own rate; from inside a `lane == 0` branch each takes 45 clocks and more.
    constexpr uint32_t id = idesc_fp4(Gm::kSide * kCols);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t q_desc = smem_desc(smem_u32(smem + Gm::kOffQ), 16, 1024);
    const uint64_t qs_desc = smem_desc(smem_u32(smem + Gm::kOffQ + kTerms * Gm::kQTerm), 16, 128, 0);
    const uint64_t k_desc = smem_desc(smem_u32(smem + Gm::kOffK), 16, 1024);
    const uint64_t ks_desc = smem_desc(smem_u32(smem + Gm::kOffKs), 16, 128, 0);
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = true;
    Ring<kKStages> ring;
    for (int s = 0; ok && next_run(p, cur, run); ++s) {
      ok = warp_wait(&sh.q_ready[s & 3], (s >> 2) & 1, abort, wl);
      // the last run's MMAs are done with the scales in tensor memory
      if (ok && i > 0) ok = warp_wait(&sh.s_full[(i - 1) & 1], ((i - 1) >> 1) & 1, abort, wl);
      if (!ok) break;
      tc_fence_after();
      const uint64_t q_off = (uint64_t)((s & 1) * (Gm::kQBuf >> 4));
      if (elect_one()) {
#pragma unroll 1
        for (int x = 0; x < 4 * Gm::kTurns; ++x) tmem_cp_scales(tm + Gm::kColQs + 4 * x, qs_desc + q_off + (uint64_t)(x * 32));
      }
      __syncwarp();
      for (int j = 0; ok && j < run.n; ++j, ++i, ring.next()) {
        const int b = i & 1;
        // the last tile's MMAs are done with the K scales in tensor memory (long before the next ones are here)
        if (j > 0) ok = warp_wait(&sh.s_full[b ^ 1], ((i - 1) >> 1) & 1, abort, wl);
        // the K scales' warp has waited for the codes and for the softmax to be through with S^T_{i-2}
        if (ok) ok = warp_wait(&sh.ks_ready[b], (i >> 1) & 1, abort, wl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + Gm::kColS + b * Gm::kSBuf, sfa = tm + Gm::kColKs;
        const uint64_t kd = k_desc + (uint64_t)(ring.st * (kStage >> 4)), ksd = ks_desc + (uint64_t)(b * (kScaleTile >> 4));
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) tmem_cp_scales(sfa + 4 * ks, ksd + (uint64_t)(ks * 32));
#pragma unroll
          for (int t = 0; t < Gm::kTurns; ++t)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_fp4_ss(d, kd + (uint64_t)(ks * 2), q_desc + q_off + (uint64_t)(t * (Gm::kSide * Gm::kQTerm >> 4) + ks * 2), id,
                          sfa + 4 * ks, tm + Gm::kColQs + 16 * t + 4 * ks, (t | ks) ? 1u : 0u);
          umma_commit(&sh.s_full[b]);
          umma_commit(&sh.k_empty[ring.st]);
          if (j == run.n - 1) umma_commit(&sh.q_free[s & 1]);
        }
        __syncwarp();
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------------------ PV issuer
    constexpr uint32_t id = idesc_f16(128, 2 * kCols, false, false, true);
    const uint64_t p_desc = smem_desc(smem_u32(smem + Gm::kOffP), 0, 8 * Gm::kPRow, Gm::kPLayout);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = true;
    while (ok && next_run(p, cur, run)) {
      for (int j = 0; ok && j < run.n; ++j, ++i) {
        const int b = i & 1;
        ok = warp_wait(&sh.vt_ready[b], (i >> 1) & 1, abort, wl);
        if (ok) ok = warp_wait(&sh.p_full[b], (i >> 1) & 1, abort, wl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tm + Gm::kColV + b * 128;
        const uint64_t pd = p_desc + (uint64_t)((Gm::kPBufs == 2 ? b : 0) * (Gm::kPBuf >> 4));
        if (elect_one()) {
          // 16 steps of 8 keys, 16 rows of P^T (an even and an odd one a key)
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16_ts(tm + Gm::kColO, a + c * 32 + ks * 8, pd + (uint64_t)((4 * c + ks) * (16 * Gm::kPRow >> 4)), id,
                          (j | c | ks) ? 1u : 0u);
          umma_commit(&sh.pv_done[b]);
        }
        __syncwarp();
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------------------ V scales
    // Lane = four keys: their 4 x 16 e4m3 bytes as fp16, [quarter of the row][key quad][group][key]. Keys
    // past the request or in a bad block get 0. A NaN scale of a key that some columns of the CTA do not
    // see would reach them as 0 * NaN: it is left out here and put into the columns that see the key by
    // the epilogue.
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = true;
    Ring<kVStages> ring;
    while (ok && next_run(p, cur, run)) {
      const int unit = p.lines > 1 ? line : run.u;
      const int seen_by_all = run.len - p.T + (unit % p.n_tg) * p.tpc;  // the last such key
      for (int j = 0; ok && j < run.n; ++j, ++i, ring.next()) {
        const int st = ring.st, b = i & 1;
        ok = warp_wait(&sh.v_full[st], ring.ph, abort, wl);
        if (ok && i >= 2) ok = warp_wait(&sh.sf_free[b], ((i >> 1) - 1) & 1, abort, wl);
        if (!ok) break;
        const uint4* src = reinterpret_cast<const uint4*>(smem + Gm::kOffV + st * kStage + kCodeTile);
        uint32_t w[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = src[lane * 4 + k];
          w[k][0] = v.x; w[k][1] = v.y; w[k][2] = v.z; w[k][3] = v.w;
        }
        const int key0 = (run.t0 + j) * kBN;
        const uint32_t bad = sh.v_bad[st];
        if (bad || key0 + kBN > run.len || key0 + kBN - 1 > seen_by_all) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = lane * 4 + k;
            const bool dead = key0 + key >= run.len || ((bad >> (key / G)) & 1u), partly = key0 + key > seen_by_all;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (dead) w[k][q] = 0;
              const uint32_t nan = partly ? __vcmpeq4(w[k][q] & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
              if (nan) {
                w[k][q] &= ~nan;
                sh.v_nan = 1;
              }
            }
          }
        }
        uint8_t* dst = smem + Gm::kOffSf + b * Gm::kSfBuf + lane * 32;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t lo01 = __byte_perm(w[0][q], w[1][q], 0x5140), hi01 = __byte_perm(w[0][q], w[1][q], 0x7362);
          const uint32_t lo23 = __byte_perm(w[2][q], w[3][q], 0x5140), hi23 = __byte_perm(w[2][q], w[3][q], 0x7362);
          uint4* d = reinterpret_cast<uint4*>(dst + q * 1024);
          d[0] = make_uint4(e4m3x2_to_f16x2((uint16_t)lo01), e4m3x2_to_f16x2((uint16_t)lo23),
                            e4m3x2_to_f16x2((uint16_t)(lo01 >> 16)), e4m3x2_to_f16x2((uint16_t)(lo23 >> 16)));
          d[1] = make_uint4(e4m3x2_to_f16x2((uint16_t)hi01), e4m3x2_to_f16x2((uint16_t)hi23),
                            e4m3x2_to_f16x2((uint16_t)(hi01 >> 16)), e4m3x2_to_f16x2((uint16_t)(hi23 >> 16)));
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.v_empty[st]);
          mbar_arrive(&sh.sf_ready[b]);
        }
      }
    }
  } else if (warp == 7) {
    // ------------------------------------------------------------------------------ K scales
    // The four scale words of a key go to the blocks of the four steps of 64 elements, lane = key % 32.
    // Keys past the request or in a bad block get 0 (their codes are whatever the stage held).
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = true;
    Ring<kKStages> ring;
    while (ok && next_run(p, cur, run)) {
      for (int j = 0; ok && j < run.n; ++j, ++i, ring.next()) {
        const int st = ring.st, b = i & 1;
        ok = warp_wait(&sh.k_full[st], ring.ph, abort, wl);
        // S^T_{i-2} has been read, so QK_{i-2} is done with its scales, and QK_i may overwrite S^T
        if (ok && i >= 2) ok = warp_wait(&sh.s_free[b], ((i >> 1) - 1) & 1, abort, wl);
        if (!ok) break;
        const uint4* src = reinterpret_cast<const uint4*>(smem + Gm::kOffK + st * kStage + kCodeTile) + lane;
        uint4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = src[32 * x];
        const int key0 = (run.t0 + j) * kBN + lane;
        const uint32_t bad = sh.k_bad[st];
        if (bad || key0 - lane + kBN > run.len) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (key0 + 32 * x >= run.len || ((bad >> ((lane + 32 * x) / G)) & 1u)) v[x] = make_uint4(0, 0, 0, 0);
        }
        uint4* dst = reinterpret_cast<uint4*>(smem + Gm::kOffKs + b * kScaleTile) + lane;
        dst[0] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
        dst[32] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
        dst[64] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
        dst[96] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.ks_ready[b]);
          mbar_arrive(&sh.k_empty[st]);
        }
      }
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------------------------ Q
    // The terms of Q for a run, a run ahead of its use; a warp takes every other row and has the next one's
    // load in flight. The first run's rows were spread over all warps but the producers.
    const Factor factor(p.scale_log2, __ldg(p.k_scale));
    Cursor cur = start;
    Run run;
    bool ok = true;
    for (int s = 0; ok && next_run(p, cur, run); ++s) {
      if (s == 0) {
        ok = warp_wait(&sh.q_first, 0, abort, wl);
      } else {
        const int unit = p.lines > 1 ? line : run.u;
        const int t_base = (unit % p.n_tg) * p.tpc;
        const int nq = min(p.tpc, p.T - t_base) * p.group;
        const uint4* base = q_rows(run, unit);
        auto fetch = [&](int row) { return row < nq ? __ldg(base + (int64_t)sh.row_off[row] * (kFp4D / 8) + lane) : make_uint4(0, 0, 0, 0); };
        if (s >= 2) ok = warp_wait(&sh.q_free[s & 1], ((s >> 1) - 1) & 1, abort, wl);
        if (!ok) break;
        if (warp == 4 && lane >= nq && lane < kCols) sh.f[s & 7][lane] = 0.0f;
        uint4 raw = fetch(warp - 4);
#pragma unroll 1
        for (int row = warp - 4; row < nq; row += 2) {
          const uint4 next = fetch(row + 2);
          quantize_q_row<kCols>(raw, row, smem + Gm::kOffQ + (s & 1) * Gm::kQBuf, sh.f[s & 7], factor);
          raw = next;
        }
        fence_proxy_async_smem();
      }
      if (ok) warp_arrive(&sh.q_ready[s & 3], lane);
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------------------------ V columns
    // A warp's tensor-memory lanes are 32 of a row's 128 code bytes (a lane is a byte: an even and an odd
    // element), its columns 64 of the tile's keys. ldmatrix hands a thread one byte column of four keys;
    // a key's column holds the converted pair (even, odd), which is what a conversion of the byte gives.
    // The columns of 16 keys are in the order 0 1 4 5 8 9 12 13, 2 3 6 7 10 11 14 15 (that of the store).
    const int quarter = warp & 3, hh = (warp - 8) >> 2;
    const uint32_t tv0 = tmem + ((uint32_t)(quarter * 32) << 16) + Gm::kColV + hh * 64;
    const int key = hh * 64 + (lane & 15);
    const uint32_t row = key * 128 + (((2 * quarter + (lane >> 4)) ^ (key & 7)) * 16);  // lanes 16-31: the second 16 bytes
    const uint32_t codes0 = smem_u32(smem + Gm::kOffV) + row;
    const uint8_t* sf0 = smem + Gm::kOffSf + quarter * 1024 + hh * 512 + (lane & 3) * 32;
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = true;
    Ring<kVStages> ring;
    while (ok && next_run(p, cur, run)) {
      for (int j = 0; ok && j < run.n; ++j, ++i, ring.next()) {
        const int st = ring.st, b = i & 1;
        ok = warp_wait(&sh.sf_ready[b], (i >> 1) & 1, abort, wl);  // the scales' warp has waited for the codes
        if (ok && i >= 2) ok = warp_wait(&sh.pv_done[b], ((i >> 1) - 1) & 1, abort, wl);  // the V tile's place is read
        if (!ok) break;
        tc_fence_after();
        const uint32_t codes = codes0 + st * kStage, tv = tv0 + b * 128;
        const uint8_t* sf = sf0 + b * Gm::kSfBuf;
        // 16 keys a step; the next step's codes and scales are read before this one's are converted
        uint32_t w[2][4];
        uint4 s4[2][2];
        auto read = [&](int kb, int to) {
          ldmatrix_t8_x2(codes + kb * 16 * 128, w[to]);
          s4[to][0] = *reinterpret_cast<const uint4*>(sf + kb * 128);
          s4[to][1] = *reinterpret_cast<const uint4*>(sf + kb * 128 + 16);
        };
        read(0, 0);
#pragma unroll 1
        for (int kb2 = 0; kb2 < 4; kb2 += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kb = kb2 + h;
            read(h ? (kb2 + 2) & 3 : kb + 1, h ^ 1);  // (the last one's is not used)
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // 16 bytes: two groups, eight bytes each
              uint32_t o[8];
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint32_t v[4];
                e2m1x8_to_f16(w[h][2 * x + g], v);
                const uint32_t s01 = g ? s4[h][x].z : s4[h][x].x, s23 = g ? s4[h][x].w : s4[h][x].y;
                const __half2 h01 = *reinterpret_cast<const __half2*>(&s01), h23 = *reinterpret_cast<const __half2*>(&s23);
                const __half2 d[4] = {__low2half2(h01), __high2half2(h01), __low2half2(h23), __high2half2(h23)};
                o[2 * g] = hmul2_u32(v[0], *reinterpret_cast<const uint32_t*>(&d[0]));
                o[2 * g + 1] = hmul2_u32(v[1], *reinterpret_cast<const uint32_t*>(&d[1]));
                o[4 + 2 * g] = hmul2_u32(v[2], *reinterpret_cast<const uint32_t*>(&d[2]));
                o[4 + 2 * g + 1] = hmul2_u32(v[3], *reinterpret_cast<const uint32_t*>(&d[3]));
              }
              tmem_st_16x256b_x2(tv + ((uint32_t)(16 * x) << 16) + kb * 16, o);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.vt_ready[b]);
          mbar_arrive(&sh.v_empty[st]);
          mbar_arrive(&sh.sf_free[b]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------------------ softmax
    const int grp = (warp - 16) >> 2;
    const int c0 = grp * kGC;
    const int quarter = warp & 3;
    const int k = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int bar_id = 1 + grp;
    // the key's two rows of P^T (see V columns for the order of the keys): weights in the first kCols
    // columns of the first row, which meets the even elements, and in the last of the second
    const int prow = 2 * ((k & ~15) + ((k >> 1) & 1) * 8 + ((k & 15) >> 2) * 2 + (k & 1));
    // byte offsets of the group's chunks of 8 columns in the two rows; both get the same weights, and every
    // other pair of keys writes its second row first, so that a store's 8 lanes meet 8 bank groups
    uint32_t p_off[2][kGC / 8];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int cc = 0; cc < kGC / 8; ++cc) {
        const uint32_t odd = x ^ ((k >> 1) & 1), r = prow + odd, chunk = odd * (kCols / 8) + grp * (kGC / 8) + cc;
        p_off[x][cc] = r * Gm::kPRow + ((chunk ^ (kCols == 16 ? (r >> 1) & 3u : r & 7u)) * 16);
      }
    auto load_scores = [&](uint32_t t, float (&x)[kGC]) {  // the terms side by side, added
#pragma unroll
      for (int q = 0; q < kGC; q += 8) {
        uint32_t u[Gm::kSide][8];
#pragma unroll
        for (int h = 0; h < Gm::kSide; ++h) tmem_ld_32x32b_x8(t + h * kCols + q, u[h]);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 8; y += 2) {
          add2(x[q + y], x[q + y + 1], __uint_as_float(u[0][y]), __uint_as_float(u[0][y + 1]), __uint_as_float(u[1][y]),
               __uint_as_float(u[1][y + 1]));
#pragma unroll
          for (int h = 2; h < Gm::kSide; ++h)
            add2(x[q + y], x[q + y + 1], x[q + y], x[q + y + 1], __uint_as_float(u[h][y]), __uint_as_float(u[h][y + 1]));
        }
      }
    };
    Cursor cur = start;
    Run run;
    int i = 0;
    bool ok = c0 < nq_max;  // a group without a live column has nothing to do
    for (int s = 0; ok && next_run(p, cur, run); ++s) {
      const int unit = p.lines > 1 ? line : run.u;
      const int t_base = (unit % p.n_tg) * p.tpc;
      const int nq = min(p.tpc, p.T - t_base) * p.group;
      const int seen_by_all = run.len - p.T + t_base;  // token t_base's position: the last key every column sees
      ok = warp_wait(&sh.q_ready[s & 3], (s >> 2) & 1, abort, wl);
      const float* f = sh.f[s & 7] + c0;
      float* m = sh.m + c0;
      float l[kGC];
#pragma unroll
      for (int q = 0; q < kGC; ++q) l[q] = 0.0f;
      if (k < kGC) m[k] = -kUnset;
      group_sync(bar_id);
      for (int j = 0; j < run.n; ++j, ++i) {
        const int b = i & 1;
        const int past = (run.t0 + j) * kBN + k - seen_by_all;  // tokens from here on do see the key
        const bool masked = (run.t0 + j) * kBN + kBN - 1 > seen_by_all;
        if (ok) ok = warp_wait(&sh.s_full[b], (i >> 1) & 1, abort, wl);
        float x[kGC];
        float tile_sum[2];
        const uint32_t ts = tmem + lane_off + Gm::kColS + b * Gm::kSBuf + c0;
        for (int pass = 0;; ++pass) {
          // weights 2^(S f - m), 0 where the column does not see the key. One that passes 2^15 shows in
          // their sum (no weight is negative; the sum's pipe has room where the maximum's has none).
          bool over = false;
          if (ok) {
            tc_fence_after();
            load_scores(ts, x);
#pragma unroll
            for (int q = 0; q < kGC; q += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(f + q);
              const float4 m4 = *reinterpret_cast<const float4*>(m + q);
              fma2(x[q], x[q + 1], x[q], x[q + 1], f4.x, f4.y, m4.x, m4.y);
              fma2(x[q + 2], x[q + 3], x[q + 2], x[q + 3], f4.z, f4.w, m4.z, m4.w);
            }
            if (masked) {
#pragma unroll
              for (int q = 0; q < kGC; ++q)
                if (past > sh.tok[c0 + q]) x[q] = -INFINITY;
            }
            if (pass == 1) {  // past 2^9 only by the rounding of scores of 2^24 and more
#pragma unroll
              for (int q = 0; q < kGC; ++q) x[q] = x[q] > 9.0f ? 9.0f : x[q];
            }
#pragma unroll
            for (int q = 0; q < kGC; ++q) x[q] = ex2_approx(x[q]);
            tile_sum[0] = x[0];
            tile_sum[1] = x[1];
#pragma unroll
            for (int q = 2; q < kGC; q += 2) add2(tile_sum[0], tile_sum[1], tile_sum[0], tile_sum[1], x[q], x[q + 1]);
            over = !(tile_sum[0] + tile_sum[1] <= kMove);  // (a NaN column hides nothing)
          }
          if (pass == 1 || !group_any(bar_id, over)) break;
          // some column's maximum moves (always so in a run's first tile): exact maxima of this tile
          float alpha = 1.0f, m_new = 0.0f;
          if (ok) {
            load_scores(ts, x);
#pragma unroll
            for (int q = 0; q < kGC; ++q) {
              x[q] *= f[q];
              if (masked && past > sh.tok[c0 + q]) x[q] = -INFINITY;
            }
          }
          {
            const float mine_max = reduce_columns<kGC, true>(x, lane);
            if (lane < kGC) sh.red[grp][quarter][lane] = mine_max;
          }
          group_sync(bar_id);
          const int cl = lane & (kGC - 1);
          {
            const float cmax = fmaxf(fmaxf(sh.red[grp][0][cl], sh.red[grp][1][cl]),
                                     fmaxf(sh.red[grp][2][cl], sh.red[grp][3][cl]));
            const float m_old = -m[cl];
            m_new = m_old;
            if (cmax - m_old > kStart) {
              m_new = cmax - kStart;
              alpha = ex2_approx(m_old - m_new);
            }
          }
          group_sync(bar_id);
          if (quarter == 0 && lane < kGC) m[lane] = -m_new;
          group_sync(bar_id);
#pragma unroll
          for (int q = 0; q < kGC; ++q) l[q] *= __shfl_sync(0xffffffffu, alpha, q);
          if (j > 0) {
            if (ok) ok = warp_wait(&sh.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort, wl);
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[kGC];
                tmem_ld_cols<kGC>(tmem + lane_off + Gm::kColO + hh * kCols + c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < kGC; ++q)
                  v[q] = __float_as_uint(__uint_as_float(v[q]) * __shfl_sync(0xffffffffu, alpha, q));
                tmem_st_cols<kGC>(tmem + lane_off + Gm::kColO + hh * kCols + c0, v);
              }
              tmem_wait_st();
            }
          }
        }
        tc_fence_before();
        if (ok) warp_arrive(&sh.s_free[b], lane);
        {  // the P^T buffer has been read
          const int last = i - Gm::kPBufs;
          if (ok && last >= 0) ok = warp_wait(&sh.pv_done[last & 1], (last >> 1) & 1, abort, wl);
        }
#pragma unroll
        for (int q = 0; q < kGC; q += 2) add2(l[q], l[q + 1], l[q], l[q + 1], x[q], x[q + 1]);
        if (ok) {
          uint8_t* pb = smem + Gm::kOffP + (Gm::kPBufs == 2 ? b : 0) * Gm::kPBuf;
#pragma unroll
          for (int cc = 0; cc < kGC / 8; ++cc) {
            const uint4 w = make_uint4(pack_f16x2(x[8 * cc], x[8 * cc + 1]), pack_f16x2(x[8 * cc + 2], x[8 * cc + 3]),
                                       pack_f16x2(x[8 * cc + 4], x[8 * cc + 5]), pack_f16x2(x[8 * cc + 6], x[8 * cc + 7]));
            *reinterpret_cast<uint4*>(pb + p_off[0][cc]) = w;
            *reinterpret_cast<uint4*>(pb + p_off[1][cc]) = w;
          }
          fence_proxy_async_smem();
          tc_fence_before();
          warp_arrive(&sh.p_full[b], lane);
        }
      }
      // the segment's sums and O
      if (ok) ok = warp_wait(&sh.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort, wl);
      const bool whole = run.n == run.tiles;
      const size_t slot = (size_t)blockIdx.x * 2 + (run.t0 > 0 ? 0 : 1);
      {
        const float part = reduce_columns<kGC, false>(l, lane);
        if (lane < kGC) sh.red[grp][quarter][lane] = part;
      }
      group_sync(bar_id);
      if (quarter == 0 && lane < kGC) {
        const float sum = sh.red[grp][0][lane] + sh.red[grp][1][lane] + sh.red[grp][2][lane] + sh.red[grp][3][lane];
        sh.fin[c0 + lane] = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (!whole && ok) {
          ws.lm[slot * kMaxCols + c0 + lane] = make_float2(sum, -m[lane]);
        }
      }
      group_sync(bar_id);
      if (ok) {
        tc_fence_after();
        const bool nan = sh.v_nan != 0;
        const float vg = __ldg(p.v_scale);
        const int kvh = unit / p.n_tg;
        const int64_t row0 = ((int64_t)run.r * p.T + t_base) * p.num_q_heads + (int64_t)kvh * p.group;
        const int d = 2 * k;  // this lane's even element
#pragma unroll 1
        for (int cq = c0; cq < c0 + kGC; cq += 8) {
          uint32_t v[8], w[8];
          tmem_ld_32x32b_x8(tmem + lane_off + Gm::kColO + cq, v);
          tmem_ld_32x32b_x8(tmem + lane_off + Gm::kColO + kCols + cq, w);
          tmem_wait_ld();
          if (nan) {  // keys that only some columns see, with a NaN V scale
            // (no column sees the keys from seen_by_all + tpc on)
            const int last = min(min(run.len, seen_by_all + p.tpc), (run.t0 + run.n) * kBN);
            for (int key = max(seen_by_all + 1, run.t0 * kBN); key < last; ++key) {
              const int col = key / p.block_size;
              const int64_t blk = col < p.max_blocks ? (int64_t)__ldg(p.block_table + (int64_t)run.r * p.bt_stride + col) : -1;
              if (blk < 0 || blk >= p.num_blocks) continue;
              const uint8_t sb = __ldg(p.v_bscale + blk * p.scale_stride_blk + (key % p.block_size) * p.scale_stride_tok +
                                       (int64_t)kvh * p.scale_stride_head + d / kFp4Group);
              if ((sb & 0x7f) != 0x7f) continue;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (key - seen_by_all <= sh.tok[cq + q]) v[q] = w[q] = 0x7fc00000u;
            }
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = cq + q;
            if (c >= nq) break;
            const float x0 = __uint_as_float(v[q]), x1 = __uint_as_float(w[q]);
            if (whole)
              // v_scale last: 1 / sum is normal, v_scale / sum need not be
              reinterpret_cast<uint32_t*>(p.out + (row0 + sh.row_off[c]) * kFp4D)[k] =
                  pack_bf16x2(x0 * sh.fin[c] * vg, x1 * sh.fin[c] * vg);
            else
              reinterpret_cast<float2*>(ws.o + (slot * nq_max + c) * kFp4D)[k] = make_float2(x0, x1);
          }
        }
        tc_fence_before();
      }
      // m, red and fin are read; the group's four warps go on or stop together (their barriers stay paired)
      ok = !group_any(bar_id, !ok);
    }
  }

  tc_fence_before();
  const bool gave_up = __syncthreads_or(*abort != 0);
  if (gave_up) {
    // before the tensor memory is freed: wait for the copies of every armed phase and every MMA issued
    if (tid == 0) {
      for (int s = 0; s < kKStages; ++s) drain_armed(&sh.k_full[s], sh.k_armed[s]);
      for (int s = 0; s < kVStages; ++s) drain_armed(&sh.v_full[s], sh.v_armed[s]);
    }
    if ((warp == 1 || warp == 2) && elect_one()) {  // (the lane that issued)
      umma_commit(&sh.drain);
      mbar_wait_drain(&sh.drain, 0);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && gave_up) record_error(p.dev_err, kErrTimeout);
}

// ------------------------------------------------------------------------------------------
// merge of the pieces of a unit that several CTAs worked on
// ------------------------------------------------------------------------------------------
// Block (b, y): CTA b's note says whether a unit began in its range and went on; kP * kH warps a column, each
// every kP-th piece and one of kH parts of the row, add its pieces up: M = max m, out = v_scale (sum 2^(m - M) O
// / sum 2^(m - M) l). The first pieces are loaded before their weights are known; a piece without a key
// (l = 0: its range is empty, or the column sees none of its keys) may hold anything and counts as
// nothing.
template <int kP, int kH>
__global__ void __launch_bounds__(256, 4)
    spec_verify_fp4_merge_kernel(const Workspace ws, int32_t lines, int32_t T, int32_t group, int32_t num_q_heads,
                                 int32_t tpc, int32_t n_tg, const float* __restrict__ v_scale,
                                 __nv_bfloat16* __restrict__ out) {
  constexpr int kCol = 8 / (kP * kH), kF = 2 / kH, kBatch = 4;  // columns; float4 a lane; pieces in flight
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The workspace is the preceding grid's output, so it takes plain loads, which stay behind the wait; the
  // read-only path is for what no grid writes while this one is there.
  const int4 note = *reinterpret_cast<const int4*>(ws.notes + blockIdx.x);
  const int pieces = note.x, unit = note.z;
  if (pieces == 0) return;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % (kP * kH), c = (threadIdx.x >> 5) / (kP * kH);
  const int first = kH == 2 ? 0 : w, part_of_row = kH == 2 ? w : 0;
  const int cols = tpc * group, y = blockIdx.y * kCol + c, col = min(y, cols - 1);
  // piece i > 0 is slot 0 of the i-th CTA after this one in the line
  auto slot = [&](int i) -> size_t { return i == 0 ? (size_t)blockIdx.x * 2 + 1 : ((size_t)blockIdx.x + (size_t)i * lines) * 2; };
  auto load_lm = [&](int i) { return i < pieces ? ws.lm[slot(i) * kMaxCols + col] : make_float2(0, 0); };
  float4 o[kBatch][kF];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = base + first + kP * i;
      const float4* src = reinterpret_cast<const float4*>(ws.o + (slot(at) * cols + col) * kFp4D) + part_of_row * 32 + lane;
#pragma unroll
      for (int h = 0; h < kF; ++h) o[i][h] = at < pieces ? src[32 * h] : make_float4(0, 0, 0, 0);
    }
  };
  const float2 lm0 = load_lm(lane);
  load(0);
  float M = lm0.x != 0.0f ? lm0.y : -INFINITY;
  for (int i = 32 + lane; i < pieces; i += 32) {
    const float2 lm = load_lm(i);
    if (lm.x != 0.0f) M = fmaxf(M, lm.y);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float4 acc[kF];
#pragma unroll
  for (int h = 0; h < kF; ++h) acc[h] = make_float4(0, 0, 0, 0);
  float L = 0.0f;
  for (int base = 0; base < pieces; base += 32) {  // lane = piece
    const float2 lm = base == 0 ? lm0 : load_lm(base + lane);
    const float weight = lm.x != 0.0f ? exp2f(lm.y - M) : 0.0f;
    const uint32_t live = __ballot_sync(0xffffffffu, lm.x != 0.0f);
    float wl = weight * lm.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, x);
    L += wl;
    for (int b = base; b < min(base + 32, pieces); b += kP * kBatch) {
      if (b > 0) load(b);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = b - base + first + kP * i;
        const float wi = __shfl_sync(0xffffffffu, weight, at);
        const bool counts = (live >> at) & 1u;
#pragma unroll
        for (int h = 0; h < kF; ++h) {
          acc[h].x += counts ? wi * o[i][h].x : 0.0f;
          acc[h].y += counts ? wi * o[i][h].y : 0.0f;
          acc[h].z += counts ? wi * o[i][h].z : 0.0f;
          acc[h].w += counts ? wi * o[i][h].w : 0.0f;
        }
      }
    }
  }
  float4 sum = acc[0];
  int e = part_of_row * 32 + lane;  // this thread's four elements
  if constexpr (kP > 1) {
    static_assert(kP == 4 && kH == 1, "a warp finishes a quarter of the row, half its lanes at work");
    __shared__ float4 part[kCol][kP][64];
    part[c][w][lane] = acc[0];
    part[c][w][32 + lane] = acc[1];
    __syncthreads();
    if (lane >= 16) return;
    e = w * 16 + lane;
    sum = part[c][0][e];
#pragma unroll
    for (int x = 1; x < kP; ++x) {
      const float4 v = part[c][x][e];
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
  }
  const int t_base = (unit % n_tg) * tpc;
  if (y >= min(tpc, T - t_base) * group) return;
  const float f = L == 0.0f ? 0.0f : 1.0f / L, vg = __ldg(v_scale);  // (v_scale / L need not be normal)
  const int t = t_base + col / group;
  const int64_t row = ((int64_t)note.y * T + t) * num_q_heads + (int64_t)(unit / n_tg) * group + col % group;
  reinterpret_cast<uint2*>(out + row * kFp4D)[e] =
      make_uint2(pack_bf16x2(sum.x * f * vg, sum.y * f * vg), pack_bf16x2(sum.z * f * vg, sum.w * f * vg));
}

template <int kCols>
pkv_status launch(const Params& p, cudaStream_t st) {
  constexpr int kSmem = 1024 + Geo<kCols>::kTiles + (int)sizeof(Shared<kCols>);
  static_assert(kSmem <= 227 * 1024, "dynamic shared memory of one CTA");
  static std::atomic<uint64_t> attr_done{0};
  once_per_device(attr_done, [] {
    cudaFuncSetAttribute(spec_verify_fp4_kernel<kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  const unsigned grid = (unsigned)(p.ctas * p.lines);
  spec_verify_fp4_kernel<kCols><<<grid, Geo<kCols>::kThreads, kSmem, st>>>(p);
  pkv_status s = check_launch("spec_verify_attn_fp4");
  if (s != PKV_OK) return s;
  cudaLaunchConfig_t cfg = {};
  // Four warps over a column's pieces where units have more than four of them on average (one token over
  // 262,144 keys, 38 pieces: 62.6 us the whole call, 65 with two over the row's halves; over 1,024 keys, 8 pieces: 15.0
  // and 15.9); else two over the halves, since the blocks, nearly all of them with work, then go through the
  // SMs in several turns (eight tokens over 32 requests of up to 40,960: 209 us; 213 with four over the pieces).
  const bool many = grid > 4ll * p.num_reqs * p.lines * p.units;
  cfg.gridDim = dim3(grid, (unsigned)((p.tpc * p.group * (many ? 4 : 2) + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, many ? spec_verify_fp4_merge_kernel<4, 1> : spec_verify_fp4_merge_kernel<1, 2>,
                     Workspace(p.ws, (int)grid), p.lines, p.T, p.group, p.num_q_heads, p.tpc, p.n_tg, p.v_scale, p.out);
  return check_launch("spec_verify_attn_fp4 (merge)");
}

}  // namespace

}  // namespace pkv

extern "C" size_t pkv_spec_verify_fp4_workspace_bytes(int32_t num_ctas) {
  return num_ctas > 0 ? (size_t)num_ctas * pkv::kWorkspaceOfCta : 0;
}

extern "C" pkv_status pkv_spec_verify_attn_fp4(
    const void* q, const uint8_t* k_fp4, const uint8_t* v_fp4, const uint8_t* k_bscale, const uint8_t* v_bscale,
    const float* k_scale, const float* v_scale, int64_t num_blocks, int64_t stride_blk, int64_t stride_tok,
    int64_t stride_head, int64_t scale_stride_blk, int64_t scale_stride_tok, int64_t scale_stride_head,
    const int32_t* block_table, int64_t bt_stride, int32_t max_blocks, const int32_t* seq_lens, int32_t num_reqs,
    int32_t T, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float softmax_scale,
    void* out, void* workspace, int64_t workspace_bytes, int32_t* dev_err, void* stream) {
  using namespace pkv;
  constexpr const char* name = "spec_verify_attn_fp4";
  clear_error();
  PKV_UNSUP(head_dim == kFp4D, "%s: head_dim must be 256 (got %d)", name, head_dim);
  if (num_reqs == 0) return PKV_OK;  // nothing to do, nothing read
  PKV_ARG(q && k_fp4 && v_fp4 && k_bscale && v_bscale && k_scale && v_scale && block_table && seq_lens && out &&
              workspace,
          "%s: null pointer argument", name);
  PKV_ARG(num_reqs > 0 && T > 0 && num_q_heads > 0 && num_kv_heads > 0 && num_blocks > 0 && block_size > 0 &&
              max_blocks > 0 && bt_stride >= max_blocks,
          "%s: bad size argument", name);
  PKV_UNSUP(num_q_heads % num_kv_heads == 0, "%s: num_q_heads %% num_kv_heads != 0", name);
  const int group = num_q_heads / num_kv_heads;
  PKV_UNSUP(group <= kMaxCols, "%s: num_q_heads / num_kv_heads must be at most %d (got %d)", name, kMaxCols, group);
  PKV_UNSUP(block_size % 8 == 0, "%s: block_size must be a multiple of 8", name);
  // (positions of a whole last tile stay below 2^31)
  PKV_UNSUP((int64_t)max_blocks * block_size <= (1ll << 31) - kBN, "%s: the table's columns reach past 2^31 - %d positions",
            name, kBN);
  PKV_ARG(stride_blk > 0 && stride_tok > 0 && stride_head > 0 && scale_stride_blk > 0 && scale_stride_tok > 0 &&
              scale_stride_head > 0,
          "%s: strides must be positive", name);
  PKV_ARG(aligned16(q) && aligned16(out) && aligned16(workspace) && aligned16(k_fp4) && aligned16(v_fp4) &&
              aligned16(k_bscale) && aligned16(v_bscale) && stride_blk % 16 == 0 && stride_tok % 16 == 0 &&
              stride_head % 16 == 0 && scale_stride_blk % 16 == 0 && scale_stride_tok % 16 == 0 &&
              scale_stride_head % 16 == 0,
          "%s: q, out, workspace, caches, scale caches and their strides must be 16-byte aligned", name);
  PKV_ARG(softmax_scale > 0.0f, "%s: softmax_scale must be positive", name);
  PKV_ARG(workspace_bytes >= (int64_t)kWorkspaceOfCta, "%s: the workspace needs at least %zu bytes", name, kWorkspaceOfCta);
  Params p{};
  // columns of a CTA: 16 when a KV head's query rows fit (half the padding, and half the softmax: one
  // token over 32 requests of up to 16,384: 67 us against 79 with 32, over one of 262,144: 63 against 78),
  // else 32, the tokens spread over column groups that read the same keys
  const bool narrow = (int64_t)T * group <= 16;
  p.tpc = T < kMaxCols / group ? T : kMaxCols / group;
  p.n_tg = (int32_t)(((int64_t)T + p.tpc - 1) / p.tpc);
  const int64_t units = (int64_t)num_kv_heads * p.n_tg;
  PKV_ARG(units < (1ll << 31) && (int64_t)num_reqs * T * num_q_heads < (1ll << 40), "%s: too many query rows", name);
  // one line per unit (the heads of a request side by side) where that keeps nine tenths of the SMs busy,
  // (eight tokens over 32 requests of up to 40,960: 209 us against 235 in one line, whose CTAs read a page's
  // heads at different times), else one line with the units one after the other and no SM idle
  int64_t ctas = workspace_bytes / (int64_t)kWorkspaceOfCta;
  if (ctas > num_sms()) ctas = num_sms();
  const bool side = units <= ctas && ctas / units * units * 10 >= ctas * 9;
  p.lines = side ? (int)units : 1;
  p.units = side ? 1 : (int)units;
  p.ctas = (int)(ctas / p.lines);
  const int G = std::gcd(block_size, kBN);
  const uint64_t cdims[4] = {(uint64_t)kFp4RowBytes, (uint64_t)num_kv_heads, (uint64_t)block_size, (uint64_t)num_blocks};
  const uint64_t cstr[3] = {(uint64_t)stride_head, (uint64_t)stride_tok, (uint64_t)stride_blk};
  const uint64_t sdims[4] = {(uint64_t)kFp4Groups, (uint64_t)num_kv_heads, (uint64_t)block_size, (uint64_t)num_blocks};
  const uint64_t sstr[3] = {(uint64_t)scale_stride_head, (uint64_t)scale_stride_tok, (uint64_t)scale_stride_blk};
  p.big_ok = block_size >= kBN;
  const void* const bases[4] = {k_fp4, k_bscale, v_fp4, v_bscale};
  const char* const names[4] = {"k_fp4", "k_bscale", "v_fp4", "v_bscale"};
  for (int i = 0; i < 8; ++i) {
    const bool scales = i & 1, big = i & 2;
    if (big && !p.big_ok) continue;
    const int t = (i >> 2) * 2 + (scales ? 1 : 0);
    const uint32_t box[4] = {(uint32_t)(scales ? kFp4Groups : kFp4RowBytes), 1, (uint32_t)(big ? kBN : G), 1};
    const pkv_status s = encode_tiled(&p.map[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, bases[t], scales ? sdims : cdims,
                                      scales ? sstr : cstr, box, names[t], !scales);
    if (s != PKV_OK) return s;
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.v_bscale = v_bscale;
  p.scale_stride_blk = scale_stride_blk;
  p.scale_stride_tok = scale_stride_tok;
  p.scale_stride_head = scale_stride_head;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks;
  p.block_size = block_size;
  p.seg = G;
  p.seq_lens = seq_lens;
  p.num_reqs = num_reqs;
  p.T = T;
  p.group = group;
  p.num_q_heads = num_q_heads;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ws = workspace;
  p.dev_err = dev_err;
  p.wait_limit_ns = take_wait_limit_ns();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return narrow ? launch<16>(p, st) : launch<32>(p, st);
}
