// kv_fp4.cuh - the 4-bit cache row shared by its writer, its reader and the attention over it.
//
// A row of 256 elements is 128 bytes of e2m1 codes (element 2i in the low half of byte i, 2i + 1 in
// the high half) and 16 e4m3 bytes, one scale per group of 16 consecutive elements; one fp32 scale
// per tensor multiplies them all: element = e2m1(code) * e4m3(group) * scale. An e2m1 magnitude
// (0, 0.5, 1, 1.5, 2, 3, 4, 6) has 2 significant bits and an e4m3 value 4, so their product has at
// most 6, between 2^-10 and 2688 when it is not zero: fp16 (and bf16) hold it exactly.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "sm103.cuh"

namespace pkv {

constexpr int kFp4D = 256;                    // elements of a row
constexpr int kFp4Group = 16;                 // elements of a scale
constexpr int kFp4RowBytes = kFp4D / 2;       // codes of a row
constexpr int kFp4Groups = kFp4D / kFp4Group;  // scale bytes of a row

// Byte i of w (two codes) -> fp16 pair (low half: the low nibble).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// 8 values -> 8 e2m1 codes, to nearest even, magnitudes past 6 as 6 (the hardware conversion).
__device__ __forceinline__ uint32_t e2m1x8_rn(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One e4m3 byte -> fp16 in both halves.
__device__ __forceinline__ uint32_t e4m3_dup_f16(uint32_t byte) {
  return e4m3x2_to_f16x2((uint16_t)((byte & 0xffu) * 0x101u));
}

// Pair index -> (token, head); the usual pair index fits 32 bits, whose division is an order cheaper.
__host__ __device__ __forceinline__ void split_pair(uint64_t pair, uint32_t heads, uint32_t& tok, uint32_t& head) {
  tok = (pair >> 32) == 0 ? (uint32_t)pair / heads : (uint32_t)(pair / heads);
  head = (uint32_t)(pair - (uint64_t)tok * heads);
}

// Consecutive (token, head) pairs of a request from pair `first` on, token 0 being position pos0 and `end` the
// position after the last: where each lies in the cache. The next block's table entry is read when a block
// is entered, so that the walk stops for no table load after its first, and only if that block holds a
// position of the request. (For the host too, where it is tested.)
struct PairWalk {
  const int32_t* table;
  uint32_t heads, block_size, max_blocks, end;
  uint32_t i, h, slot, col;  // token, head, slot in block, block column
  uint32_t next_pos;         // the next block's first position
  int32_t blk, blk_next;     // -1: past the table, or the request
  __host__ __device__ __forceinline__ int32_t entry(uint32_t c) const {
    if (c >= max_blocks) return -1;
#ifdef __CUDA_ARCH__
    return __ldg(table + c);
#else
    return table[c];
#endif
  }
  __host__ __device__ __forceinline__ PairWalk(const int32_t* t, uint32_t heads_, uint32_t bs, uint32_t mb, uint32_t pos0,
                                               uint32_t end_, uint64_t first)
      : table(t), heads(heads_), block_size(bs), max_blocks(mb), end(end_) {
    split_pair(first, heads, i, h);
    col = (pos0 + i) / bs;
    slot = pos0 + i - col * bs;
    next_pos = col * bs + bs;
    blk = entry(col);
    blk_next = next_pos < end ? entry(col + 1) : -1;
  }
  __host__ __device__ __forceinline__ void next() {
    if (++h < heads) return;
    h = 0;
    ++i;
    if (++slot < block_size) return;
    slot = 0;
    ++col;
    next_pos += block_size;
    blk = blk_next;
    blk_next = next_pos < end ? entry(col + 1) : -1;
  }
};

// 32 contiguous bytes, 32-byte aligned, as one access.
struct alignas(32) Bytes32 {
  uint32_t w[8];
};
__device__ __forceinline__ Bytes32 ldg_bytes32(const void* p) {
  Bytes32 r;
  asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
      : "l"(p));
  return r;
}
__device__ __forceinline__ void stg_bytes32(void* p, const Bytes32& r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
               "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

}  // namespace pkv
