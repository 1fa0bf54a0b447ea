// Layout of the paged 4-bit key/value cache ("KV4"), shared by its kernels.
//
// The pool holds n_pages pages; a page holds page_size token rows for every kv
// head. One (page, kv head) block is contiguous: K codes [P][d/2], V codes
// [P][d/2], K parameters [P], V parameters [P] (a parameter word is the bf16
// scale s in bits 0..15 and the bf16 centre z in bits 16..31), P (d + 8) bytes,
// a multiple of 16: one bulk copy brings a block.
//
// A row of d values x is z + s (q - 8) with codes q in 0..15. Word w of a
// row's codes holds dims 8w .. 8w+7: nibble j (j < 4) is dim 8w + 2j and nibble
// j + 4 is dim 8w + 2j + 1, so that (word >> 4j) & 0x000F000F is the dim pair
// (8w + 2j, 8w + 2j + 1) in the two halves of a bf16 pair. At d = 128 the two
// 32-byte halves of a row are swapped in rows whose index has bit 1 set: the
// lanes of a warp that read 8 bytes of four different rows then touch
// different banks.
#pragma once

#include "w12_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace kv4 {

constexpr int kMaxPage = 128;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: a smaller scale stores the row as a constant

__host__ __device__ constexpr int64_t block_bytes(int page_size, int d) { return int64_t(page_size) * (d + 8); }

inline bool page_ok(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

inline bool cache_ok(const w12_kv4* c) {
  return c->n_pages >= 1 && c->Hkv >= 1 && c->Hkv <= 1024 && page_ok(c->page_size) &&
         (c->head_dim == 64 || c->head_dim == 128) &&
         c->n_pages <= int64_t(0x7FFFFFFF) / c->page_size;  // slots are int32
}

// Byte of word w of row r within the row's codes.
__host__ __device__ constexpr int word_off(int d, int r, int w) {
  return d == 128 ? ((w ^ (((r >> 1) & 1) << 3)) << 2) : (w << 2);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// (a & mask) | bits in one instruction (left to itself the compiler takes two, with
// an immediate each).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
  return r;
}

// fp16 pairs: a + b and a b + c.
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Two fp32 values -> one word of bf16 (round to nearest even): lo in bits 0..15.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Dim pair (2j, 2j + 1) of a code word as two fp32 values z + s (q - 8). The
// nibble becomes the mantissa of 2^23 + q, from which 2^23 + 8 leaves q - 8.
__device__ __forceinline__ float2 value_pair(uint32_t w, int j, float s, float z) {
  const float a = __uint_as_float(and_or(w >> (4 * j), 15u, 0x4B000000u)) - 8388616.f;
  const float b = __uint_as_float(and_or(w >> (4 * j + 16), 15u, 0x4B000000u)) - 8388616.f;
  return make_float2(fmaf(s, a, z), fmaf(s, b, z));
}

}  // namespace kv4
}  // namespace w12
