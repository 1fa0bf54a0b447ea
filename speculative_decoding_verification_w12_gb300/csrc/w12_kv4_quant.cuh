// Rows of the 4-bit cache as a few lanes hold them: input elements by type, a row's range,
// its scale and centre, and its code words. Shared by the kernels that write the cache.
#pragma once

#include "w12_kv4.cuh"

namespace w12 {
namespace kv4 {

// Input elements by type: 8 of them as loaded, their least and largest value over
// a row's lanes (NaN passes), and their values.
struct F32 {
  static constexpr int kSize = 4;
  uint32_t w[8];
  __device__ __forceinline__ float value(int i) const { return __uint_as_float(w[i]); }
  template <int kLanes>
  static __device__ __forceinline__ void range(const F32& a, const F32& b, float& lo, float& hi) {
    lo = hi = a.value(0);
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      const float x = i < 8 ? a.value(i) : b.value(i - 8);
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(x));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(x));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(__shfl_xor_sync(0xFFFFFFFFu, lo, o)));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(__shfl_xor_sync(0xFFFFFFFFu, hi, o)));
    }
  }
};

// 16-bit types: pairs, and (largest, -least) as one pair on its way through the lanes.
template <bool kBf16>
struct Half {
  static constexpr int kSize = 2;
  uint32_t w[4];
  static __device__ __forceinline__ float2 pair(uint32_t v) {
    if constexpr (kBf16) return make_float2(bf16_lo(v), bf16_hi(v));
    float2 f;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(v));
    return f;
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kBf16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ float value(int i) const {
    const float2 f = pair(w[i >> 1]);
    return (i & 1) ? f.y : f.x;
  }
  template <int kLanes>
  static __device__ __forceinline__ void range(const Half& a, const Half& b, float& lo, float& hi) {
    constexpr uint32_t kSign = 0x80008000u;
    uint32_t up = a.w[0], down = a.w[0] ^ kSign;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const uint32_t x = i < 4 ? a.w[i] : b.w[i - 4];
      up = max2(up, x);
      down = max2(down, x ^ kSign);
    }
    // (largest of the even elements, least negated) and the same of the odd ones.
    uint32_t v = max2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = max2(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    const float2 f = pair(v);
    hi = f.x;
    lo = -f.y;
  }
};

// kOnce: memory that nothing reads again.
template <typename E, bool kVec, bool kOnce = false>
__device__ __forceinline__ E load8(const uint8_t* p) {
  E e;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < int(sizeof(E) / 16); ++i) {
      const uint4* at = reinterpret_cast<const uint4*>(p) + i;
      reinterpret_cast<uint4*>(e.w)[i] = kOnce ? __ldcs(at) : __ldg(at);
    }
  } else if constexpr (E::kSize == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) e.w[i] = uint32_t(h[2 * i]) | (uint32_t(h[2 * i + 1]) << 16);
  }
  return e;
}

// Two fp32 operations by one instruction, each rounded by itself. A product alone is fma2 with a
// -0 that the compiler does not know (it would join a product and a sum of pairs into one rounding).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 r, x, y, z;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 r, x, y;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Scale, centre and 1 / s of a row.
struct RowScale {
  uint32_t par;
  float z, inv;
  bool finite, inside;  // inside: no code of the row needs its clamp
};

// Of the row that kLanes lanes hold, two pieces each.
template <int kLanes, typename E>
__device__ __forceinline__ RowScale row_scale(const E& a, const E& b) {
  float lo, hi;
  E::template range<kLanes>(a, b, lo, hi);
  constexpr float kR = 1.0f / 15.0f;
  uint32_t sb = pack_bf16x2(__fsub_rn(__fmul_rn(hi, kR), __fmul_rn(lo, kR)), 0.f);
  float s = __uint_as_float(sb << 16);
  if (s < kTiny) {
    sb = 0;
    s = 0.f;
  }
  const uint32_t zb = pack_bf16x2(0.f, fmaf(8.f, s, lo));  // in bits 16..31
  RowScale r;
  r.z = __uint_as_float(zb);
  r.inv = s > 0.f ? __frcp_rn(s) : 0.f;
  r.par = sb | zb;
  r.finite = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;  // false for NaN
  // (x - z) inv grows with x, so the row's ends bound it.
  r.inside = __fmul_rn(__fsub_rn(lo, r.z), r.inv) >= -8.5f && __fmul_rn(__fsub_rn(hi, r.z), r.inv) < 7.5f;
  return r;
}

// A lane's code word. q = clamp(round(t), -8, 7) + 8 as the low bits of 1.5 2^23 +
// 8 + t (adding it rounds t to the nearest integer, ties to even, like rint); the
// eight sums of the constant's own bits come off at the end.
template <bool kClamp, typename E>
__device__ __forceinline__ uint32_t code_word(const E& e, const RowScale& r) {
  constexpr float kMagic = 12582920.f;
  constexpr uint32_t kBits = 0x4B400000u;
  uint32_t word = 0, base = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 4 * ((i >> 1) + 4 * (i & 1));
    float t = __fmul_rn(__fsub_rn(e.value(i), r.z), r.inv);
    if constexpr (kClamp) t = fminf(fmaxf(t, -8.f), 7.f);
    word += __float_as_uint(__fadd_rn(t, kMagic)) << at;
    base += kBits << at;
  }
  return word - base;
}

// The same two elements at a time; nz: -0.
template <bool kClamp, typename E>
__device__ __forceinline__ uint32_t code_word2(const E& e, const RowScale& r, float nz) {
  constexpr float kMagic = 12582920.f;
  constexpr uint32_t kBits = 0x4B400000u;
  uint32_t word = 0, base = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = fma2(add2(make_float2(e.value(2 * i), e.value(2 * i + 1)), both(-r.z)), both(r.inv), both(nz));
    if constexpr (kClamp) t = make_float2(fminf(fmaxf(t.x, -8.f), 7.f), fminf(fmaxf(t.y, -8.f), 7.f));
    t = add2(t, both(kMagic));
    word += (__float_as_uint(t.x) << 4 * i) + (__float_as_uint(t.y) << (4 * i + 16));
    base += (kBits << 4 * i) + (kBits << (4 * i + 16));
  }
  return word - base;
}

// The lane's two code words and its row's parameter word (z). Most rows have no code
// outside -8 .. 7 (their centre's rounding is far below a step), and a warp of such
// rows saves the clamps, a third of its work an element.
template <int kLanes, bool kPairs = false, typename E>
__device__ __forceinline__ uint3 quantise16(const E& a, const E& b, float nz = 0.f) {
  const RowScale r = row_scale<kLanes>(a, b);
  uint3 q;
  if (__all_sync(0xFFFFFFFFu, r.inside)) {
    q.x = kPairs ? code_word2<false>(a, r, nz) : code_word<false>(a, r);
    q.y = kPairs ? code_word2<false>(b, r, nz) : code_word<false>(b, r);
  } else {
    q.x = kPairs ? code_word2<true>(a, r, nz) : code_word<true>(a, r);
    q.y = kPairs ? code_word2<true>(b, r, nz) : code_word<true>(b, r);
  }
  q.z = r.par;
  return r.finite ? q : make_uint3(0x88888888u, 0x88888888u, 0x7FC07FC0u);
}

}  // namespace kv4
}  // namespace w12
