// Device pieces that the tensor-memory attention kernels share: waits for TMEM
// loads, the MN-major operand descriptor, the tree mask, and the softmax of a
// score row held in registers. Inline PTX and arithmetic written for this library.
#pragma once

#include "w12_dev.cuh"

namespace w12 {
namespace attn_impl {

#define W12_TIE8(v, o)                                                                                   \
  "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), "+r"(v[o + 5]), "+r"(v[o + 6]), \
      "+r"(v[o + 7])

// Wait for every outstanding tcgen05.ld of this thread; ties all 128 values
// to the wait (for loads issued as several 16-column pieces).
__device__ __forceinline__ void tmem_ld_wait64(uint32_t (&v)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : W12_TIE8(v, 0), W12_TIE8(v, 8), W12_TIE8(v, 16), W12_TIE8(v, 24), W12_TIE8(v, 32), W12_TIE8(v, 40),
                 W12_TIE8(v, 48), W12_TIE8(v, 56)
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait128(uint32_t (&v)[128]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : W12_TIE8(v, 0), W12_TIE8(v, 8), W12_TIE8(v, 16), W12_TIE8(v, 24), W12_TIE8(v, 32), W12_TIE8(v, 40),
                 W12_TIE8(v, 48), W12_TIE8(v, 56), W12_TIE8(v, 64), W12_TIE8(v, 72), W12_TIE8(v, 80),
                 W12_TIE8(v, 88), W12_TIE8(v, 96), W12_TIE8(v, 104), W12_TIE8(v, 112), W12_TIE8(v, 120)
               :
               : "memory");
}

// Shared-memory matrix descriptor of an MN-major operand stored with the
// 128-byte swizzle: rows along K are 128 bytes of 64 MN-consecutive values,
// 8-row groups 1024 bytes apart (stride byte offset), and the next 64 values
// along MN `lbo` bytes further (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Longest sleep of a waiting thread between looks at the flag that ends its wait and at the
// clock (a long one does not spend issue slots on polling); never longer than the wait's bound.
constexpr uint64_t kSleepNs = 10000;
inline uint32_t sleep_ns(uint64_t limit_ns) { return uint32_t(limit_ns < kSleepNs ? limit_ns : kSleepNs); }

// mbar_try_wait with the time that the hardware may keep the thread asleep.
__device__ __forceinline__ bool mbar_try_wait_hint(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// Wait for the barrier's phase, `sleep` at a time, up to `limit` or until `stop` is set: whether it
// has come. (mbar_wait sleeps for as long as the hardware likes: a bound of microseconds does not hold.)
__device__ __forceinline__ bool mbar_wait_asleep(uint64_t* bar, uint32_t parity, uint64_t limit, uint32_t sleep,
                                                 const volatile int* stop) {
  if (mbar_try_wait_hint(bar, parity, sleep)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0; i < 0x80000000u; ++i) {
    if (mbar_try_wait_hint(bar, parity, sleep)) return true;
    if (*stop || globaltimer_ns() - t0 > limit) break;
  }
  return false;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// l 2^d for d <= 0, where l may be as large as 2^d is small: in two factors, as 2^d alone
// may be below the fp32 range.
__device__ __forceinline__ float scaled_down(float l, float d) {
  const float half = fast_exp2(0.5f * d);
  return l * half * half;
}

// Two fp32 values -> one word of bf16 (round to nearest even): lo in bits 0..15.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The same for fp16, and back.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  float lo, hi;
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(v));
  return make_float2(lo, hi);
}

__device__ __forceinline__ uint32_t word_sel(const uint32_t (&a)[4], int i) {
  return i == 0 ? a[0] : i == 1 ? a[1] : i == 2 ? a[2] : i == 3 ? a[3] : 0u;
}

// Bits sh .. sh+31 of the 128-bit value a (zero outside [0, 128)).
__device__ __forceinline__ uint32_t bits32(const uint32_t (&a)[4], int sh) {
  if (sh <= -32 || sh >= 128) return 0u;
  const int wi = sh >= 0 ? sh >> 5 : -1;
  const int r = sh - wi * 32;  // 0..31
  const uint32_t lo = word_sel(a, wi), hi = word_sel(a, wi + 1);
  return r == 0 ? lo : (lo >> r) | (hi << (32 - r));
}

// A request's parent row spread over the warp: lane l holds parents[l + 32k]
// in pr[k] (one round of loads).
__device__ __forceinline__ void parent_row(const int32_t* pb, int T, int (&pr)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    pr[k] = -1;
    if (32 * k < T && i < T) pr[k] = __ldg(pb + i);
  }
}

// Ancestors of node t (itself included) as a 128-bit set, for every lane of
// the warp at once (warp-collective), from the parent row the warp holds
// (parent_row): each lane walks its node's path by shuffles. A malformed row
// (parents[0] != -1, or parents[i] outside [0, i)) sets W12_ERR_BAD_TREE and
// every lane keeps only its own node.
__device__ __forceinline__ void tree_ancestors(const int (&pr)[4], int t, int T, bool active, uint32_t (&anc)[4],
                                               int32_t* status) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    if (i < T) bad |= i == 0 ? pr[k] != -1 : (pr[k] < 0 || pr[k] >= i);
  }
  anc[0] = anc[1] = anc[2] = anc[3] = 0u;
  const bool row_bad = __any_sync(0xFFFFFFFFu, bad);
  if (row_bad && lane == 0) set_status(status, W12_ERR_BAD_TREE);
  int j = active ? t : -1;
  if (row_bad && j >= 0) {
#pragma unroll
    for (int w = 0; w < 4; ++w) anc[w] = (j >> 5) == w ? 1u << (j & 31) : 0u;
    j = -1;
  }
  // Parents strictly decrease along a valid path: at most T steps.
  for (int step = 0; step <= T && __any_sync(0xFFFFFFFFu, j >= 0); ++step) {
    const int jj = j >= 0 ? j : 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) anc[w] |= (j >= 0 && (jj >> 5) == w) ? 1u << (jj & 31) : 0u;
    // Only the words that hold nodes < T are exchanged (T is uniform).
    const int w = jj >> 5;
    int pj = __shfl_sync(0xFFFFFFFFu, pr[0], jj & 31);
    if (T > 32) {
      const int p1 = __shfl_sync(0xFFFFFFFFu, pr[1], jj & 31);
      pj = w == 1 ? p1 : pj;
    }
    if (T > 64) {
      const int p2 = __shfl_sync(0xFFFFFFFFu, pr[2], jj & 31);
      pj = w == 2 ? p2 : pj;
    }
    if (T > 96) {
      const int p3 = __shfl_sync(0xFFFFFFFFu, pr[3], jj & 31);
      pj = w == 3 ? p3 : pj;
    }
    j = j >= 0 ? pj : -1;
  }
}

// Scores of keys key0 .. key0+127 that the row may not see become -inf: it
// sees all of the prefix (keys < Pb) and the draft keys Pb + j of its
// ancestors j; none past the request's keys.
template <int N>
__device__ __forceinline__ void mask_block(uint32_t (&v)[N], int key0, int Pb, const uint32_t (&anc)[4], bool valid) {
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    const int lim_w = Pb - key0 - 32 * w;  // keys 32w + k with k < lim_w are prefix keys
    const uint32_t pre = lim_w >= 32 ? ~0u : lim_w <= 0 ? 0u : ((1u << lim_w) - 1u);
    const uint32_t allow = valid ? (pre | bits32(anc, key0 + 32 * w - Pb)) : 0u;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (!((allow >> k) & 1u)) v[32 * w + k] = __float_as_uint(-INFINITY);
  }
}

// Maximum of the N scores (eight independent chains).
template <int N>
__device__ __forceinline__ float block_max(const uint32_t (&v)[N]) {
  float mx8[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) mx8[a] = __uint_as_float(v[a]);
#pragma unroll
  for (int k = 8; k < N; ++k) mx8[k & 7] = fmaxf(mx8[k & 7], __uint_as_float(v[k]));
  return fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])), fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
}

// Two lanes of fp32 in one instruction (sm_100 family): d = a * b + c and
// d = a + b, each lane rounded as its scalar form.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// P_k = 2^(c s_k + negm), packed as bf16 pairs into v[0 .. N/2-1] in place
// (pair k overwrites v[k], which pair k/2 has already read); returns the fp32 sum.
// The scale and the sum run two lanes per instruction (the softmax is bound
// by instruction issue, not by the exp2 unit).
template <int N>
__device__ __forceinline__ float exp_pack(uint32_t (&v)[N], float c, float negm) {
  float2 ps4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 c2 = make_float2(c, c), m2 = make_float2(negm, negm);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    const float2 x = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2, m2);
    const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    ps4[k & 3] = add2(ps4[k & 3], p);
    v[k] = pack_bf16x2(p.x, p.y);
  }
  const float2 s = add2(add2(ps4[0], ps4[1]), add2(ps4[2], ps4[3]));
  return s.x + s.y;
}

// O row (kCols columns) *= f (warp-collective: every lane of the warp calls it).
template <int kCols = 128>
__device__ __forceinline__ void rescale_row(uint32_t o_row, float f) {
#pragma unroll
  for (int ch = 0; ch < kCols / 16; ++ch) {
    uint32_t o[16];
    tmem_ld16(o_row + uint32_t(ch * 16), o);
    tmem_ld_wait(o);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
    tmem_st16(o_row + uint32_t(ch * 16), o);
  }
}

}  // namespace attn_impl
}  // namespace w12
