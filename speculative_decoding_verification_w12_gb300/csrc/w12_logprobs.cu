// Log probabilities of given tokens, entropy and top alternatives of logits rows.
//
// With x = scale * logit: lse = log sum e^x, logprob(t) = x_t - lse,
// entropy = lse - sum p x, and the k largest logprobs with their tokens (ties:
// lowest token first). One pass: a CTA holds a chunk of one row in registers (as
// it came: 16-byte pieces), finds its maximum m, the sums s0 = sum 2^y and
// s1 = sum 2^y y over y = (x - m) log2(e), and its k largest elements; the row's
// last CTA to finish joins the chunks:
//   M = max m_i, d_i = (m_i - M) log2(e), S0 = sum 2^d_i s0_i,
//   S1 = sum 2^d_i (s1_i + d_i s0_i), lse = M + log S0, entropy = log S0 - ln 2 S1 / S0.
// Sums are fp32, over at most 64 elements a thread and then trees. Bound by the
// read of the logits for many rows, by launch and join latency for few.
//
// Top k of a set held by the CTA's threads: an element's key is its value as an
// ordered 32-bit integer over the complement of its index, so keys are unique
// and their order is the output's. Each warp finds the r = ceil(k / warps)
// largest of its lanes' own maxima; the least of the warps' r-th is a value that
// at least k elements reach, so only elements from it on are candidates (a few
// dozen; a thread looks only into pieces whose maximum reaches it). They go to a
// list in shared memory, and a candidate's rank is the number of larger ones. A
// list that would overflow (equal values, or values sorted along the row) takes
// the k maxima one by one instead.
//
// Elements of -inf (masked tokens) are no candidates: slots of the top list
// that no element fills get token -1 and logprob -inf. A row of nothing else
// has lse = -inf, every logprob -inf and entropy 0. NaN or +inf in a row makes
// lse, entropy and logprobs NaN.
#include <math.h>

#include "w12_attn_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace logprobs_impl {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kCap = 1024;  // candidates listed in shared memory
constexpr int kStaged = 1280;   // chunk candidates the join holds in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const void* logits;
  int64_t V, pitch;  // pitch in elements
  float scale;
  const int32_t* tokens;
  int n, k, nch;
  float *logprob, *entropy, *lse, *top_lp;
  int32_t* top_id;
  float4* part;     // [M, nch]: (m, s0, s1, -)
  uint64_t* cand;   // [M, nch, k]: keys, largest first (0 = none)
  int32_t* done;    // [M]: chunks finished (zero between calls)
  int32_t* status;
};

__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return (uint64_t(order_of(x)) << 32) | uint32_t(~index);
}

__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, uint32_t(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
  return (uint64_t(hi) << 32) | lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_fmax(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

struct TopSmem {
  uint64_t list[kCap];
  uint64_t warp_key[kWarps];
  int count;
};

// The k largest of the listed candidates, largest first, in out[0 .. k) (0 where
// there are fewer); n is their number. With n > kCap the list does not hold them
// all: each(f) calls f(key) for all keys of the thread (0 = none).
template <typename Each>
__device__ __forceinline__ void rank_candidates(TopSmem& sm, int n, int k, uint64_t* out, Each&& each) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (n <= kCap) {
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = sm.list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sm.list[j] > key;
      if (rank < k) out[rank] = key;
    }
    for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
    return;
  }
  uint64_t below = ~uint64_t(0);
  for (int i = 0; i < k; ++i) {
    uint64_t m = 0;
    each([&](uint64_t key) {
      if (key < below && key > m) m = key;
    });
    m = warp_max(m);
    __syncthreads();
    if (lane == 0) sm.warp_key[warp] = m;
    __syncthreads();
    m = sm.warp_key[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = max(m, sm.warp_key[w]);
    if (tid == 0) out[i] = m;
    below = m;
  }
}

__device__ __forceinline__ void list_candidate(TopSmem& sm, uint64_t key) {
  const int at = atomicAdd(&sm.count, 1);
  if (at < kCap) sm.list[at] = key;
}

// Warps whose lanes all hold elements where the first `threads` threads do (at
// least 1): the ones whose r-th maxima bound the k-th of all.
__device__ __forceinline__ int live_warps(int64_t threads) {
  return int(max(int64_t(1), min(int64_t(kWarps), threads / 32)));
}

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };

template <int kType>
__device__ __forceinline__ float element(const void* base, int64_t i) {
  if constexpr (kType == kF32) return static_cast<const float*>(base)[i];
  const uint16_t b = static_cast<const uint16_t*>(base)[i];
  if constexpr (kType == kBf16) return __uint_as_float(uint32_t(b) << 16);
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(b));
  return f;
}

// The elements of a 16-byte piece as fp32, and the largest of them (NaN ignored).
template <int kType>
struct Piece {
  static constexpr int kN = kType == kF32 ? 4 : 8;
  static constexpr uint32_t kMinusInf = kType == kF32 ? 0xFF800000u : kType == kBf16 ? 0xFF80FF80u : 0xFC00FC00u;

  static __device__ __forceinline__ void values(const uint4& v, float (&x)[kN]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == kF32) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (kType == kBf16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(w[i]));
      }
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kType == kBf16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& v) {
    float x[kN];
    if constexpr (kType == kF32) {
      values(v, x);
      return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    } else {
      const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
      values(make_uint4(m, m, m, m), x);
      return fmaxf(x[0], x[1]);
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keeps the pieces as loaded between passes: without it the compiler holds their
// converted values (twice the registers) from one pass to the next.
template <int kPieces>
__device__ __forceinline__ void as_loaded(uint4 (&raw)[kPieces]) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    asm volatile("" : "+r"(raw[i].x), "+r"(raw[i].y), "+r"(raw[i].z), "+r"(raw[i].w));
}

// kPieces 16-byte pieces a thread: piece i of thread t is the chunk's elements
// (i * kThreads + t) * kN .. + kN - 1 (kVec: one 16-byte load).
template <int kType, int kPieces, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ Params p) {
  using Pc = Piece<kType>;
  constexpr int kN = Pc::kN;
  __shared__ TopSmem sm;
  __shared__ float red[2][kWarps];
  __shared__ uint32_t wtop[2][kWarps];  // each warp's largest and r-th largest lane maximum
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = blockIdx.x;
  const int64_t row = blockIdx.y;
  constexpr int64_t kEsize = kType == kF32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(p.logits) + row * p.pitch * kEsize;
  const int64_t c0 = int64_t(chunk) * (kThreads * kPieces * kN);

  grid_dep_wait();
  grid_dep_launch();
  uint4 raw[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t e0 = c0 + (i * kThreads + tid) * kN;
    if (kVec && e0 + kN <= p.V) {
      raw[i] = __ldg(reinterpret_cast<const uint4*>(base + e0 * kEsize));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = Pc::kMinusInf;
        if constexpr (kType == kF32) {
          if (e0 + j < p.V) w[j] = reinterpret_cast<const uint32_t*>(base)[e0 + j];
        } else {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(base);
          if (e0 + 2 * j < p.V) w[j] = (w[j] & 0xFFFF0000u) | h[e0 + 2 * j];
          if (e0 + 2 * j + 1 < p.V) w[j] = (w[j] & 0x0000FFFFu) | (uint32_t(h[e0 + 2 * j + 1]) << 16);
        }
      }
      raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // x = scale * logit + 0: monotonic in the logit, and a zero of either sign is one value.
  float top[kPieces], mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    top[i] = fmaf(Pc::largest(raw[i]), p.scale, 0.f);
    mine = fmaxf(mine, top[i]);
  }
  const int live = live_warps((p.V - c0) / kN);
  {
    // Lanes of equal value leave together: the r-th taken is then lower, a weaker bound.
    const int r = max(1, (p.k + live - 1) / live);
    uint32_t o = mine > -INFINITY ? order_of(mine) : 0u, cut = 0u;
    for (int i = 0; i < r; ++i) {
      cut = __reduce_max_sync(0xFFFFFFFFu, o);
      if (i == 0 && lane == 0) wtop[0][warp] = cut;
      if (o == cut) o = 0u;
    }
    if (lane == 0) wtop[1][warp] = cut;
    if (tid == 0) sm.count = 0;
  }
  __syncthreads();
  uint32_t mo = wtop[0][0], cut = wtop[1][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    mo = max(mo, wtop[0][w]);
    if (w < live) cut = min(cut, wtop[1][w]);
  }
  const float m = mo ? value_of(mo) : -INFINITY;
  const uint32_t i0 = uint32_t(c0) + tid * kN;
  as_loaded(raw);
  if (p.k > 0) {
    // cut = 0 (a warp without r maxima): every element is a candidate.
    const float least = cut ? value_of(cut) : -INFINITY;
    if (mine >= least) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (top[i] >= least) {
          float x[kN];
          Pc::values(raw[i], x);
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            x[j] = fmaf(x[j], p.scale, 0.f);
            if (x[j] >= least && x[j] > -INFINITY) list_candidate(sm, key_of(x[j], i0 + i * (kThreads * kN) + j));
          }
        }
    }
  }
  float s0, s1;
  as_loaded(raw);
  {
    // Masked elements: y = -inf is held at -200, whose power is 0. NaN passes.
    // (x - m first: m log2(e) alone may pass the fp32 range.)
    const float bb = m == -INFINITY ? 0.f : -m;
    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
    const float2 c2 = make_float2(p.scale, p.scale), b2 = make_float2(bb, bb);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float x[kN];
      Pc::values(raw[i], x);
#pragma unroll
      for (int j = 0; j < kN; j += 2) {
        float2 y = attn_impl::fma2(make_float2(x[j], x[j + 1]), c2, b2);
        y.x = max_nan(y.x * kLog2e, -200.f);
        y.y = max_nan(y.y * kLog2e, -200.f);
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        a0 = attn_impl::add2(a0, e);
        a1 = attn_impl::fma2(e, y, a1);
      }
    }
    s0 = warp_sum(a0.x + a0.y);
    s1 = warp_sum(a1.x + a1.y);
  }
  as_loaded(raw);
  if (lane == 0) {
    red[0][warp] = s0;
    red[1][warp] = s1;
  }
  __syncthreads();
  const int64_t slot = row * p.nch + chunk;
  if (tid == 0) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a += red[0][w];
      b += red[1][w];
    }
    p.part[slot] = make_float4(m, a, b, 0.f);
  }
  if (p.k > 0)
    rank_candidates(sm, sm.count, p.k, p.cand + slot * p.k, [&](auto&& f) {
      as_loaded(raw);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        float x[kN];
        Pc::values(raw[i], x);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          x[j] = fmaf(x[j], p.scale, 0.f);
          f(x[j] > -INFINITY ? key_of(x[j], i0 + i * (kThreads * kN) + j) : uint64_t(0));
        }
      }
    });
  // The row's last chunk joins them all.
  __syncthreads();
  if (tid == 0) {
    fence_acq_rel_gpu();
    const int before = atomic_add_acq_rel_gpu(p.done + row, 1);
    last = before == p.nch - 1;
    if (last) p.done[row] = 0;
  }
  __syncthreads();
  if (!last) return;
  fence_acq_rel_gpu();
  // Loads of both kinds are in flight together.
  const float4* part = p.part + row * p.nch;
  const uint64_t* cand = p.cand + row * p.nch * p.k;
  const int total = p.nch * p.k;
  __shared__ uint64_t staged[kStaged];
  const bool in_smem = total <= kStaged;
  float4 first = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  if (tid < p.nch) first = __ldcg(part + tid);
  uint64_t best = 0;
  for (int i = tid; i < total; i += kThreads) {
    const uint64_t key = __ldcg(cand + i);
    best = max(best, key);
    if (in_smem) staged[i] = key;
  }
  float M = first.x;
  for (int i = tid + kThreads; i < p.nch; i += kThreads) M = fmaxf(M, __ldcg(part + i).x);
  M = warp_fmax(M);
  if (lane == 0) red[0][warp] = M;
  const int live2 = live_warps(total);
  {
    const int r = max(1, (p.k + live2 - 1) / live2);
    uint64_t mine2 = best, cut2 = 0;
    for (int i = 0; i < r; ++i) {
      cut2 = warp_max(mine2);
      if (mine2 == cut2) mine2 = 0;
    }
    if (lane == 0) sm.warp_key[warp] = cut2;
    if (tid == 0) sm.count = 0;
  }
  __syncthreads();
  M = red[0][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, red[0][w]);
  if (p.k > 0) {
    uint64_t cut2 = sm.warp_key[0];
    for (int w = 1; w < live2; ++w) cut2 = min(cut2, sm.warp_key[w]);
    cut2 = max(cut2, uint64_t(1));  // key 0 is no element
    if (best >= cut2)
      for (int i = tid; i < total; i += kThreads) {
        const uint64_t key = in_smem ? staged[i] : __ldcg(cand + i);
        if (key >= cut2) list_candidate(sm, key);
      }
  }
  float S0 = 0.f, S1 = 0.f;
  for (int i = tid; i < p.nch; i += kThreads) {
    const float4 v = i < kThreads ? first : __ldcg(part + i);
    if (v.x == -INFINITY && v.y == 0.f) continue;  // a chunk of masked tokens (NaN sums stay in)
    const float d = v.x == M ? 0.f : max_nan((v.x - M) * kLog2e, -200.f), w = ex2(d);
    S0 = fmaf(w, v.y, S0);
    S1 += w * fmaf(d, v.y, v.z);
  }
  S0 = warp_sum(S0);
  S1 = warp_sum(S1);
  __syncthreads();
  if (lane == 0) {
    red[0][warp] = S0;
    red[1][warp] = S1;
  }
  __shared__ uint64_t best_keys[kMaxK];
  if (p.k > 0)
    rank_candidates(sm, sm.count, p.k, best_keys, [&](auto&& f) {
      for (int i = tid; i < total; i += kThreads) f(in_smem ? staged[i] : __ldcg(cand + i));
    });
  __syncthreads();
  S0 = S1 = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    S0 += red[0][w];
    S1 += red[1][w];
  }
  const bool nothing = M == -INFINITY && S0 == 0.f;
  const float logS = logf(S0);
  const float lse = nothing ? -INFINITY : M + logS;
  if (tid == 0) {
    p.lse[row] = lse;
    p.entropy[row] = nothing ? 0.f : logS - kLn2 * (S1 / S0);
  }
  for (int j = tid; j < p.n; j += kThreads) {
    const int t = p.tokens[row * p.n + j];
    float lp = 0.f;
    if (t >= 0 && t < p.V) {
      lp = nothing ? -INFINITY : element<kType>(base, t) * p.scale - lse;
    } else if (t != -1) {
      set_status(p.status, W12_ERR_ARG);
      lp = NAN;
    }
    p.logprob[row * p.n + j] = lp;
  }
  if (tid < p.k) {
    const uint64_t key = best_keys[tid];
    p.top_id[row * p.k + tid] = key ? int32_t(~uint32_t(key)) : -1;
    p.top_lp[row * p.k + tid] = key ? value_of(uint32_t(key >> 32)) - lse : -INFINITY;
  }
}

// 16-byte pieces a thread: 8 where the rows then still give every SM a few chunks,
// 4 below that (short calls are latency-bound: more, smaller chunks).
static int pieces_of(int64_t M, int64_t V, int esize) {
  const int64_t c = int64_t(kThreads) * 8 * (16 / esize);
  return M * ((V + c - 1) / c) >= 600 ? 8 : 4;
}

static int chunks_of(int64_t M, int64_t V, int esize) {
  const int64_t c = int64_t(kThreads) * pieces_of(M, V, esize) * (16 / esize);
  return int((V + c - 1) / c);
}

static bool shape_ok(int64_t M, int64_t V, int k) {
  return M >= 1 && M <= 65535 && V >= 1 && V < (int64_t(1) << 30) && k >= 0 && k <= kMaxK;
}

// For either element size (fp32 has the more chunks of a given size, but may
// take the larger pieces earlier).
static size_t ws_bytes_of(int64_t M, int64_t V, int k) {
  const int64_t a = chunks_of(M, V, 4), b = chunks_of(M, V, 2), nch = a > b ? a : b;
  return size_t(round_up(M * 4, 256) + M * nch * 16 + M * nch * k * 8);
}

template <int kType, int kPieces>
static cudaError_t launch(const cudaLaunchConfig_t& cfg, const Params& p, bool vec) {
  return vec ? cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, kPieces, true>, p)
             : cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, kPieces, false>, p);
}

template <int kType>
static cudaError_t launch(const cudaLaunchConfig_t& cfg, const Params& p, int pieces, bool vec) {
  return pieces == 8 ? launch<kType, 8>(cfg, p, vec) : launch<kType, 4>(cfg, p, vec);
}

}  // namespace logprobs_impl
}  // namespace w12

using namespace w12;
using namespace w12::logprobs_impl;

extern "C" {

size_t w12_logprobs_ws_bytes(int64_t M, int64_t V, int k) { return shape_ok(M, V, k) ? ws_bytes_of(M, V, k) : 0; }

int w12_logprobs(const void* logits, int dtype, int64_t M, int64_t V, int64_t row_stride, float scale,
                 const int32_t* tokens, int n, int k, float* logprob, float* entropy, float* lse, float* top_logprob,
                 int32_t* top_id, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int esize = dtype == W12_F32 ? 4 : 2;
  if (!logits || dtype < W12_F32 || dtype > W12_F16 || !aligned(logits, esize) || !(scale > 0.f) || scale > 1e30f ||
      n < 0 || (n > 0 && (!tokens || !logprob)) || !entropy || !lse || (k > 0 && (!top_logprob || !top_id)))
    return W12_ERR_ARG;
  if (!shape_ok(M, V, k) || row_stride < V || n > 65536) return W12_ERR_SHAPE;
  if (!ws || !aligned(ws, 16) || ws_bytes < ws_bytes_of(M, V, k)) return W12_ERR_WORKSPACE;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  Params p{};
  p.logits = logits;
  p.V = V;
  p.pitch = row_stride;
  p.scale = scale;
  p.tokens = tokens;
  p.n = n;
  p.k = k;
  p.nch = chunks_of(M, V, esize);
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_lp = top_logprob;
  p.top_id = top_id;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.done = reinterpret_cast<int32_t*>(w);
  p.part = reinterpret_cast<float4*>(w + round_up(M * 4, 256));
  p.cand = reinterpret_cast<uint64_t*>(w + round_up(M * 4, 256) + M * p.nch * 16);
  p.status = dev_status;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.nch), unsigned(M));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  const int pieces = pieces_of(M, V, esize);
  const bool vec = aligned(logits, 16) && (row_stride * esize) % 16 == 0;
  return cuda_status(dtype == W12_F32    ? launch<kF32>(cfg, p, pieces, vec)
                     : dtype == W12_BF16 ? launch<kBf16>(cfg, p, pieces, vec)
                                         : launch<kF16>(cfg, p, pieces, vec));
}

}  // extern "C"
