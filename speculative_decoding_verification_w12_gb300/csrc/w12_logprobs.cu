// Log probabilities of given tokens, entropy and top alternatives of logits rows.
//
// With x = scale * logit: lse = log sum e^x, logprob(t) = x_t - lse,
// entropy = lse - sum p x, and the k largest logprobs with their tokens (ties:
// lowest token first). One pass: a CTA takes a chunk of one row into registers,
// finds its maximum m and the sums s0 = sum e^(x - m), s1 = sum e^(x - m) (x - m),
// and its k largest elements; the row's last CTA to finish joins the chunks:
//   M = max m_i, w_i = e^(m_i - M), S0 = sum w_i s0_i,
//   S1 = sum w_i (s1_i + (m_i - M) s0_i), lse = M + log S0, entropy = log S0 - S1 / S0.
// Sums are fp32 over at most kThreads x kEpt elements a chunk, the joins likewise.
//
// Top k of a set held by the CTA's threads: an element's key is its value as an
// ordered 32-bit integer over the complement of its index, so keys are unique
// and their order is the output's. Each warp finds the r = ceil(k / warps)
// largest of its lanes' own maxima; the least of the warps' r-th is a key that
// at least k elements reach, so only elements from it on are candidates (a few
// dozen). They go to a list in shared memory, and a candidate's rank is the
// number of larger ones. A list that would overflow (values sorted along the
// row can do that) takes the k maxima one by one instead.
//
// Elements of -inf (masked tokens) are no candidates: slots of the top list
// that no element fills get token -1 and logprob -inf. A row of nothing else
// has lse = -inf, every logprob -inf and entropy 0. NaN or +inf in a row makes
// lse, entropy and logprobs NaN.
#include <math.h>

#include "w12_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace logprobs_impl {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kCap = 1024;  // candidates listed in shared memory
constexpr float kLog2e = 1.4426950408889634f;

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

// The k largest keys of the CTA, largest first, in out[0 .. k) (0 where there are
// fewer). `best` is the thread's largest key; each(f) calls f(key) for all of the
// thread's keys (0 = none). The first `live` warps are those whose lanes all hold
// elements (at least 1 is taken). Every thread of the CTA calls it.
template <typename Each>
__device__ __forceinline__ void cta_top_k(TopSmem& sm, uint64_t best, int k, int live, uint64_t* out, Each&& each) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = (k + live - 1) / live;
  uint64_t mine = best, cut = 0;
  for (int i = 0; i < r; ++i) {
    cut = warp_max(mine);
    if (mine == cut) mine = 0;
  }
  if (lane == 0) sm.warp_key[warp] = cut;
  if (tid == 0) sm.count = 0;
  __syncthreads();
  cut = sm.warp_key[0];
  for (int w = 1; w < live; ++w) cut = min(cut, sm.warp_key[w]);
  cut = max(cut, uint64_t(1));  // key 0 is no element
  if (best >= cut)
    each([&](uint64_t key) {
      if (key >= cut) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCap) sm.list[at] = key;
      }
    });
  __syncthreads();
  const int n = sm.count;
  if (n <= kCap) {
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = sm.list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += sm.list[j] > key;
      if (rank < k) out[rank] = key;
    }
    for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
  } else {
    // More than kCap candidates: one maximum at a time.
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
}

// Warps whose lanes all hold elements where the first `threads` threads do.
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

// kEpt elements a thread, in pieces of 8 (kVec: 16-byte loads): piece i of
// thread t holds elements (i * kThreads + t) * 8 .. + 7 of the chunk.
template <int kType, int kEpt, bool kVec>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ Params p) {
  constexpr int kPieces = kEpt / 8;
  __shared__ TopSmem sm;
  __shared__ float red[3][kWarps];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = blockIdx.x;
  const int64_t row = blockIdx.y;
  constexpr int64_t kEsize = kType == kF32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(p.logits) + row * p.pitch * kEsize;
  const int64_t c0 = int64_t(chunk) * (kThreads * kEpt);

  grid_dep_wait();
  grid_dep_launch();
  float x[kEpt];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t e0 = c0 + (i * kThreads + tid) * 8;
    bool done = false;
    if constexpr (kVec) {
      if (e0 + 8 <= p.V) {
        done = true;
        const uint4* src = reinterpret_cast<const uint4*>(base + e0 * kEsize);
        if constexpr (kType == kF32) {
          const uint4 a = __ldg(src), b = __ldg(src + 1);
          x[8 * i] = __uint_as_float(a.x), x[8 * i + 1] = __uint_as_float(a.y);
          x[8 * i + 2] = __uint_as_float(a.z), x[8 * i + 3] = __uint_as_float(a.w);
          x[8 * i + 4] = __uint_as_float(b.x), x[8 * i + 5] = __uint_as_float(b.y);
          x[8 * i + 6] = __uint_as_float(b.z), x[8 * i + 7] = __uint_as_float(b.w);
        } else {
          const uint4 a = __ldg(src);
          const uint16_t* hlf = reinterpret_cast<const uint16_t*>(&a);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[8 * i + j] = element<kType>(hlf, j);
        }
      }
    }
    if (!done) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[8 * i + j] = e0 + j < p.V ? element<kType>(base, e0 + j) : -INFINITY;
    }
  }
  float mine = -INFINITY;
  int at = 0;  // where the thread's largest element is (its lowest index)
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    x[i] = fmaf(x[i], p.scale, 0.f);  // + 0: a zero of either sign is one value
    if (x[i] > mine) {
      mine = x[i];
      at = i;
    }
  }
  const float wm = warp_fmax(mine);
  if (lane == 0) red[0][warp] = wm;
  __syncthreads();
  float m = red[0][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red[0][w]);
  const float ref = m == -INFINITY ? 0.f : m;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    const float t = x[i] - ref;
    const float e = exp2f(t * kLog2e);
    s0 += e;
    s1 = fmaf(e, fmaxf(t, -1e30f), s1);  // 0 where e is 0, also at t = -inf
  }
  s0 = warp_sum(s0);
  s1 = warp_sum(s1);
  if (lane == 0) {
    red[1][warp] = s0;
    red[2][warp] = s1;
  }
  __syncthreads();
  const int64_t slot = row * p.nch + chunk;
  if (tid == 0) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a += red[1][w];
      b += red[2][w];
    }
    p.part[slot] = make_float4(m, a, b, 0.f);
  }
  if (p.k > 0) {
    const uint32_t i0 = uint32_t(c0) + tid * 8;
    auto index = [&](int i) { return i0 + uint32_t(i >> 3) * (kThreads * 8) + uint32_t(i & 7); };
    const uint64_t best = mine > -INFINITY ? key_of(mine, index(at)) : 0;
    cta_top_k(sm, best, p.k, live_warps((p.V - c0) / 8), p.cand + slot * p.k, [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < kEpt; ++i) f(x[i] > -INFINITY ? key_of(x[i], index(i)) : uint64_t(0));
    });
  }
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
  const float4* part = p.part + row * p.nch;
  float M = -INFINITY;
  for (int i = tid; i < p.nch; i += kThreads) M = fmaxf(M, __ldcg(part + i).x);
  M = warp_fmax(M);
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
  M = red[0][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, red[0][w]);
  float S0 = 0.f, S1 = 0.f;
  for (int i = tid; i < p.nch; i += kThreads) {
    const float4 v = __ldcg(part + i);
    if (v.x == -INFINITY && v.y == 0.f) continue;  // a chunk of masked tokens (NaN sums stay in)
    const float d = v.x == M ? 0.f : v.x - M, w = exp2f(d * kLog2e);
    S0 = fmaf(w, v.y, S0);
    S1 += w * fmaf(fmaxf(d, -1e30f), v.y, v.z);
  }
  S0 = warp_sum(S0);
  S1 = warp_sum(S1);
  __syncthreads();
  if (lane == 0) {
    red[1][warp] = S0;
    red[2][warp] = S1;
  }
  __syncthreads();
  S0 = S1 = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    S0 += red[1][w];
    S1 += red[2][w];
  }
  const bool nothing = M == -INFINITY && S0 == 0.f;
  const float logS = logf(S0);
  const float lse = nothing ? -INFINITY : M + logS;
  if (tid == 0) {
    p.lse[row] = lse;
    p.entropy[row] = nothing ? 0.f : logS - S1 / S0;
  }
  for (int j = tid; j < p.n; j += kThreads) {
    const int t = p.tokens[row * p.n + j];
    float lp = 0.f;
    if (t >= 0 && t < p.V) {
      lp = nothing ? -INFINITY : element<kType>(base, t) * p.scale - lse;
    } else if (t >= p.V || t < -1) {
      set_status(p.status, W12_ERR_ARG);
      lp = NAN;
    }
    p.logprob[row * p.n + j] = lp;
  }
  if (p.k > 0) {
    // Candidates of all chunks; a chunk's are sorted, so each thread's own best
    // is the first of those it holds.
    const uint64_t* cand = p.cand + row * p.nch * p.k;
    const int total = p.nch * p.k;
    uint64_t best = 0;
    for (int i = tid; i < total; i += kThreads) best = max(best, __ldcg(cand + i));
    __shared__ uint64_t top[kMaxK];
    cta_top_k(sm, best, p.k, live_warps(total), top, [&](auto&& f) {
      for (int i = tid; i < total; i += kThreads) f(__ldcg(cand + i));
    });
    __syncthreads();
    if (tid < p.k) {
      const uint64_t key = top[tid];
      p.top_id[row * p.k + tid] = key ? int32_t(~uint32_t(key)) : -1;
      p.top_lp[row * p.k + tid] = key ? value_of(uint32_t(key >> 32)) - lse : -INFINITY;
    }
  }
}

// Elements a thread: 64 where the rows then still give every SM a few chunks, 16
// below that (short calls are latency-bound: more, smaller chunks).
static int ept_of(int64_t M, int64_t V) { return M * ((V + 64 * kThreads - 1) / (64 * kThreads)) >= 600 ? 64 : 16; }

static int chunks_of(int64_t M, int64_t V) {
  const int64_t c = int64_t(kThreads) * ept_of(M, V);
  return int((V + c - 1) / c);
}

static bool shape_ok(int64_t M, int64_t V, int k) {
  return M >= 1 && M <= 65535 && V >= 1 && V < (int64_t(1) << 30) && k >= 0 && k <= kMaxK;
}

static size_t ws_bytes_of(int64_t M, int64_t V, int k) {
  const int64_t nch = chunks_of(M, V);
  return size_t(round_up(M * 4, 256) + M * nch * 16 + M * nch * k * 8);
}

template <int kType, int kEpt>
static cudaError_t launch(const cudaLaunchConfig_t& cfg, const Params& p, bool vec) {
  return vec ? cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, kEpt, true>, p)
             : cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, kEpt, false>, p);
}

template <int kType>
static cudaError_t launch(const cudaLaunchConfig_t& cfg, const Params& p, int ept, bool vec) {
  return ept == 64 ? launch<kType, 64>(cfg, p, vec) : launch<kType, 16>(cfg, p, vec);
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
  p.nch = chunks_of(M, V);
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
  const int ept = ept_of(M, V);
  const bool vec = aligned(logits, 16) && (row_stride * esize) % 16 == 0;
  return cuda_status(dtype == W12_F32    ? launch<kF32>(cfg, p, ept, vec)
                     : dtype == W12_BF16 ? launch<kBf16>(cfg, p, ept, vec)
                                         : launch<kF16>(cfg, p, ept, vec));
}

}  // extern "C"
