// Log probabilities of given tokens, entropy and top alternatives of logits rows.
//
// With x = scale * logit: lse = log sum e^x, logprob(t) = x_t - lse,
// entropy = lse - sum p x, and the k largest logprobs with their tokens (ties:
// lowest token first). One pass over chunks of 16 KB of a row. Persistent CTAs take
// runs of consecutive chunks (a run ends with its row); a copy warp streams the
// chunks into a ring in shared memory. A thread keeps, over a run, a reference r
// (its first maximum; it moves only when a value exceeds it by more than 40) and
//   s0 = sum 2^y, s1 = sum 2^y y,  y = (x - r) log2(e),
// so the warps go through the run without a barrier. At its end they are joined:
//   M = max r_i, d_i = (r_i - M) log2(e), S0 = sum 2^d_i s0_i,
//   S1 = sum 2^d_i (s1_i + d_i s0_i), lse = M + log S0, entropy = log S0 - ln 2 S1 / S0,
// and likewise a row's runs by the one that finishes last. Sums are fp32: at most
// a run's share of a thread, then trees. 256 rows of
// 151,936 bf16 logits: 21.8 us without a list (3.6 TB/s, half a copy's rate), 33.8 us
// with the 8 largest (2.3 TB/s); 16 fp32 rows 6.4 us and, with the 20 largest, 12.3.
// Bound by issue (58 % of the slots) and the barriers of the lists for many rows, by
// launch and join latency for few.
//
// Top k of a run: an element's key is its value as an ordered 32-bit integer over
// the complement of its index, so keys are unique and their order is the
// output's. In the first chunk each warp finds the r = ceil(k / warps) largest of
// its lanes' own maxima; the least of the warps' r-th is a value that at least k
// elements reach, so only elements from it on are candidates (a few dozen). They
// go to a list in shared memory; a candidate's rank is the number of larger ones,
// and the k-th is the bound for the run's other chunks, where a thread looks only
// into pieces whose maximum reaches it. A list that would overflow (equal values,
// or values that rise along the row) is not used: the k maxima are then taken one
// by one from the logits.
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

constexpr int kThreads = 256;  // and a copy warp
constexpr int kWarps = kThreads / 32;
constexpr int kMaxK = 32;
constexpr int kCap = 1024;  // candidates listed in shared memory
constexpr int kPieces = 4;     // 16-byte pieces of a chunk that a thread holds
constexpr int kChunkBytes = kThreads * kPieces * 16;
constexpr int kStages = 2;
constexpr int kCtas = 4;       // CTAs an SM
constexpr float kFar = 40.f;   // a value this far above its thread's reference moves it
constexpr int kStaged = 1280;   // chunk candidates the join holds in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const void* logits;
  int64_t V, pitch;  // pitch in elements
  float scale;
  const int32_t* tokens;
  int n, k, nch;
  int64_t chunks;   // M nch
  uint64_t limit_ns;
  uint32_t sleep_ns;
  float *logprob, *entropy, *lse, *top_lp;
  int32_t* top_id;
  float4* part;     // [M, nch], by run of the row: (m, s0, s1, -)
  uint64_t* cand;   // [M, nch, k]: keys, largest first (0 = none)
  int32_t* done;    // [grid]: chunks done of the row that begins in the CTA's run and ends in another's (zero between calls)
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

// (NaN is below every number.)
__device__ __forceinline__ float warp_fmax(float v) {
  return value_of(__reduce_max_sync(0xFFFFFFFFu, v == v ? order_of(v) : 0x007FFFFFu));
}

struct Smem {
  alignas(128) uint8_t ring[kStages][kChunkBytes];
  uint64_t list[kCap];
  uint64_t staged[kStaged];
  uint64_t best[kMaxK];
  uint64_t warp_key[kWarps];
  uint64_t full[kStages], empty[kStages];
  float red[kWarps];
  float2 sums[kWarps];
  uint32_t wtop[kWarps];  // each warp's r-th largest lane maximum
  int count;              // candidates of the run
  int last;               // whether the run completed its row
  int failed;
};

// Barrier of the computing threads.
__device__ __forceinline__ void sync() { named_bar_sync(1, kThreads); }

// The k largest of the n <= kCap listed candidates, largest first, in out[0 .. k)
// (0 where there are fewer); four lanes count a candidate's larger ones.
__device__ __forceinline__ void rank_list(const uint64_t* list, int n, int k, uint64_t* out) {
  const int tid = threadIdx.x, warp = tid >> 5;
  for (int i0 = 0; i0 < n; i0 += kThreads / 4) {
    const int i = i0 + (tid >> 2);
    if (i0 + (warp << 3) >= n) break;  // no candidate in this warp
    const uint64_t key = i < n ? list[i] : ~uint64_t(0);
    int rank = 0;
#pragma unroll 4
    for (int j = tid & 3; j < n; j += 4) rank += list[j] > key;
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 1);
    rank += __shfl_xor_sync(0xFFFFFFFFu, rank, 2);
    if (i < n && (tid & 3) == 0 && rank < k) out[rank] = key;
  }
  for (int i = n + tid; i < k; i += kThreads) out[i] = 0;
}

// The same one maximum at a time: each(f) calls f(key) for all keys of the thread
// (0 = none). Every computing thread calls it.
template <typename Each>
__device__ __forceinline__ void rank_all(Smem& s, int k, uint64_t* out, Each&& each) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t below = ~uint64_t(0);
  for (int i = 0; i < k; ++i) {
    uint64_t m = 0;
    each([&](uint64_t key) {
      if (key < below && key > m) m = key;
    });
    m = warp_max(m);
    sync();
    if (lane == 0) s.warp_key[warp] = m;
    sync();
    m = s.warp_key[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = max(m, s.warp_key[w]);
    if (tid == 0) out[i] = m;
    below = m;
  }
}

__device__ __forceinline__ void list_candidate(Smem& s, uint64_t key) {
  const int at = atomicAdd(&s.count, 1);
  if (at < kCap) s.list[at] = key;
}

// Warps whose lanes all hold elements where the first `threads` threads do (at
// least 1): the ones whose r-th maxima bound the k-th of all.
__device__ __forceinline__ int live_warps(int64_t threads) {
  return int(max(int64_t(1), min(int64_t(kWarps), threads / 32)));
}

using attn_impl::mbar_wait_asleep;

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
__device__ __forceinline__ void as_loaded(uint4 (&raw)[kPieces]) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    asm volatile("" : "+r"(raw[i].x), "+r"(raw[i].y), "+r"(raw[i].z), "+r"(raw[i].w));
}

// (r, s0, s1) of a set with the reference moved to `to` (>= r); an empty set adds nothing.
__device__ __forceinline__ void moved(float r, float to, float& s0, float& s1) {
  if (r == to || (r == -INFINITY && s0 == 0.f)) return;  // (NaN sums stay in)
  const float d = max_nan((r - to) * kLog2e, -200.f), f = ex2(d);
  s1 = f * fmaf(d, s0, s1);
  s0 *= f;
}

// Joins (r, s0, s1) of all computing threads; every one gets the result. Loops stay
// loops: what runs once a run is mostly not in the instruction cache, where its length
// counts for more than its steps.
__device__ __forceinline__ float3 join_sums(Smem& s, float r, float s0, float s1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float wm = warp_fmax(r);
  if (lane == 0) s.red[warp] = wm;
  sync();
  const float M = warp_fmax(s.red[lane % kWarps]);
  moved(r, M, s0, s1);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
    s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
  }
  if (lane == 0) s.sums[warp] = make_float2(s0, s1);
  sync();
  float2 v = s.sums[lane % kWarps];
#pragma unroll 1
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  return make_float3(M, v.x, v.y);
}

// Joins the np runs of a finished row and writes its outputs. Every computing
// thread calls it.
template <int kType>
__device__ __noinline__ void join_row(const Params& p, int64_t row, int np, Smem& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* base = static_cast<const uint8_t*>(p.logits) + row * p.pitch * (kType == kF32 ? 4 : 2);
  // Loads of both kinds are in flight together.
  const float4* part = p.part + row * p.nch;
  const uint64_t* cand = p.cand + row * p.nch * p.k;
  const int total = np * p.k;
  const bool in_smem = total <= kStaged;
  float4 v = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  if (tid < np) v = __ldcg(part + tid);
  uint64_t best = 0;
  for (int i = tid; i < total; i += kThreads) {
    const uint64_t key = __ldcg(cand + i);
    best = max(best, key);
    if (in_smem) s.staged[i] = key;
  }
  float r = v.x, s0 = v.y, s1 = v.z;
  for (int i = tid + kThreads; i < np; i += kThreads) {
    float4 u = __ldcg(part + i);
    const float to = fmaxf(r, u.x);
    moved(r, to, s0, s1);
    moved(u.x, to, u.y, u.z);
    r = to;
    s0 += u.y;
    s1 += u.z;
  }
  const int live = live_warps(total);
  if (p.k > 0) {
    const int n = (p.k + live - 1) / live;
    uint64_t mine = best, cut = 0;
    for (int i = 0; i < n; ++i) {
      cut = warp_max(mine);
      if (mine == cut) mine = 0;
    }
    if (lane == 0) s.warp_key[warp] = cut;
  }
  if (tid == 0) s.count = 0;
  const float3 all = join_sums(s, r, s0, s1);
  r = all.x, s0 = all.y, s1 = all.z;
  if (p.k > 0) {
    uint64_t cut = s.warp_key[0];
    for (int w = 1; w < live; ++w) cut = min(cut, s.warp_key[w]);
    cut = max(cut, uint64_t(1));  // key 0 is no element
    if (best >= cut)
      for (int i = tid; i < total; i += kThreads) {
        const uint64_t key = in_smem ? s.staged[i] : __ldcg(cand + i);
        if (key >= cut) list_candidate(s, key);
      }
    sync();
    if (s.count <= kCap)
      rank_list(s.list, s.count, p.k, s.best);
    else
      rank_all(s, p.k, s.best, [&](auto&& f) {
        for (int i = tid; i < total; i += kThreads) f(in_smem ? s.staged[i] : __ldcg(cand + i));
      });
    sync();
  }
  const bool nothing = r == -INFINITY && s0 == 0.f;
  const float logS = logf(s0);
  const float lse = nothing ? -INFINITY : r + logS;
  if (tid == 0) {
    p.lse[row] = lse;
    p.entropy[row] = nothing ? 0.f : logS - kLn2 * (s1 / s0);
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
    const uint64_t key = s.best[tid];
    p.top_id[row * p.k + tid] = key ? int32_t(~uint32_t(key)) : -1;
    p.top_lp[row * p.k + tid] = key ? value_of(uint32_t(key >> 32)) - lse : -INFINITY;
  }
}

// Chunk c is elements (c % nch) * kPer .. of row c / nch; piece i of thread t is
// the chunk's elements (i * kThreads + t) * kN .. + kN - 1. kVec: rows start on
// 16-byte boundaries and come by bulk copies, but for a last part of a piece.
template <int kType, bool kVec>
__global__ void __launch_bounds__(kThreads + 32, kCtas) logprobs_kernel(const __grid_constant__ Params p) {
  using Pc = Piece<kType>;
  constexpr int kN = Pc::kN;
  constexpr int kEsize = kType == kF32 ? 4 : 2;
  constexpr int kPer = kChunkBytes / kEsize;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  volatile int* failed = &s.failed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t c_begin = int64_t(blockIdx.x) * p.chunks / gridDim.x;
  const int64_t c_end = int64_t(blockIdx.x + 1) * p.chunks / gridDim.x;
  const int total = int(c_end - c_begin);
  const uint8_t* logits = static_cast<const uint8_t*>(p.logits);
  int64_t row = c_begin / p.nch;
  int chunk = int(c_begin - row * p.nch);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kWarps);
    }
    s.count = 0;
    s.failed = 0;
    fence_barrier_init();
  }
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------- copies
    if (!kVec || lane != 0) return;
    int c = 0;
    for (; c < total; ++c) {
      const int st = c % kStages;
      if (c >= kStages && !mbar_wait_asleep(&s.empty[st], uint32_t(c / kStages - 1) & 1u, p.limit_ns, p.sleep_ns, failed)) {
        set_status(p.status, W12_ERR_TIMEOUT);
        *failed = 1;
        break;
      }
      const int64_t left = (p.V - int64_t(chunk) * kPer) * kEsize;
      const uint32_t bytes = uint32_t(left < kChunkBytes ? left : int64_t(kChunkBytes)) & ~15u;
      mbar_arrive_expect_tx(&s.full[st], bytes);
      if (bytes) bulk_load(s.ring[st], logits + (row * p.pitch + int64_t(chunk) * kPer) * kEsize, bytes, &s.full[st]);
      if (++chunk == p.nch) {
        chunk = 0;
        ++row;
      }
    }
    // The CTA ends only with every copy landed.
    for (int i = c > kStages ? c - kStages : 0; i < c; ++i)
      mbar_wait(&s.full[i % kStages], uint32_t(i / kStages) & 1u, drain_limit_ns(p.limit_ns));
    return;
  }

  // ---------------------------------------------------------------- compute
  const float2 c2 = make_float2(p.scale, p.scale);
  int done = 0;                              // chunks of the run
  float ref = -INFINITY, s0 = 0.f, s1 = 0.f;
  float least = -INFINITY;                   // candidates reach it
  for (int c = 0; c < total; ++c) {
    const int64_t e0 = int64_t(chunk) * kPer;
    const uint8_t* base = logits + row * p.pitch * kEsize;
    uint4 raw[kPieces];
    if constexpr (kVec) {
      const int st = c % kStages;
      // A warp frees a stage only if it has seen the copy land. After an expired wait it goes on
      // to the CTA's barriers, but the copying warp must not find a stage free that a copy is
      // still on its way to: that would request a second one on an open phase of its barrier.
      const bool go = !*failed;
      const bool mine = go && mbar_wait_asleep(&s.full[st], uint32_t(c / kStages) & 1u, p.limit_ns, p.sleep_ns, failed);
      if (go && !mine) {
        set_status(p.status, W12_ERR_TIMEOUT);
        *failed = 1;
      }
      const bool landed = __all_sync(0xFFFFFFFFu, mine);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) raw[i] = *reinterpret_cast<const uint4*>(&s.ring[st][(i * kThreads + tid) * 16]);
      fence_proxy_async_smem();  // before the copy that refills the stage
      __syncwarp();
      if (landed && lane == 0) mbar_arrive(&s.empty[st]);
    }
    if (!kVec || e0 + kPer > p.V) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int64_t at = e0 + (i * kThreads + tid) * kN;
        if (kVec && at + kN <= p.V) continue;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = Pc::kMinusInf;
          if constexpr (kType == kF32) {
            if (at + j < p.V) w[j] = reinterpret_cast<const uint32_t*>(base)[at + j];
          } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(base);
            if (at + 2 * j < p.V) w[j] = (w[j] & 0xFFFF0000u) | h[at + 2 * j];
            if (at + 2 * j + 1 < p.V) w[j] = (w[j] & 0x0000FFFFu) | (uint32_t(h[at + 2 * j + 1]) << 16);
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
    if (mine > ref + kFar) {
      moved(ref, mine, s0, s1);
      ref = mine;
    }
    if (p.k > 0 && done == 0) {
      // A run's first chunk: a value that k of its elements reach (0: not known).
      // Lanes of equal value leave together: the r-th taken is then lower.
      const int live = live_warps((p.V - e0) / kN), r = (p.k + live - 1) / live;
      uint32_t o = mine > -INFINITY ? order_of(mine) : 0u, cut = 0u;
      for (int i = 0; i < r; ++i) {
        cut = __reduce_max_sync(0xFFFFFFFFu, o);
        if (o == cut) o = 0u;
      }
      if (lane == 0) s.wtop[warp] = cut;
      sync();
      cut = s.wtop[0];
      for (int w = 1; w < live; ++w) cut = min(cut, s.wtop[w]);
      least = cut ? value_of(cut) : -INFINITY;
    }
    const uint32_t i0 = uint32_t(e0) + tid * kN;
    as_loaded(raw);
    if (p.k > 0 && mine >= least && mine > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (top[i] >= least) {
          float x[kN];
          Pc::values(raw[i], x);
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            x[j] = fmaf(x[j], p.scale, 0.f);
            if (x[j] >= least && x[j] > -INFINITY) list_candidate(s, key_of(x[j], i0 + i * (kThreads * kN) + j));
          }
        }
    }
    as_loaded(raw);
    {
      // Masked elements: y = -inf is held at -200, whose power is 0. NaN passes.
      // (x - r first: r log2(e) alone may pass the fp32 range.)
      const float b = ref == -INFINITY ? 0.f : -ref;
      const float2 b2 = make_float2(b, b);
      float2 a0 = make_float2(0.f, 0.f), a1 = a0;
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
      s0 += a0.x + a0.y;
      s1 += a1.x + a1.y;
    }
    ++done;
    const bool ends = chunk == p.nch - 1 || c + 1 == total;
    if (p.k > 0 && done == 1 && !ends) {
      // The bound for the rest of the run: the k-th of the first chunk.
      sync();
      const int n = s.count;
      if (n <= kCap) {
        rank_list(s.list, n, p.k, s.best);
        sync();
        const uint64_t kth = s.best[p.k - 1];
        if (kth) least = value_of(uint32_t(kth >> 32));
        if (tid < p.k) s.list[tid] = s.best[tid];
        if (tid == 0) s.count = n < p.k ? n : p.k;
      }
      sync();
    }
    if (ends) {
      // The run's results: slot by the run's place among those of its row.
      const int64_t g = gridDim.x;
      const int64_t x0 = row * p.nch;
      const int first = int(((x0 + 1) * g - 1) / p.chunks);  // the CTA that holds the row's first chunk
      const int64_t slot = x0 + (int64_t(blockIdx.x) - first);
      const float3 all = join_sums(s, ref, s0, s1);
      if (tid == 0) p.part[slot] = make_float4(all.x, all.y, all.z, 0.f);
      if (p.k > 0) {
        uint64_t* out = p.cand + slot * p.k;
        if (s.count <= kCap) {  // (join_sums' barriers: the list is whole)
          rank_list(s.list, s.count, p.k, out);
        } else {
          const int64_t r0 = e0 + kPer - int64_t(done) * kPer, r1 = min(p.V, e0 + kPer);
          rank_all(s, p.k, out, [&](auto&& f) {
            for (int64_t e = r0 + tid; e < r1; e += kThreads) {
              const float x = fmaf(element<kType>(base, e), p.scale, 0.f);
              f(x > -INFINITY ? key_of(x, uint32_t(e)) : uint64_t(0));
            }
          });
        }
      }
      sync();
      if (tid == 0) {
        // (The barriers around order all threads' stores before it and their loads after.)
        bool last = done == p.nch;  // the whole row
        if (!last) {
          last = atomic_add_acq_rel_gpu(p.done + first, done) + done == p.nch;
          if (last) p.done[first] = 0;
        }
        s.last = last;
        s.count = 0;
      }
      sync();
      if (s.last) {
        const int end = int(((x0 + p.nch) * g - 1) / p.chunks);  // the CTA of the row's last chunk
        join_row<kType>(p, row, end - first + 1, s);
        sync();
        if (tid == 0) s.count = 0;
      }
      done = 0;
      ref = -INFINITY;
      s0 = s1 = 0.f;
      least = -INFINITY;
    }
    if (++chunk == p.nch) {
      chunk = 0;
      ++row;
    }
  }
}

static int esize_of(int dtype) { return dtype == W12_F32 ? 4 : 2; }

static int64_t chunks_of(int64_t V, int esize) { return (V * esize + kChunkBytes - 1) / kChunkBytes; }

static bool shape_ok(int64_t M, int64_t V, int k) {
  return M >= 1 && M <= 65535 && V >= 1 && V < (int64_t(1) << 30) && k >= 0 && k <= kMaxK;
}

// For any element type (fp32 has the most chunks).
static size_t ws_bytes_of(int64_t M, int64_t V, int k) {
  const int64_t nch = chunks_of(V, 4);
  return size_t(kRunCounters * 4 + M * nch * 16 + M * nch * k * 8);
}

template <int kType>
static cudaError_t launch(cudaLaunchConfig_t cfg, const Params& p, bool vec) {
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(logprobs_kernel<kType, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Smem)));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(logprobs_kernel<kType, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Smem)));
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  return vec ? cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, true>, p)
             : cudaLaunchKernelEx(&cfg, logprobs_kernel<kType, false>, p);
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
  const int esize = esize_of(dtype);
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
  p.nch = int(chunks_of(V, esize));
  p.chunks = M * p.nch;
  p.limit_ns = wait_limit_ns();
  p.sleep_ns = attn_impl::sleep_ns(p.limit_ns);
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_lp = top_logprob;
  p.top_id = top_id;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.done = reinterpret_cast<int32_t*>(w);
  p.part = reinterpret_cast<float4*>(w + kRunCounters * 4);
  p.cand = reinterpret_cast<uint64_t*>(w + kRunCounters * 4 + M * p.nch * 16);
  p.status = dev_status;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  int64_t room = int64_t(device_sm_count()) * kCtas;
  if (room > kRunCounters) room = kRunCounters;
  cfg.gridDim = dim3(unsigned(p.chunks < room ? p.chunks : room));
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.blockDim = dim3(kThreads + 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  const bool vec = aligned(logits, 16) && (row_stride * esize) % 16 == 0;
  return cuda_status(dtype == W12_F32    ? launch<kF32>(cfg, p, vec)
                     : dtype == W12_BF16 ? launch<kBf16>(cfg, p, vec)
                                         : launch<kF16>(cfg, p, vec));
}

}  // extern "C"
