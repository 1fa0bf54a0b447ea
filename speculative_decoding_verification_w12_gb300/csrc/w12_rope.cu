// Norms of query and key heads with the rotation by position, in one pass; the same on the
// way into the paged 4-bit cache; positions of a draft tree's nodes.
//
// A head's row x of d values, normed (weights w) and rotated by its token's position:
//   y_i  = (x_i r) w_i,  r = 1 / sqrt(mean x^2 + eps)
//   y_i' = y_i c - y_j s,  y_j' = y_j c + y_i s   for the pairs (i, j) of the first rot values,
// c and s from a table of fp32 cosines and sines (a position's angle may be far from zero:
// whoever makes the table works it out in 64 bits). Keys: every product and sum of these lines
// is rounded by itself, and r is the fp32 value next to the exact one, so that a row's result
// depends on nothing but the row, and what the cache gets is bitwise what its append writes for
// rows rotated to fp32. (A code at the border of two would otherwise hang on the order of a sum.)
// Queries need no such care: plain fp32 sums and fused products, half of the instructions. All of it
// runs two values an instruction (fma2): append of 32,768 rows 46 us, one value 52.
//
// A group of d/16 lanes takes one row, a lane two words of 8 values that hold whole pairs:
// words l and l + rot/16 where halves are paired (the words past rot two by two), any where
// neighbours are. The floor is HBM: each row read once and written once. 16,384 tokens of 40 + 8
// heads of 128 in bf16 take 66 us, 6.2 TB/s, where a copy of as much takes 61: a group of lanes
// has four heads of a token in flight (two: 75 us; of fp32 rows two: 92 us, 6.7 TB/s, four 102). With
// the quantiser of the cache's append behind it those 46 us are 3.7 TB/s: 35.7 M instructions fill 63 % of
// the issue slots, DRAM is 37 % busy, and the 18 warps of an SM wait for results (1.6 cycles an issue) and loads (1.2).
#include <type_traits>

#include "w12_kv4_quant.cuh"

namespace w12 {
namespace kv4 {

// Small blocks, 100 registers a thread: 20 warps an SM with 128 bytes a thread in flight. Blocks of 256
// at 80 registers take 78 us where these take 68 (16,384 tokens, 40 + 8 heads of 128, bf16), 128
// registers 76, 72 86; without the loads' and stores' mark that memory is passed through once 74.
constexpr int kRopeThreads = 128, kRopeBlocks = 5;

struct RopeParams {
  const float* table;
  const float *qw, *kw;
  const int32_t *positions, *slots;
  int64_t n, max_pos;
  const void* x[3];            // Q, K, V
  int64_t tok[3], head[3];     // strides in elements
  int H[3];
  unsigned first[3];           // first block of the K rows, of the V rows, past the last
  void* out[2];                // Q, K
  uint8_t* pool;
  int64_t block;
  int n_pages, P, p_shift;
  int rot, pairs, out_type, vec;
  float eps, nz;               // nz: -0, see fma2
  int32_t* status;
};

// A sum of fp32 numbers as a pair, hi + lo. add() is off by 2^-48 of it where lo is small beside hi;
// join() makes that so, exactly: lo is then at most half a last place of hi.
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void join() {
    const float s = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(s, hi));
    hi = s;
  }
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
};

// Sum over the lanes of a row.
template <int kRow>
__device__ __forceinline__ float over_row(float v) {
#pragma unroll
  for (int o = kRow / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The sum of squares of a row that kRow lanes hold, in fp32 (about 2^-21 of it).
template <int kRow>
__device__ __forceinline__ float sum_squares(const float (&x)[16]) {
  float2 s[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
    s[i & 1] = fma2(v, v, s[i & 1]);
  }
  return over_row<kRow>(__fadd_rn(__fadd_rn(s[0].x, s[0].y), __fadd_rn(s[1].x, s[1].y)));
}

// The same as a pair, from that sum `rough`, which is finite. Each square is cut in two at 2^-16
// of the whole (of 2^e, the power of two below it): by a fused addition of c = 1.5 2^m (whose last
// place is 2^(m - 23)) the upper parts are whole multiples of it, and their sums exact in any order.
// The rests are at most 2^(e - 17) each, 2^(e - 10) together, so lo may be 2^-10 of hi. Their roundings: 128
// of a rest, in units of 2^(e - 41), and in the sums 35 for each lane's two runs of eight and 16 to join
// them (8 lanes), 3 times 128 over the lanes: 1200 in all, 2^-30.7 of the whole, half of that of the factor.
template <int kRow>
__device__ __forceinline__ Sum2 sum_squares2(const float (&x)[16], float rough) {
  const float c = __uint_as_float((__float_as_uint(rough) & 0x7F800000u) + (7u << 23) + 0x400000u);
  float2 hi = both(0.f), lo = both(0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
    const float2 less = fma2(fma2(v, v, both(c)), both(-1.f), both(c));  // minus the upper parts
    hi = fma2(less, both(-1.f), hi);
    lo = add2(lo, fma2(v, v, less));
  }
  return Sum2{over_row<kRow>(__fadd_rn(hi.x, hi.y)), over_row<kRow>(__fadd_rn(lo.x, lo.y))};
}

// fp32(1 / sqrt(m.hi + m.lo)), m joined: one step of Newton's iteration from the approximation, which
// is off by 2^-22 or so: the step leaves 2^-60 of r. Its residual 1 - m r^2 (2^-21 at most) is exact to 2^-43.
__device__ __forceinline__ float rsqrt_of(Sum2 m) {
  const float r = rsqrtf(m.hi);
  const float p = __fmul_rn(r, r), pe = fmaf(r, r, -p);
  const float t = __fmul_rn(m.hi, p), te = fmaf(m.hi, p, -t);
  float e = __fsub_rn(__fsub_rn(1.f, t), te);
  e = fmaf(-m.hi, pe, e);
  e = fmaf(-m.lo, p, e);
  return fmaf(r, e * fmaf(0.375f, e, 0.5f), r);
}

// The factor of a row's norm; kNearest: the fp32 value next to the exact one (before its rounding it is
// off by 2^-31.7 of itself, less than 2^-7 of the distance of two fp32 values, which is 2^-24 or more of
// them: so near the middle of two it is either). A row whose squares
// leave the fp32 range (values past 2^51) is made 2^76 smaller first: x then has what the factor
// is for, and the squares' sum is at most 2^111, below the 2^121 where c has no exponent left.
template <int kD, bool kNearest>
__device__ __forceinline__ float norm_factor(float (&x)[16], float eps) {
  constexpr int kRow = kD / 16;
  float rough = sum_squares<kRow>(x);
  const bool huge = !(rough < 1e35f);
  if (__any_sync(0xFFFFFFFFu, huge)) {
    const float scale = huge ? 0x1p-76f : 1.f;
    if (huge) eps = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], scale);
    rough = sum_squares<kRow>(x);
  }
  Sum2 s;
  if constexpr (kNearest) {
    s = sum_squares2<kRow>(x, rough < INFINITY ? rough : 0.f);
    s.join();
    s.hi *= 1.f / kD;
    s.lo *= 1.f / kD;
    s.add(eps);
  } else {
    s = Sum2{fmaf(rough, 1.f / kD, eps), 0.f};
  }
  // (The lanes of a row take one way: their rough sums are the same.)
  return rough < INFINITY ? rsqrt_of(s) : rough == INFINITY ? 0.f : NAN;
}

// What a lane's 16 values meet at a position: cosines and sines of their 8 pairs.
struct Turn {
  float c[8], s[8];
};

// Pairs of the lane's values and their cosines and sines. Halves paired: value i of word wa with
// value i of word wb; the table's place is that of wa. Neighbours paired: 2i and 2i + 1 of each
// word, the places those of both words.
__device__ __forceinline__ Turn load_turn(const float* tab, int wa, int wb, int rot, bool pairs) {
  Turn t;
  const int half = rot >> 1;
  const int at[2] = {pairs ? 4 * wa : 8 * wa, pairs ? 4 * wb : 8 * wa + 4};
  const bool in[2] = {pairs ? wa * 8 < rot : wb * 8 < rot, wb * 8 < rot};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
    if (in[k]) {
      c = *reinterpret_cast<const float4*>(tab + at[k]);
      s = *reinterpret_cast<const float4*>(tab + half + at[k]);
    }
    t.c[4 * k] = c.x, t.c[4 * k + 1] = c.y, t.c[4 * k + 2] = c.z, t.c[4 * k + 3] = c.w;
    t.s[4 * k] = s.x, t.s[4 * k + 1] = s.y, t.s[4 * k + 2] = s.z, t.s[4 * k + 3] = s.w;
  }
  return t;
}

// A pair turned; kEach: every product and sum rounded by itself.
template <bool kEach>
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float u = kEach ? __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)) : fmaf(-b, s, a * c);
  const float v = kEach ? __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)) : fmaf(a, s, b * c);
  a = u;
  b = v;
}

// Rotates the lane's 16 values x[0 .. 7] (word wa), x[8 .. 15] (wb); words past rot stay.
template <bool kEach>
__device__ __forceinline__ void rotate16(float (&x)[16], const Turn& t, bool in_a, bool in_b, bool pairs, float nz) {
  if (pairs) {
    if (in_a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn_pair<kEach>(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
    }
    if (in_b) {
#pragma unroll
      for (int i = 4; i < 8; ++i) turn_pair<kEach>(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
    }
  } else if (in_b) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[8 + i], x[9 + i]);
      const float2 c = make_float2(t.c[i], t.c[i + 1]), s = make_float2(t.s[i], t.s[i + 1]), less = make_float2(-s.x, -s.y);
      const float2 ac = fma2(a, c, both(nz)), bc = fma2(b, c, both(nz));
      const float2 u = kEach ? add2(ac, fma2(b, less, both(nz))) : fma2(b, less, ac);
      const float2 v = kEach ? add2(bc, fma2(a, s, both(nz))) : fma2(a, s, bc);
      x[i] = u.x, x[i + 1] = u.y;
      x[8 + i] = v.x, x[9 + i] = v.y;
    }
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 values to out + at, in the type W12_F32, W12_BF16 or W12_F16.
__device__ __forceinline__ void store8(void* out, int64_t at, int type, const float* x) {
  if (type == W12_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    __stcs(o, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(o + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    uint4 v;
    if (type == W12_BF16)
      v = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    else
      v = make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]), pack_f16x2(x[6], x[7]));
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at), v);
  }
}

// kHeads: heads of one token that a group of lanes takes one behind the other (weights and
// table are read once for all of them, and all their loads are in flight together). kPlain:
// queries go out in bf16, and all of a row is rotated by halves; the other cases are found as it runs.
template <int kD, typename E, bool kCache, int kHeads, bool kPlain>
__global__ void __launch_bounds__(kRopeThreads, kHeads == 1 ? 1 : kRopeBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRow = kD / 16;  // lanes of a row
  grid_dep_wait();
  grid_dep_launch();
  // A block's rows are all of one kind: 0 queries, 1 keys, 2 values.
  const int kind = blockIdx.x < p.first[0] ? 0 : (!kCache || blockIdx.x < p.first[1]) ? 1 : 2;
  const uint32_t base = blockIdx.x - (kind == 0 ? 0u : p.first[kind - 1]);
  const uint32_t unit = base * uint32_t(kRopeThreads / kRow) + threadIdx.x / kRow;
  const int l = threadIdx.x % kRow;
  const uint32_t H = uint32_t(p.H[kind]), groups = (H + kHeads - 1) / kHeads;
  const uint32_t tok = unit / groups, h0 = (unit - tok * groups) * kHeads;
  const bool live = tok < uint32_t(p.n);
  const int rot = kPlain ? kD : p.rot;
  const bool pairs = !kPlain && p.pairs;
  // The lane's two words.
  int wa = l, wb = l + kRow;
  const int R = rot >> 3;
  if (!kPlain && kind != 2 && !pairs && R < 2 * kRow) {
    wa = l < (R >> 1) ? l : R + 2 * (l - (R >> 1));
    wb = l < (R >> 1) ? l + (R >> 1) : wa + 1;
  }
  // (Past the last row or head the loads are the last one's again.)
  const uint32_t from = live ? tok : uint32_t(p.n) - 1;
  E a[kHeads], b[kHeads];
  const uint8_t* x0 = static_cast<const uint8_t*>(p.x[kind]) + int64_t(from) * p.tok[kind] * E::kSize;
  const int64_t step = p.head[kind] * E::kSize;
  if (p.vec) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const uint8_t* x = x0 + (kHeads == 1 ? h0 : min(h0 + k, H - 1)) * step;
      a[k] = load8<E, true, true>(x + wa * 8 * E::kSize);
      b[k] = load8<E, true, true>(x + wb * 8 * E::kSize);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const uint8_t* x = x0 + (kHeads == 1 ? h0 : min(h0 + k, H - 1)) * step;
      a[k] = load8<E, false>(x + wa * 8 * E::kSize);
      b[k] = load8<E, false>(x + wb * 8 * E::kSize);
    }
  }
  const int pos = p.positions[from], slot = kCache && live ? p.slots[from] : -1;
  const bool there = pos >= 0 && pos < p.max_pos;
  if (!there && pos != -1) set_status(p.status, W12_ERR_ARG);
  const int page = slot >> p.p_shift;
  const bool in = slot >= 0 && page < p.n_pages;
  if (kCache && !in && slot != -1) set_status(p.status, W12_ERR_ARG);
  const int r = slot & (p.P - 1), rr = kind == 2 ? p.P + r : r;
  // Where the row of head h of this token goes in the cache.
  auto keep = [&](uint32_t h, const uint3& q) {
    uint8_t* blk = p.pool + (int64_t(page) * p.H[1] + h) * p.block;
    uint8_t* codes = blk + rr * (kD / 2);
    *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, wa)) = q.x;
    *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, wb)) = q.y;
    if (l == 0) *reinterpret_cast<uint32_t*>(blk + p.P * kD + rr * 4) = q.z;
  };
  if (kCache && kind == 2) {
    if constexpr (kCache) {
#pragma unroll
      for (int k = 0; k < kHeads; ++k) {
        const uint3 q = quantise16<kRow, true>(a[k], b[k], p.nz);
        if (in && there && h0 + k < H) keep(h0 + k, q);
      }
    }
    return;
  }
  const bool in_a = kPlain || wa * 8 < rot, in_b = kPlain || wb * 8 < rot;
  const Turn turn = load_turn(p.table + int64_t(there ? pos : 0) * rot, wa, wb, rot, pairs);
  if (!there) {  // no token: zeros, whatever the rows hold
#pragma unroll
    for (int k = 0; k < kHeads; ++k) a[k] = b[k] = E{};
  }
  const float* w = kind ? p.kw : p.qw;
  float g[16];
  if (w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(w + (k < 2 ? wa * 8 + 4 * k : wb * 8 + 4 * (k - 2)));
      g[4 * k] = f.x, g[4 * k + 1] = f.y, g[4 * k + 2] = f.z, g[4 * k + 3] = f.w;
    }
  }
  auto row = [&](int k, auto is_key) {
    constexpr bool kKey = decltype(is_key)::value;
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = a[k].value(i);
      x[8 + i] = b[k].value(i);
    }
    if (w) {
      const float f = norm_factor<kD, kKey>(x, p.eps);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float2 y = fma2(fma2(make_float2(x[i], x[i + 1]), both(f), both(p.nz)), make_float2(g[i], g[i + 1]), both(p.nz));
        x[i] = y.x, x[i + 1] = y.y;
      }
    }
    rotate16<kKey>(x, turn, in_a, in_b, pairs, p.nz);
    const bool mine = kHeads == 1 || h0 + k < H;
    if constexpr (kCache && kKey) {
      F32 u, v;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u.w[i] = __float_as_uint(x[i]);
        v.w[i] = __float_as_uint(x[8 + i]);
      }
      const uint3 q = quantise16<kRow, true>(u, v, p.nz);
      if (in && there && mine) keep(h0 + k, q);
    } else if (live && mine) {
      const int64_t at = (int64_t(tok) * H + h0 + k) * kD;
      const int type = kCache || kPlain ? int(W12_BF16) : p.out_type;
      store8(p.out[kKey], at + wa * 8, type, x);
      store8(p.out[kKey], at + wb * 8, type, x + 8);
    }
  };
  if (kind == 0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) row(k, std::false_type());
  } else {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) row(k, std::true_type());
  }
}

// ---------------------------------------------------------------- positions
//
// A tree's depths by pointer jumping in shared memory: after step k a node knows the sum of
// its first 2^k steps up and the node where they end.
constexpr int kTreeThreads = 256;

struct PositionParams {
  const int32_t *prefix, *parents, *q_len;
  int32_t *out, *status;
  int T, blocks;
};

__global__ void __launch_bounds__(kTreeThreads) positions_kernel(const __grid_constant__ PositionParams p) {
  __shared__ int up[2][kTreeThreads], dist[2][kTreeThreads];
  __shared__ int bad;
  grid_dep_wait();
  grid_dep_launch();
  const int b = int(blockIdx.x / unsigned(p.blocks)), t = int(blockIdx.x % unsigned(p.blocks)) * kTreeThreads + threadIdx.x;
  const int64_t at = int64_t(b) * p.T + t;
  const int prefix = p.prefix[b];
  int n = p.q_len ? p.q_len[b] : p.T;
  const bool odd = n < 0 || n > p.T || prefix < 0 || int64_t(prefix) + n > (int64_t(1) << 31);
  if (odd) {
    if (threadIdx.x == 0) set_status(p.status, W12_ERR_ARG);
    n = 0;
  }
  int depth = t;
  if (p.parents) {  // T <= kTreeThreads: one block a tree
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int u = 0, d = 0;
    if (t < n) {
      u = p.parents[at];
      d = t > 0;
      if (t == 0 ? u != -1 : (u < 0 || u >= t)) bad = 1;
      if (t == 0) u = 0;
    }
    up[0][t] = u;
    dist[0][t] = d;
    __syncthreads();
    if (bad) {
      if (threadIdx.x == 0) set_status(p.status, W12_ERR_BAD_TREE);
      n = 0;
    } else {
      int k = 0;
      for (int reach = 1; reach < n; reach *= 2, k ^= 1) {
        const int v = up[k][t];
        up[k ^ 1][t] = up[k][v];
        dist[k ^ 1][t] = dist[k][t] + dist[k][v];
        __syncthreads();
      }
      depth = dist[k][t];
    }
  }
  if (t < p.T) p.out[at] = t < n ? prefix + depth : -1;
}

static cudaLaunchConfig_t config(unsigned grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cfg;
}

constexpr int kGroup = 4;  // heads of a group of lanes, where there are rows enough

// Of fp32 rows half as many: as many bytes in flight.
template <bool kCache, bool kGrouped, bool kPlain>
static cudaError_t launch_rope(const cudaLaunchConfig_t& cfg, const RopeParams& p, int d, int dtype) {
  constexpr int kWide = kGrouped ? kGroup : 1, kF32 = kGrouped ? kGroup / 2 : 1;
  if (d == 128)
    return dtype == W12_F32    ? cudaLaunchKernelEx(&cfg, rope_kernel<128, F32, kCache, kF32, kPlain>, p)
           : dtype == W12_BF16 ? cudaLaunchKernelEx(&cfg, rope_kernel<128, Half<true>, kCache, kWide, kPlain>, p)
                               : cudaLaunchKernelEx(&cfg, rope_kernel<128, Half<false>, kCache, kWide, kPlain>, p);
  return dtype == W12_F32    ? cudaLaunchKernelEx(&cfg, rope_kernel<64, F32, kCache, kF32, kPlain>, p)
         : dtype == W12_BF16 ? cudaLaunchKernelEx(&cfg, rope_kernel<64, Half<true>, kCache, kWide, kPlain>, p)
                             : cudaLaunchKernelEx(&cfg, rope_kernel<64, Half<false>, kCache, kWide, kPlain>, p);
}

// The launch over the rows that p names, by groups of heads where they fill the GPU.
template <bool kCache>
static int launch_rows(RopeParams p, int d, int dtype, void* stream) {
  const int units = kRopeThreads / (d / 16);  // of a block
  auto blocks = [&](int kind, int heads) -> int64_t {
    return p.x[kind] ? (p.n * ((p.H[kind] + heads - 1) / heads) + units - 1) / units : 0;
  };
  // Four blocks an SM of them: 2048 tokens, 40 + 8 heads of 128, bf16 8.5 us (single heads 12.2); with
  // two, 256 tokens fp32 into the cache 4.1 us (single heads 3.3).
  const int64_t few = 4 * int64_t(device_sm_count());
  const int group = dtype == W12_F32 ? kGroup / 2 : kGroup;
  const int heads = blocks(0, group) + blocks(1, group) + blocks(2, group) >= few ? group : 1;
  int64_t at = 0;
  for (int k = 0; k < 3; ++k) p.first[k] = unsigned(at += blocks(k, heads));
  const bool plain = p.rot == d && !p.pairs && (kCache || p.out_type == W12_BF16);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(unsigned(at), kRopeThreads, static_cast<cudaStream_t>(stream), attr);
  return cuda_status(heads == 1 ? launch_rope<kCache, false, false>(cfg, p, d, dtype)
                     : plain    ? launch_rope<kCache, true, true>(cfg, p, d, dtype)
                                : launch_rope<kCache, true, false>(cfg, p, d, dtype));
}

// The parts that both entry points check and fill in alike.
static int rope_params(const w12_rope* r, int d, int dtype, int64_t n, const int32_t* positions, int32_t* status, RopeParams* p) {
  if (!r || !positions || n < 0 || dtype < W12_F32 || dtype > W12_F16) return W12_ERR_ARG;
  if (!r->table || !aligned(r->table, 16) || (r->q_norm && !aligned(r->q_norm, 16)) || (r->k_norm && !aligned(r->k_norm, 16)))
    return W12_ERR_ARG;
  if ((r->q_norm || r->k_norm) && !(r->eps >= 1e-12f && r->eps < INFINITY)) return W12_ERR_ARG;
  if ((d != 64 && d != 128) || r->rot_dim < 16 || r->rot_dim > d || r->rot_dim % 16 || r->max_pos < 1 || r->max_pos > 0x7FFFFFFF)
    return W12_ERR_SHAPE;
  p->table = r->table;
  p->max_pos = r->max_pos;
  p->rot = r->rot_dim;
  p->pairs = r->interleaved != 0;
  p->qw = r->q_norm;
  p->kw = r->k_norm;
  p->eps = r->eps;
  p->nz = -0.f;
  p->positions = positions;
  p->n = n;
  p->status = status;
  return W12_OK;
}

// Rows of one kind: their strides and alignment.
static int rope_rows(RopeParams* p, int kind, const void* x, int64_t tok, int64_t head, int H, int esize, int64_t* strides) {
  p->H[kind] = H > 0 ? H : 1;
  if (!x) return W12_OK;
  if (!aligned(x, uintptr_t(esize))) return W12_ERR_ARG;
  if (H < 1 || H > 1024 || p->n > int64_t(0x7FFFFFFF) / H) return W12_ERR_SHAPE;
  p->x[kind] = x;
  p->tok[kind] = tok;
  p->head[kind] = head;
  *strides |= (tok | head) * esize | int64_t(reinterpret_cast<uintptr_t>(x) & 15);
  return W12_OK;
}

}  // namespace kv4
}  // namespace w12

using namespace w12;
using namespace w12::kv4;

extern "C" {

int w12_qk_norm_rope(const w12_rope* rope, int head_dim, const void* Q, int64_t q_token_stride, int64_t q_head_stride, int Hq,
                     const void* K, int64_t k_token_stride, int64_t k_head_stride, int Hkv, int dtype, int64_t n,
                     const int32_t* positions, void* Q_out, void* K_out, int out_dtype, int32_t* dev_status, void* stream) {
  RopeParams p{};
  int st = rope_params(rope, head_dim, dtype, n, positions, dev_status, &p);
  if (st) return st;
  if ((!Q && !K) || (Q && (!Q_out || !aligned(Q_out, 16))) || (K && (!K_out || !aligned(K_out, 16))) || out_dtype < W12_F32 ||
      out_dtype > W12_F16)
    return W12_ERR_ARG;
  const int esize = dtype == W12_F32 ? 4 : 2;
  int64_t strides = 0;
  if ((st = rope_rows(&p, 0, Q, q_token_stride, q_head_stride, Hq, esize, &strides)) ||
      (st = rope_rows(&p, 1, K, k_token_stride, k_head_stride, Hkv, esize, &strides)))
    return st;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  if (n == 0) return W12_OK;
  p.vec = strides % 16 == 0;
  p.out[0] = Q_out;
  p.out[1] = K_out;
  p.out_type = out_dtype;
  return launch_rows<false>(p, head_dim, dtype, stream);
}

int w12_kv4_append_rope(const w12_kv4* cache, const w12_rope* rope, const void* Q, int64_t q_token_stride, int64_t q_head_stride,
                        int Hq, const void* K, int64_t k_token_stride, int64_t k_head_stride, const void* V,
                        int64_t v_token_stride, int64_t v_head_stride, int dtype, int64_t n, const int32_t* positions,
                        const int32_t* slots, uint16_t* Q_out, int32_t* dev_status, void* stream) {
  RopeParams p{};
  if (!cache || !cache->pool || !slots || !aligned(cache->pool, 16)) return W12_ERR_ARG;
  if (!cache_ok(cache)) return W12_ERR_SHAPE;
  int st = rope_params(rope, cache->head_dim, dtype, n, positions, dev_status, &p);
  if (st) return st;
  if (!K || !V || (Q && (!Q_out || !aligned(Q_out, 16)))) return W12_ERR_ARG;
  const int esize = dtype == W12_F32 ? 4 : 2, d = cache->head_dim;
  int64_t strides = 0;
  if ((st = rope_rows(&p, 0, Q, q_token_stride, q_head_stride, Hq, esize, &strides)) ||
      (st = rope_rows(&p, 1, K, k_token_stride, k_head_stride, cache->Hkv, esize, &strides)) ||
      (st = rope_rows(&p, 2, V, v_token_stride, v_head_stride, cache->Hkv, esize, &strides)))
    return st;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  if (n == 0) return W12_OK;
  p.vec = strides % 16 == 0;
  p.out[0] = Q_out;
  p.slots = slots;
  p.pool = cache->pool;
  p.block = block_bytes(cache->page_size, d);
  p.n_pages = int(cache->n_pages);
  p.P = cache->page_size;
  p.p_shift = p.P == 16 ? 4 : p.P == 32 ? 5 : p.P == 64 ? 6 : 7;
  return launch_rows<true>(p, d, dtype, stream);
}

int w12_tree_positions(const int32_t* prefix_len, const int32_t* parents, const int32_t* q_len, int B, int T, int32_t* positions,
                       int32_t* dev_status, void* stream) {
  if (!prefix_len || !positions) return W12_ERR_ARG;
  if (B < 1 || T < 1 || (parents && T > kTreeMax) || B > 65535 || T > (1 << 23)) return W12_ERR_SHAPE;
  PositionParams p{prefix_len, parents, q_len, positions, dev_status, T, (T + kTreeThreads - 1) / kTreeThreads};
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  static_assert(kTreeMax == kTreeThreads, "one block a tree");
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(unsigned(B) * unsigned(p.blocks), kTreeThreads, static_cast<cudaStream_t>(stream), attr);
  return cuda_status(cudaLaunchKernelEx(&cfg, positions_kernel, p));
}

}  // extern "C"
