// Norms of query and key heads with the rotation by position, in one pass; the same on the
// way into the paged 4-bit cache; positions of a draft tree's nodes.
//
// A head's row x of d values, normed (weights w) and rotated by its token's position:
//   y_i  = (x_i r) w_i,  r = fp32(1 / sqrt(mean x^2 + eps))
//   y_i' = y_i c - y_j s,  y_j' = y_j c + y_i s   for the pairs (i, j) of the first rot values,
// c and s from a table of fp32 cosines and sines (a position's angle may be far from zero:
// whoever makes the table works it out in 64 bits). Every product and sum of these lines is
// rounded by itself, and r is the fp32 value next to the exact one (the sum of squares is
// kept as a pair of fp32 numbers): so a row's result depends on nothing but the row, and
// what the cache gets is bitwise what its append writes for rows rotated to fp32. A code at
// the border of two would otherwise hang on the order of a sum.
//
// A group of d/16 lanes takes one row, a lane two words of 8 values that hold whole pairs:
// words l and l + rot/16 where halves are paired (the words past rot two by two), any where
// neighbours are. The floor is HBM: each row read once and written once.
#include "w12_kv4_quant.cuh"

namespace w12 {
namespace kv4 {

constexpr int kRopeThreads = 256;

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
  float eps;
  int32_t* status;
};

// Sum of fp32 numbers as a pair: hi + lo is the sum to about 2^-46 of it.
struct Sum2 {
  float hi, lo;
  // (The same for a + b as for b + a: lanes that join their sums get one result.)
  __device__ __forceinline__ void add(float x, float e) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    const float off = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
    hi = s;
    lo = __fadd_rn(__fadd_rn(lo, e), off);
  }
};

// Sum of squares of a row that kLanes lanes hold, 16 values each, times 2^(2 down).
template <int kLanes>
__device__ __forceinline__ Sum2 sum_squares(const float (&x)[16], float scale) {
  Sum2 s{0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = __fmul_rn(x[i], scale), p = __fmul_rn(v, v);
    s.add(p, fmaf(v, v, -p));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xFFFFFFFFu, s.hi, o), l = __shfl_xor_sync(0xFFFFFFFFu, s.lo, o);
    s.add(h, l);
  }
  return s;
}

// fp32(1 / sqrt(m.hi + m.lo)): one step of Newton's iteration from the approximation, its
// residual 1 - m r^2 exact to about 2^-46.
__device__ __forceinline__ float rsqrt_of(Sum2 m) {
  const float r = rsqrtf(m.hi);
  const float p = __fmul_rn(r, r), pe = fmaf(r, r, -p);
  const float t = __fmul_rn(m.hi, p), te = fmaf(m.hi, p, -t);
  float e = __fsub_rn(__fsub_rn(1.f, t), te);
  e = fmaf(-m.hi, pe, e);
  e = fmaf(-m.lo, p, e);
  return fmaf(r, e * fmaf(0.375f, e, 0.5f), r);
}

// The factor of a row's norm. Rows whose squares leave the fp32 range (values near 2^64) are
// summed again 2^70 smaller.
template <int kD>
__device__ __forceinline__ float norm_factor(const float (&x)[16], float eps) {
  constexpr int kLanes = kD / 16;
  Sum2 s = sum_squares<kLanes>(x, 1.f);
  float up = 1.f;
  const bool huge = !(s.hi < 1e37f);
  if (__any_sync(0xFFFFFFFFu, huge)) {
    const Sum2 t = sum_squares<kLanes>(x, 0x1p-70f);
    if (huge) {
      s = t;
      up = 0x1p-70f;
      eps = 0.f;
    }
  }
  s.hi *= 1.f / kD;
  s.lo *= 1.f / kD;
  if (!(s.hi < INFINITY)) return s.hi == INFINITY ? 0.f : NAN;
  s.add(eps, 0.f);
  return __fmul_rn(rsqrt_of(s), up);
}

// Rotates the lane's words (see the top). tab: the position's row of the table.
__device__ __forceinline__ void rotate16(float (&x)[16], const float* tab, int wa, int wb, int rot, bool pairs) {
  const int half = rot >> 1;
  if (pairs) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = k ? wb : wa;
      if (w * 8 < rot) {
        const float4 c4 = *reinterpret_cast<const float4*>(tab + 4 * w), s4 = *reinterpret_cast<const float4*>(tab + half + 4 * w);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[8 * k + 2 * i], b = x[8 * k + 2 * i + 1];
          x[8 * k + 2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
          x[8 * k + 2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
      }
    }
  } else if (wb * 8 < rot) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c4 = *reinterpret_cast<const float4*>(tab + 8 * wa + 4 * k),
                   s4 = *reinterpret_cast<const float4*>(tab + half + 8 * wa + 4 * k);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[4 * k + i], b = x[8 + 4 * k + i];
        x[4 * k + i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
        x[8 + 4 * k + i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
      }
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
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    const bool b = type == W12_BF16;
    uint4 v;
    v.x = b ? pack_bf16x2(x[0], x[1]) : pack_f16x2(x[0], x[1]);
    v.y = b ? pack_bf16x2(x[2], x[3]) : pack_f16x2(x[2], x[3]);
    v.z = b ? pack_bf16x2(x[4], x[5]) : pack_f16x2(x[4], x[5]);
    v.w = b ? pack_bf16x2(x[6], x[7]) : pack_f16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = v;
  }
}

template <int kD, typename E, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kRow = kD / 16;  // lanes of a row
  grid_dep_wait();
  grid_dep_launch();
  // A block's rows are all of one kind: 0 queries, 1 keys, 2 values.
  const int kind = blockIdx.x < p.first[0] ? 0 : (!kCache || blockIdx.x < p.first[1]) ? 1 : 2;
  const uint32_t base = blockIdx.x - (kind == 0 ? 0u : p.first[kind - 1]);
  const uint32_t row = base * uint32_t(kRopeThreads / kRow) + threadIdx.x / kRow;
  const int l = threadIdx.x % kRow;
  const uint32_t H = uint32_t(p.H[kind]);
  const uint32_t tok = row / H, h = row - tok * H;
  const bool live = tok < uint32_t(p.n);
  const bool turns = kind != 2;
  // The lane's two words.
  int wa = l, wb = l + kRow;
  const int R = p.rot >> 3;
  if (turns && !p.pairs && R < 2 * kRow) {
    wa = l < (R >> 1) ? l : R + 2 * (l - (R >> 1));
    wb = l < (R >> 1) ? l + (R >> 1) : wa + 1;
  }
  E a{}, b{};
  int pos = -1, slot = -1;
  if (live) {
    const uint8_t* x = static_cast<const uint8_t*>(p.x[kind]) + (int64_t(tok) * p.tok[kind] + int64_t(h) * p.head[kind]) * E::kSize;
    if (p.vec) {
      a = load8<E, true>(x + wa * 8 * E::kSize);
      b = load8<E, true>(x + wb * 8 * E::kSize);
    } else {
      a = load8<E, false>(x + wa * 8 * E::kSize);
      b = load8<E, false>(x + wb * 8 * E::kSize);
    }
    pos = p.positions[tok];
    if (kCache) slot = p.slots[tok];
  }
  const bool there = pos >= 0 && pos < p.max_pos;
  if (!there && pos != -1) set_status(p.status, W12_ERR_ARG);
  uint3 q{};
  if (kCache && kind == 2) {
    if constexpr (kCache) q = quantise16<kRow>(a, b);
  } else {
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = a.value(i);
      x[8 + i] = b.value(i);
    }
    const float* w = kind ? p.kw : p.qw;
    if (w) {
      const float r = norm_factor<kD>(x, p.eps);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 g = *reinterpret_cast<const float4*>(w + (k < 2 ? wa * 8 + 4 * k : wb * 8 + 4 * (k - 2)));
        x[4 * k] = __fmul_rn(__fmul_rn(x[4 * k], r), g.x);
        x[4 * k + 1] = __fmul_rn(__fmul_rn(x[4 * k + 1], r), g.y);
        x[4 * k + 2] = __fmul_rn(__fmul_rn(x[4 * k + 2], r), g.z);
        x[4 * k + 3] = __fmul_rn(__fmul_rn(x[4 * k + 3], r), g.w);
      }
    }
    if (there) {
      rotate16(x, p.table + int64_t(pos) * p.rot, wa, wb, p.rot, p.pairs);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    if (!kCache || kind == 0) {
      if (live) {
        const int64_t at = int64_t(row) * kD;
        const int type = kCache ? int(W12_BF16) : p.out_type;
        store8(p.out[kind], at + wa * 8, type, x);
        store8(p.out[kind], at + wb * 8, type, x + 8);
      }
      return;
    }
    if constexpr (kCache) {
      F32 u, v;
      for (int i = 0; i < 8; ++i) {
        u.w[i] = __float_as_uint(x[i]);
        v.w[i] = __float_as_uint(x[8 + i]);
      }
      q = quantise16<kRow>(u, v);
    }
  }
  const int page = slot >> p.p_shift;
  const bool in = slot >= 0 && page < p.n_pages;
  if (!in && slot != -1) set_status(p.status, W12_ERR_ARG);
  if (!in || !there) return;
  const int r = slot & (p.P - 1);
  uint8_t* blk = p.pool + (int64_t(page) * p.H[1] + h) * p.block;
  const int rr = kind == 2 ? p.P + r : r;
  uint8_t* codes = blk + rr * (kD / 2);
  *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, wa)) = q.x;
  *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, wb)) = q.y;
  if (l == 0) *reinterpret_cast<uint32_t*>(blk + p.P * kD + rr * 4) = q.z;
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

template <bool kCache>
static cudaError_t launch_rope(const cudaLaunchConfig_t& cfg, const RopeParams& p, int d, int dtype) {
  if (d == 128)
    return dtype == W12_F32    ? cudaLaunchKernelEx(&cfg, rope_kernel<128, F32, kCache>, p)
           : dtype == W12_BF16 ? cudaLaunchKernelEx(&cfg, rope_kernel<128, Half<true>, kCache>, p)
                               : cudaLaunchKernelEx(&cfg, rope_kernel<128, Half<false>, kCache>, p);
  return dtype == W12_F32    ? cudaLaunchKernelEx(&cfg, rope_kernel<64, F32, kCache>, p)
         : dtype == W12_BF16 ? cudaLaunchKernelEx(&cfg, rope_kernel<64, Half<true>, kCache>, p)
                             : cudaLaunchKernelEx(&cfg, rope_kernel<64, Half<false>, kCache>, p);
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
  p->positions = positions;
  p->n = n;
  p->status = status;
  return W12_OK;
}

// Rows of one kind: their strides, alignment and blocks.
static int rope_rows(RopeParams* p, int kind, const void* x, int64_t tok, int64_t head, int H, int d, int esize, int64_t* blocks,
                     int64_t* strides) {
  *blocks = 0;
  p->H[kind] = H > 0 ? H : 1;
  if (!x) return W12_OK;
  if (!aligned(x, uintptr_t(esize))) return W12_ERR_ARG;
  if (H < 1 || H > 1024 || p->n > int64_t(0x7FFFFFFF) / H) return W12_ERR_SHAPE;
  p->x[kind] = x;
  p->tok[kind] = tok;
  p->head[kind] = head;
  *strides |= (tok | head) * esize | int64_t(reinterpret_cast<uintptr_t>(x) & 15);
  const int rows = kRopeThreads / (d / 16);
  *blocks = (p->n * H + rows - 1) / rows;
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
  int64_t nq, nk, strides = 0;
  if ((st = rope_rows(&p, 0, Q, q_token_stride, q_head_stride, Hq, head_dim, esize, &nq, &strides)) ||
      (st = rope_rows(&p, 1, K, k_token_stride, k_head_stride, Hkv, head_dim, esize, &nk, &strides)))
    return st;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  if (n == 0) return W12_OK;
  p.vec = strides % 16 == 0;
  p.out[0] = Q_out;
  p.out[1] = K_out;
  p.out_type = out_dtype;
  p.first[0] = unsigned(nq);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(unsigned(nq + nk), kRopeThreads, static_cast<cudaStream_t>(stream), attr);
  return cuda_status(launch_rope<false>(cfg, p, head_dim, dtype));
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
  int64_t nq, nk, nv, strides = 0;
  if ((st = rope_rows(&p, 0, Q, q_token_stride, q_head_stride, Hq, d, esize, &nq, &strides)) ||
      (st = rope_rows(&p, 1, K, k_token_stride, k_head_stride, cache->Hkv, d, esize, &nk, &strides)) ||
      (st = rope_rows(&p, 2, V, v_token_stride, v_head_stride, cache->Hkv, d, esize, &nv, &strides)))
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
  p.first[0] = unsigned(nq);
  p.first[1] = unsigned(nq + nk);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(unsigned(nq + nk + nv), kRopeThreads, static_cast<cudaStream_t>(stream), attr);
  return cuda_status(launch_rope<true>(cfg, p, d, dtype));
}

int w12_tree_positions(const int32_t* prefix_len, const int32_t* parents, const int32_t* q_len, int B, int T, int32_t* positions,
                       int32_t* dev_status, void* stream) {
  if (!prefix_len || !positions) return W12_ERR_ARG;
  if (B < 1 || T < 1 || (parents && T > kTreeMax) || B > 65535) return W12_ERR_SHAPE;
  PositionParams p{prefix_len, parents, q_len, positions, dev_status, T, (T + kTreeThreads - 1) / kTreeThreads};
  if (int64_t(B) * p.blocks > 0x7FFFFFFF) return W12_ERR_SHAPE;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  static_assert(kTreeMax == kTreeThreads, "one block a tree");
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(unsigned(B) * unsigned(p.blocks), kTreeThreads, static_cast<cudaStream_t>(stream), attr);
  return cuda_status(cudaLaunchKernelEx(&cfg, positions_kernel, p));
}

}  // extern "C"
