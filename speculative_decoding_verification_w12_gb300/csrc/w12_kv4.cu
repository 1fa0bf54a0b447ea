// Rows of the paged 4-bit cache: quantised writes, reads, and the commit of an
// accepted path. See w12_kv4.cuh for the layout.
//
// Quantiser, per (token, kv head) row of K and of V, all in fp32:
//   s = bf16(max/15 - min/15), z = bf16(min + 8 s),
//   q = clamp(round((x - z) / s) + 8, 0, 15), x ~ z + s (q - 8).
// The two roundings to bf16 come before the codes, which make up for them inside the
// range; at its ends a value is off by up to s/2, the rounding of z and 15 times that of s.
// So rows whose values are far from zero beside their spread keep them to about half a bf16
// step of z (spread 1 around 100: 0.9 s, around 1000: 3.2 s), as bf16 itself would. bf16
// keeps the range of any input. A row with a value that is not finite gets
// s = z = NaN: all of it reads as NaN. A scale below 2^-100 stores z alone.
//
// The floor of all three is HBM: append reads the input rows and writes d + 8
// bytes a (token, head), read the reverse. In append a group of d/8 lanes takes one
// (token, head), half of it K and half V, and a lane two code words (8 dims each) of
// its row, one in each half of the row: loads and stores are contiguous over the
// lanes, and a row's scale is worked out by d/16 lanes only (by d/8, each with a word of
// K and one of V as in read, 40.5 us where it is 36.7). Indices are 32-bit: a 64-bit
// division a row costs more than the quantiser.
//
// 28,305 tokens of 8 heads x 128 in bf16 (4 requests): append 36.7 us, 4.0 TB/s of
// the 147 MB it has to move, 59 % of a copy's rate, held back by the issue of about
// 260 instructions a lane; read 32.7 us, 4.5 TB/s, most of it writes (halving its
// arithmetic changed nothing). A tree's 256 tokens take 1.7 us (append), 3.4 us (commit)
// and 1.7 us (read), which is launch latency.
#include "w12_kv4.cuh"

namespace w12 {
namespace kv4 {

constexpr int kRowThreads = 256;

struct RowParams {
  uint8_t* pool;
  int64_t block;  // bytes of a (page, kv head) block
  int n_pages, Hkv, P, p_shift;
  const void *K, *V;
  int64_t k_tok, k_head, v_tok, v_head;  // strides in elements
  uint16_t *Ko, *Vo;
  const int32_t* slots;
  int64_t n;
  int32_t* status;
};

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

template <typename E, bool kVec>
__device__ __forceinline__ E load8(const uint8_t* p) {
  E e;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < int(sizeof(E) / 16); ++i)
      reinterpret_cast<uint4*>(e.w)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
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

// The lane's two code words and its row's parameter word (z). Most rows have no code
// outside -8 .. 7 (their centre's rounding is far below a step), and a warp of such
// rows saves the clamps, a third of its work an element.
template <int kLanes, typename E>
__device__ __forceinline__ uint3 quantise16(const E& a, const E& b) {
  const RowScale r = row_scale<kLanes>(a, b);
  uint3 q;
  if (__all_sync(0xFFFFFFFFu, r.inside)) {
    q.x = code_word<false>(a, r);
    q.y = code_word<false>(b, r);
  } else {
    q.x = code_word<true>(a, r);
    q.y = code_word<true>(b, r);
  }
  q.z = r.par;
  return r.finite ? q : make_uint3(0x88888888u, 0x88888888u, 0x7FC07FC0u);
}

template <int kD, typename E, bool kVec>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const __grid_constant__ RowParams p) {
  constexpr int kLanes = kD / 8;
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t unit = blockIdx.x * uint32_t(kRowThreads / kLanes) + threadIdx.x / kLanes;  // < 2^31 + a CTA's
  constexpr int kRow = kLanes / 2;  // lanes of a row
  const int w = threadIdx.x % kRow;
  const bool is_v = threadIdx.x & kRow;
  const uint32_t tok = unit / uint32_t(p.Hkv), h = unit - tok * uint32_t(p.Hkv);
  const bool live = tok < uint32_t(p.n);
  // The inputs do not wait for the slot: all loads are in flight together.
  E a{}, b{};
  int slot = -1;
  if (live) {
    const int64_t at = int64_t(tok) * (is_v ? p.v_tok : p.k_tok) + int64_t(h) * (is_v ? p.v_head : p.k_head) + w * 8;
    const uint8_t* x = static_cast<const uint8_t*>(is_v ? p.V : p.K) + at * E::kSize;
    a = load8<E, kVec>(x);
    b = load8<E, kVec>(x + kRow * 8 * E::kSize);
    slot = p.slots[tok];
  }
  const int page = slot >> p.p_shift;
  const bool in = slot >= 0 && page < p.n_pages;
  if (!in && slot != -1) set_status(p.status, W12_ERR_ARG);
  const uint3 q = quantise16<kRow>(a, b);
  if (!in) return;
  const int r = slot & (p.P - 1);
  uint8_t* blk = p.pool + (int64_t(page) * p.Hkv + h) * p.block;
  uint8_t* codes = blk + (is_v ? p.P + r : r) * (kD / 2);
  *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, w)) = q.x;
  *reinterpret_cast<uint32_t*>(codes + word_off(kD, r, w + kRow)) = q.y;
  if (w == 0) *reinterpret_cast<uint32_t*>(blk + p.P * kD + (is_v ? p.P + r : r) * 4) = q.z;
}

template <int kD>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const __grid_constant__ RowParams p) {
  constexpr int kLanes = kD / 8;
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t unit = blockIdx.x * uint32_t(kRowThreads / kLanes) + threadIdx.x / kLanes;
  const int w = threadIdx.x % kLanes;
  const uint32_t tok = unit / uint32_t(p.Hkv), h = unit - tok * uint32_t(p.Hkv);
  if (tok >= uint32_t(p.n)) return;
  const int slot = p.slots[tok];
  const int page = slot >> p.p_shift;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (slot >= 0 && page < p.n_pages) {
    const int r = slot & (p.P - 1);
    const uint8_t* blk = p.pool + (int64_t(page) * p.Hkv + h) * p.block;
    const uint8_t* codes = blk + r * (kD / 2) + word_off(kD, r, w);
    const uint32_t* par = reinterpret_cast<const uint32_t*>(blk + p.P * kD) + r;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(codes);
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(codes + p.P * (kD / 2));
    const uint32_t kp = par[0], vp = par[p.P];
    uint32_t *ko = &k.x, *vo = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = value_pair(kw, j, bf16_lo(kp), bf16_hi(kp)), b = value_pair(vw, j, bf16_lo(vp), bf16_hi(vp));
      ko[j] = pack_bf16x2(a.x, a.y);
      vo[j] = pack_bf16x2(b.x, b.y);
    }
  } else if (slot != -1) {
    set_status(p.status, W12_ERR_ARG);
  }
  const int64_t at = int64_t(unit) * kD + w * 8;
  *reinterpret_cast<uint4*>(p.Ko + at) = k;
  *reinterpret_cast<uint4*>(p.Vo + at) = v;
}

// ------------------------------------------------------------------- commit
//
// One thread per 16-byte piece of the codes (or 4-byte parameter word) of one
// (cache, request, kv head). Like the dense commit: path[k] >= k, so a row is
// never read after an earlier step of the path overwrote it, and no other
// thread touches the piece. The loads of up to kBatch steps are in flight
// together before their stores.
constexpr int kCommitThreads = 128;
constexpr int kCommitCaches = 64;
constexpr int kBatch = 8;

struct CommitParams {
  uint8_t* pools[kCommitCaches];
  int64_t n_pages, block;
  int n_caches, B, Hkv, P, p_shift, max_pages, path_stride, first;
  const int32_t *table, *prefix_len, *path, *path_len;
  int32_t* new_len;
  int32_t* status;
};

template <int kD>
__global__ void __launch_bounds__(kCommitThreads) kv4_commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int kPieces = kD / 2 / 16;     // 16-byte pieces of a row's codes
  constexpr int kCols = 2 * kPieces + 2;   // K codes, V codes, K and V parameters
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.y, ci = blockIdx.z;
  const int col = blockIdx.x * kCommitThreads + threadIdx.x;
  const int32_t* path = p.path + int64_t(b) * p.path_stride;
  const int32_t* tab = p.table + int64_t(b) * p.max_pages;
  const int64_t P0 = p.prefix_len[b];
  const int n = p.path_len[b];
  // Validity of the path: increasing, and every row on a page of the pool.
  // Rows prefix .. prefix + path[n - 1] cover all that the commit touches.
  bool ok = n >= 1 && n <= p.path_stride && P0 >= 0;
  int last = -1;
  for (int k = 0; ok && k < n; ++k) {
    const int v = path[k];
    ok = v > last && ((P0 + v) >> p.p_shift) < p.max_pages;
    if (ok) {
      const int ps = tab[(P0 + v) >> p.p_shift], pd = tab[(P0 + k) >> p.p_shift];
      ok = ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages;
    }
    last = v;
  }
  if (blockIdx.x == 0 && ci == 0 && threadIdx.x == 0 && p.first) {
    if (!ok) set_status(p.status, W12_ERR_BAD_TREE);
    if (p.new_len) p.new_len[b] = int32_t(ok ? P0 + n : P0);
  }
  if (!ok || col >= p.Hkv * kCols) return;
  const int h = col / kCols, c = col - h * kCols;
  uint8_t* pool = p.pools[ci] + int64_t(h) * p.block;
  const int64_t page_stride = int64_t(p.Hkv) * p.block;
  auto at = [&](int64_t pos) -> uint8_t* {
    const int r = int(pos & (p.P - 1));
    uint8_t* blk = pool + int64_t(tab[pos >> p.p_shift]) * page_stride;
    if (c >= 2 * kPieces) return blk + p.P * kD + ((c - 2 * kPieces) * p.P + r) * 4;
    const int which = c >= kPieces, piece = c - which * kPieces;
    return blk + (which * p.P + r) * (kD / 2) + word_off(kD, r, piece * 4);
  };
  const bool wide = c < 2 * kPieces;
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (k0 + i < n) {
        const uint8_t* src = at(P0 + path[k0 + i]);
        if (wide) v[i] = *reinterpret_cast<const uint4*>(src);
        else v[i].x = *reinterpret_cast<const uint32_t*>(src);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (k0 + i < n && path[k0 + i] != k0 + i) {
        uint8_t* dst = at(P0 + k0 + i);
        if (wide) *reinterpret_cast<uint4*>(dst) = v[i];
        else *reinterpret_cast<uint32_t*>(dst) = v[i].x;
      }
  }
}

static int log2_of(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : 7; }

static cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cfg;
}

template <int kD, typename E>
static cudaError_t launch_append(const cudaLaunchConfig_t& cfg, const RowParams& p, bool vec) {
  return vec ? cudaLaunchKernelEx(&cfg, kv4_append_kernel<kD, E, true>, p)
             : cudaLaunchKernelEx(&cfg, kv4_append_kernel<kD, E, false>, p);
}

template <int kD>
static cudaError_t launch_append(const cudaLaunchConfig_t& cfg, const RowParams& p, int dtype, bool vec) {
  return dtype == W12_F32    ? launch_append<kD, F32>(cfg, p, vec)
         : dtype == W12_BF16 ? launch_append<kD, Half<true>>(cfg, p, vec)
                             : launch_append<kD, Half<false>>(cfg, p, vec);
}

static int row_params(const w12_kv4* c, const int32_t* slots, int64_t n, int32_t* status, RowParams* p) {
  if (!c || !c->pool || !slots || n < 0 || !aligned(c->pool, 16)) return W12_ERR_ARG;
  if (!cache_ok(c) || n > int64_t(0x7FFFFFFF) / c->Hkv) return W12_ERR_SHAPE;
  p->pool = c->pool;
  p->n_pages = int(c->n_pages);
  p->block = block_bytes(c->page_size, c->head_dim);
  p->Hkv = c->Hkv;
  p->P = c->page_size;
  p->p_shift = log2_of(c->page_size);
  p->slots = slots;
  p->n = n;
  p->status = status;
  return W12_OK;
}

}  // namespace kv4
}  // namespace w12

using namespace w12;
using namespace w12::kv4;

extern "C" {

int64_t w12_kv4_page_bytes(int Hkv, int head_dim, int page_size) {
  const w12_kv4 c{nullptr, 1, Hkv, head_dim, page_size};
  return cache_ok(&c) ? Hkv * block_bytes(page_size, head_dim) : 0;
}

int w12_kv4_append(const w12_kv4* cache, const void* K, const void* V, int dtype, int64_t n, int64_t k_token_stride,
                   int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                   int32_t* dev_status, void* stream) {
  RowParams p{};
  const int st = row_params(cache, slots, n, dev_status, &p);
  if (st) return st;
  if (!K || !V || dtype < W12_F32 || dtype > W12_F16) return W12_ERR_ARG;
  const int esize = dtype == W12_F32 ? 4 : 2;
  if (!aligned(K, esize) || !aligned(V, esize)) return W12_ERR_ARG;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  if (n == 0) return W12_OK;
  p.K = K;
  p.V = V;
  p.k_tok = k_token_stride;
  p.k_head = k_head_stride;
  p.v_tok = v_token_stride;
  p.v_head = v_head_stride;
  const int64_t all = (k_token_stride | k_head_stride | v_token_stride | v_head_stride) * esize;
  const bool vec = aligned(K, 16) && aligned(V, 16) && all % 16 == 0;
  const int64_t threads = n * p.Hkv * (cache->head_dim / 8);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(dim3(unsigned((threads + kRowThreads - 1) / kRowThreads)), kRowThreads,
                                        static_cast<cudaStream_t>(stream), attr);
  return cuda_status(cache->head_dim == 128 ? launch_append<128>(cfg, p, dtype, vec)
                                            : launch_append<64>(cfg, p, dtype, vec));
}

int w12_kv4_read(const w12_kv4* cache, const int32_t* slots, int64_t n, uint16_t* K_out, uint16_t* V_out,
                 int32_t* dev_status, void* stream) {
  RowParams p{};
  const int st = row_params(cache, slots, n, dev_status, &p);
  if (st) return st;
  if (!K_out || !V_out || !aligned(K_out, 16) || !aligned(V_out, 16)) return W12_ERR_ARG;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  if (n == 0) return W12_OK;
  p.Ko = K_out;
  p.Vo = V_out;
  const int64_t threads = n * p.Hkv * (cache->head_dim / 8);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(dim3(unsigned((threads + kRowThreads - 1) / kRowThreads)), kRowThreads,
                                        static_cast<cudaStream_t>(stream), attr);
  return cuda_status(cache->head_dim == 128 ? cudaLaunchKernelEx(&cfg, kv4_read_kernel<128>, p)
                                            : cudaLaunchKernelEx(&cfg, kv4_read_kernel<64>, p));
}

int w12_kv4_commit(const w12_kv4* caches, int n_caches, int B, const int32_t* table, int max_pages,
                   const int32_t* prefix_len, const int32_t* path, int path_stride, const int32_t* path_len,
                   int32_t* new_len, int32_t* dev_status, void* stream) {
  if (!caches || n_caches < 1 || B < 1 || B > 65535 || !table || max_pages < 1 || !prefix_len || !path ||
      path_stride < 1 || !path_len)
    return W12_ERR_ARG;
  const w12_kv4& c0 = caches[0];
  for (int i = 0; i < n_caches; ++i) {
    const w12_kv4& c = caches[i];
    if (!c.pool || !aligned(c.pool, 16)) return W12_ERR_ARG;
    if (!cache_ok(&c) || c.n_pages != c0.n_pages || c.Hkv != c0.Hkv || c.head_dim != c0.head_dim ||
        c.page_size != c0.page_size)
      return W12_ERR_SHAPE;
  }
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  const int cols = c0.Hkv * (c0.head_dim / 16 + 2);
  for (int i0 = 0; i0 < n_caches; i0 += kCommitCaches) {
    CommitParams p{};
    p.n_caches = n_caches - i0 < kCommitCaches ? n_caches - i0 : kCommitCaches;
    for (int i = 0; i < p.n_caches; ++i) p.pools[i] = caches[i0 + i].pool;
    p.n_pages = c0.n_pages;
    p.block = block_bytes(c0.page_size, c0.head_dim);
    p.B = B;
    p.Hkv = c0.Hkv;
    p.P = c0.page_size;
    p.p_shift = log2_of(c0.page_size);
    p.max_pages = max_pages;
    p.path_stride = path_stride;
    p.first = i0 == 0;
    p.table = table;
    p.prefix_len = prefix_len;
    p.path = path;
    p.path_len = path_len;
    p.new_len = new_len;
    p.status = dev_status;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        config(dim3(unsigned((cols + kCommitThreads - 1) / kCommitThreads), unsigned(B), unsigned(p.n_caches)),
               kCommitThreads, static_cast<cudaStream_t>(stream), attr);
    const int st = cuda_status(c0.head_dim == 128 ? cudaLaunchKernelEx(&cfg, kv4_commit_kernel<128>, p)
                                                  : cudaLaunchKernelEx(&cfg, kv4_commit_kernel<64>, p));
    if (st) return st;
  }
  return W12_OK;
}

}  // extern "C"
