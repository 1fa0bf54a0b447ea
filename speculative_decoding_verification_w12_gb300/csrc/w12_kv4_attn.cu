// Attention over the paged 4-bit cache: simple form, one warp per query row.
#include <algorithm>

#include "w12_kv4_rows.cuh"

namespace w12 {
namespace kv4_attn {

constexpr int kWarps = 4;

template <int kD>
__global__ void __launch_bounds__(kWarps * 32) kv4_attn_simple_kernel(const __grid_constant__ Params p) {
  __shared__ float qs[kWarps][kD];
  constexpr int kPer = kD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t rows = int64_t(p.B) * p.T * p.Hq;
  const int64_t row = int64_t(blockIdx.x) * kWarps + warp;
  if (row >= rows) return;
  const int hq = int(row % p.Hq), t = int((row / p.Hq) % p.T), b = int(row / (int64_t(p.Hq) * p.T));
  const int h = hq / p.G;
  int n = p.q_len ? p.q_len[b] : p.T, a = p.prefix_len[b];
  if (n < 0 || n > p.T || a < 0 || a > p.max_len - n) {
    set_status(p.status, W12_ERR_ARG);
    n = min(max(n, 0), p.T);
    a = min(max(a, 0), p.max_len - n);
  }
  uint16_t* o = p.O + row * kD;
  if (t >= n) {
    for (int i = lane; i < kD; i += 32) o[i] = 0;
    return;
  }
  const uint16_t* q = p.Q + b * p.q_b + t * p.q_t + hq * p.q_h;
  for (int i = lane; i < kD; i += 32) qs[warp][i] = __uint_as_float(uint32_t(q[i]) << 16);
  __syncwarp();
  const int32_t* par = p.parents ? p.parents + int64_t(b) * p.T : nullptr;
  uint32_t anc[kMaxTree / 32] = {0, 0, 0, 0};
  if (par) {
    bool bad = false;
    for (int i = 0; i < p.T; ++i) bad |= i == 0 ? par[0] != -1 : (par[i] < 0 || par[i] >= i);
    if (bad) set_status(p.status, W12_ERR_BAD_TREE);
    for (int i = t; i >= 0; i = bad ? -1 : par[i]) anc[i >> 5] |= 1u << (i & 31);
  }
  const int keys = par ? a + n : a + t + 1;
  float m = -INFINITY, l = 0.f, acc[kPer];
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < keys; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < keys && (!par || j < a || ((anc[(j - a) >> 5] >> ((j - a) & 31)) & 1u));
    const uint8_t* blk = nullptr;
    const int r = j & (p.P - 1);
    if (see) {
      const int page = p.table[int64_t(b) * p.max_pages + (j >> p.p_shift)];
      if (page < 0 || page >= p.n_pages) {
        set_status(p.status, W12_ERR_ARG);
        see = false;
      } else {
        blk = p.pool + (int64_t(page) * p.Hkv + h) * p.block;
      }
    }
    float x = -INFINITY, vs = 0.f, vz = 0.f;
    if (see) {
      const uint32_t kp = *reinterpret_cast<const uint32_t*>(blk + p.P * kD + r * 4);
      const uint32_t vp = *reinterpret_cast<const uint32_t*>(blk + p.P * kD + (p.P + r) * 4);
      vs = bf16_lo(vp);
      vz = bf16_hi(vp);
      float dot = 0.f;
      for (int w = 0; w < kD / 8; ++w) {
        const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + r * (kD / 2) + word_off(kD, r, w));
        for (int i = 0; i < 4; ++i) {
          const float2 v = value_pair(word, i, bf16_lo(kp), bf16_hi(kp));
          dot = fmaf(v.x, qs[warp][8 * w + 2 * i], dot);
          dot = fmaf(v.y, qs[warp][8 * w + 2 * i + 1], dot);
        }
      }
      x = dot * p.c;
    }
    float mx = x;
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, s));
    const float mn = fmaxf(m, mx);
    const float f = m == -INFINITY ? 0.f : ex2(m - mn);
    const float e = see ? ex2(x - (mn == -INFINITY ? 0.f : mn)) : 0.f;
    m = mn;
    float es = e;
    for (int s = 16; s > 0; s >>= 1) es += __shfl_xor_sync(0xFFFFFFFFu, es, s);
    l = l * f + es;
    for (int i = 0; i < kPer; ++i) acc[i] *= f;
    for (int k = 0; k < 32; ++k) {
      const bool sk = __shfl_sync(0xFFFFFFFFu, int(see), k);
      const float ek = __shfl_sync(0xFFFFFFFFu, e, k), sv = __shfl_sync(0xFFFFFFFFu, vs, k), zv = __shfl_sync(0xFFFFFFFFu, vz, k);
      const uint8_t* bk = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(blk), k));
      const int rk = (j0 + k) & (p.P - 1);
      if (!sk) continue;
      const uint8_t* codes = bk + (p.P + rk) * (kD / 2);
      for (int i = 0; i < kPer; i += 2) {
        const int dim = lane * kPer + i;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + word_off(kD, rk, dim >> 3));
        const float2 v = value_pair(word, (dim & 7) >> 1, sv, zv);
        acc[i] = fmaf(ek, v.x, acc[i]);
        acc[i + 1] = fmaf(ek, v.y, acc[i + 1]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(o + lane * kPer + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
}

// How a call is run: by the rows a kv head has, T G.
struct Plan {
  int kind;   // 1, 2: few rows (one or two 8-row tiles); 0: a warp a row
  int ntile, rows;
  int64_t grid, items;
  size_t cnt, ml, o, total;  // workspace: counts, then partial (m, l), then partial O
};

static int sms_or_default() {
  const int sms = device_sm_count();
  return sms > 0 ? sms : 152;
}

static Plan plan_of(int B, int T, int Hq, int Hkv, int d, int64_t max_len) {
  Plan q{};
  const int64_t R = int64_t(T) * (Hq / Hkv);
  q.kind = R <= 8 ? 1 : R <= 16 ? 2 : 0;
  q.ntile = 1;
  q.rows = q.kind == 1 ? 8 : q.kind == 2 ? 16 : 0;
  q.items = int64_t(B) * Hkv * q.ntile;
  const int64_t units = q.items * ((max_len + kKeys - 1) / kKeys);
  q.grid = std::min<int64_t>(units, int64_t(sms_or_default()) * (q.kind == 1 ? RowsCfg<128, 1>::kCtas : 1));
  q.cnt = size_t(round_up(q.items * 4, 256));
  q.ml = size_t(round_up(q.grid * 2 * q.rows * 8, 256));
  q.o = size_t(q.grid) * 2 * q.rows * d * 4;
  q.total = q.cnt + q.ml + q.o + 256;
  return q;
}

template <int kD, int kNT>
static cudaError_t launch_rows(const Params& p, int64_t grid, cudaStream_t stream) {
  using C = RowsCfg<kD, kNT>;
  static bool ready[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kv4_attn_rows_kernel<kD, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_attn_rows_kernel<kD, kNT>, p);
}

static bool shape_ok(int B, int T, int Hq, int Hkv, int head_dim, int page_size, int64_t max_len) {
  return B >= 1 && B <= 65535 && T >= 1 && T <= (1 << 20) && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= 1024 &&
         (head_dim == 64 || head_dim == 128) && page_ok(page_size) && max_len >= 1 && max_len < (int64_t(1) << 31) - 256;
}

}  // namespace kv4_attn
}  // namespace w12

using namespace w12;
using namespace w12::kv4;

extern "C" {

size_t w12_kv4_attention_ws_bytes(int B, int T, int Hq, int Hkv, int head_dim, int page_size, int64_t max_kv_len) {
  return kv4_attn::shape_ok(B, T, Hq, Hkv, head_dim, page_size, max_kv_len)
             ? kv4_attn::plan_of(B, T, Hq, Hkv, head_dim, max_kv_len).total
             : 0;
}

int w12_kv4_attention(const uint16_t* Q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                      const w12_kv4* cache, const int32_t* table, int max_pages, int B, int T, int Hq,
                      int64_t max_kv_len, const int32_t* prefix_len, const int32_t* q_len, const int32_t* parents,
                      float scale, uint16_t* O, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!Q || !cache || !cache->pool || !table || !prefix_len || !O || !aligned(Q, 16) || !aligned(O, 16) ||
      !aligned(cache->pool, 16) || ((q_batch_stride | q_token_stride | q_head_stride) & 7) || !(scale > 0.f) ||
      scale > 1e30f)
    return W12_ERR_ARG;
  if (!cache_ok(cache) ||
      !kv4_attn::shape_ok(B, T, Hq, cache->Hkv, cache->head_dim, cache->page_size, max_kv_len) || max_pages < 1 ||
      max_kv_len > int64_t(max_pages) * cache->page_size || (parents && T > kv4_attn::kMaxTree))
    return W12_ERR_SHAPE;
  if (!ws || !aligned(ws, 16) ||
      ws_bytes < w12_kv4_attention_ws_bytes(B, T, Hq, cache->Hkv, cache->head_dim, cache->page_size, max_kv_len))
    return W12_ERR_WORKSPACE;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  kv4_attn::Params p{};
  p.Q = Q;
  p.q_b = q_batch_stride;
  p.q_t = q_token_stride;
  p.q_h = q_head_stride;
  p.O = O;
  p.pool = cache->pool;
  p.n_pages = cache->n_pages;
  p.block = block_bytes(cache->page_size, cache->head_dim);
  p.table = table;
  p.prefix_len = prefix_len;
  p.q_len = q_len;
  p.parents = parents;
  p.status = dev_status;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = cache->Hkv;
  p.G = Hq / cache->Hkv;
  p.P = cache->page_size;
  p.p_shift = __builtin_ctz(unsigned(cache->page_size));
  p.max_pages = max_pages;
  p.max_len = int(max_kv_len);
  p.c = float(double(scale) * 1.4426950408889634);
  p.limit_ns = wait_limit_ns();
  const kv4_attn::Plan pl = kv4_attn::plan_of(B, T, Hq, cache->Hkv, cache->head_dim, max_kv_len);
  p.ntile = pl.ntile;
  p.rows_per_tile = pl.rows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.cnt = reinterpret_cast<int32_t*>(w);
  p.part_ml = reinterpret_cast<float2*>(w + pl.cnt);
  p.part_o = reinterpret_cast<float*>(w + pl.cnt + pl.ml);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pl.kind == 1)
    return cuda_status(cache->head_dim == 128 ? kv4_attn::launch_rows<128, 1>(p, pl.grid, s)
                                              : kv4_attn::launch_rows<64, 1>(p, pl.grid, s));
  if (pl.kind == 2)
    return cuda_status(cache->head_dim == 128 ? kv4_attn::launch_rows<128, 2>(p, pl.grid, s)
                                              : kv4_attn::launch_rows<64, 2>(p, pl.grid, s));
  const int64_t rows = int64_t(B) * T * Hq;
  const int64_t grid = (rows + kv4_attn::kWarps - 1) / kv4_attn::kWarps;
  if (grid > 0x7FFFFFFF) return W12_ERR_SHAPE;
  if (cache->head_dim == 128)
    kv4_attn::kv4_attn_simple_kernel<128><<<unsigned(grid), kv4_attn::kWarps * 32, 0, s>>>(p);
  else
    kv4_attn::kv4_attn_simple_kernel<64><<<unsigned(grid), kv4_attn::kWarps * 32, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
