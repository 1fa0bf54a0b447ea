// Attention over the paged 4-bit cache: the choice of kernel and the launch.
#include <algorithm>

#include "w12_kv4_rows.cuh"
#include "w12_kv4_tile.cuh"

namespace w12 {
namespace kv4_attn {

static bool shape_ok(int B, int T, int Hq, int Hkv, int head_dim, int page_size, int64_t max_len) {
  return B >= 1 && B <= 65535 && T >= 1 && T <= (1 << 20) && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= 1024 &&
         (head_dim == 64 || head_dim == 128) && page_ok(page_size) && max_len >= 1 && max_len < (int64_t(1) << 31) - 256 &&
         int64_t(B) * ((int64_t(T) * (Hq / Hkv) + 127) / 128) * Hkv < (int64_t(1) << 31);
}

// How a call is run: by T G, the rows a kv head has. Up to 8 rows go to the rows kernel
// in one 8-row tile, up to 16 in two, more to 128-row tiles. 8 kv heads, pages of 64, us,
// rows kernel / tiles:
//             1 x 777      1 x 8192     16 x 2048    16 x 8192    64 x 2048-8192
//   d 128  9  13.5 / 19.2  19.9 / 33.7  33.9 / 41.3  74.5 / 85.7  194 / 197
//         12  15.1 / 18.2  22.9 / 32.1  35.5 / 40.7  76.4 / 85.4  205 / 198
//         16  15.8 / 18.4  23.7 / 32.2  36.5 / 40.6  77.5 / 85.3  208 / 198
//   d  64  9   9.4 / 16.0  13.2 / 26.8  23.7 / 32.9  50.3 / 71.0  132 / 165
//         16  11.0 / 14.8  16.2 / 26.0  25.1 / 31.9  51.6 / 70.3  141 / 164
// (one tile, d 128, 64 requests: 1 row 104 / 203, 8 rows 113 / 200). The two 8-row tiles lose by 3 to
// 5 % in one corner, 11 rows or more at d 128 over more than 300 MB, and win elsewhere.
struct Plan {
  int kind;   // few rows: their 8-row tiles (1 or 2); 0: 128-row tiles
  int ntile, rows;
  int64_t grid;
  size_t ml, o, total;  // workspace: kRunCounters counts, then partial (m, l), then partial O
};

static int sms_or_default() {
  const int sms = device_sm_count();
  return sms > 0 ? sms : 152;
}

static Plan plan_of(int B, int T, int Hq, int Hkv, int d, int64_t max_len) {
  Plan q{};
  const int64_t R = int64_t(T) * (Hq / Hkv);
  q.kind = R <= 8 ? 1 : R <= 16 ? 2 : 0;
  q.rows = q.kind ? 8 * q.kind : 128;
  q.ntile = int((R + q.rows - 1) / q.rows);
  const int64_t units = int64_t(B) * Hkv * q.ntile * ((max_len + kKeys - 1) / kKeys);
  q.grid = std::min<int64_t>(units, int64_t(sms_or_default()) * (q.kind == 1 ? RowsCfg<128, 1>::kCtas : 1));
  q.grid = std::min<int64_t>(q.grid, kRunCounters);
  q.ml = size_t(round_up(q.grid * 2 * q.rows * 8, 256));
  q.o = size_t(q.grid) * 2 * q.rows * d * 4;
  q.total = kRunCounters * 4 + q.ml + q.o;
  return q;
}

// Launch of one kernel with its shared memory (granted once a device). regs: registers a
// thread that it counts on being launched with.
template <typename Kernel>
static cudaError_t launch(Kernel* kernel, bool (&ready)[64], int threads, int smem, const Params& p, int64_t grid,
                          cudaStream_t stream, int regs = 0) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes has;
    e = cudaFuncGetAttributes(&has, kernel);
    if (e != cudaSuccess) return e;
    if (has.numRegs < regs) return cudaErrorInvalidConfiguration;  // (warps would wait for registers for good)
    ready[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int kD>
static cudaError_t launch_kind(int kind, const Params& p, int64_t grid, cudaStream_t stream) {
  static bool ready[3][64] = {};
  if (kind == 1)
    return launch(kv4_attn_rows_kernel<kD, 1>, ready[1], RowsCfg<kD, 1>::kThreads, RowsCfg<kD, 1>::kSmem, p, grid, stream);
  if (kind == 2)
    return launch(kv4_attn_rows_kernel<kD, 2>, ready[2], RowsCfg<kD, 2>::kThreads, RowsCfg<kD, 2>::kSmem, p, grid, stream);
  return launch(kv4_attn_tile_kernel<kD>, ready[0], TileCfg<kD>::kThreads, int(TileCfg<kD>::kSmem), p, grid, stream,
                TileCfg<kD>::kLaunchRegs);
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
  const kv4_attn::Plan pl = kv4_attn::plan_of(B, T, Hq, cache->Hkv, cache->head_dim, max_kv_len);
  if (!ws || !aligned(ws, 16) || ws_bytes < pl.total) return W12_ERR_WORKSPACE;
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
  p.sleep_ns = attn_impl::sleep_ns(p.limit_ns);
  p.ntile = pl.ntile;
  p.rows_per_tile = pl.rows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.cnt = reinterpret_cast<int32_t*>(w);
  p.part_ml = reinterpret_cast<float2*>(w + kRunCounters * 4);
  p.part_o = reinterpret_cast<float*>(w + kRunCounters * 4 + pl.ml);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(cache->head_dim == 128 ? kv4_attn::launch_kind<128>(pl.kind, p, pl.grid, s)
                                            : kv4_attn::launch_kind<64>(pl.kind, p, pl.grid, s));
}

}  // extern "C"
