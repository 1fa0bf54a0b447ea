// Low-rank adapters of many requests beside a shared projection:
//   Y[m, :] += scale_a B_a (A_a x_m),  a = ids[m],  m < M <= 256.
//
// Two launches. The first groups the rows by adapter into tiles of up to 16 (every block
// does that for itself from the ids: 256 numbers), multiplies a tile's rows by A_a and
// leaves T = scale (A x) for the second, which adds B_a T to the tile's rows of Y. So an
// adapter that several requests share is read once for each 16 of their rows, and a row
// without an adapter costs nothing.
//
// Both are products of mma.sync m16n8k16 with 16 rows at a time: what is read decides, and a
// tensor-memory tile of 128 rows would be nearly empty. T is fp32; the second product takes
// it as the sum of three bf16 numbers (8 + 8 + 8 bits), since Y is fp32 and a T rounded to
// bf16 would leave 2^-9 of the adapter's part. The order of K within a product is free, so a
// lane's operands are 16 (A, X) or 8 bytes (B) in a row of memory.
//
// The first launch splits K over a cluster of eight blocks (and their eight warps); the
// blocks' sums meet in distributed shared memory, in a fixed order.
#include "w12_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSplit = 8;        // blocks of a cluster, along K
constexpr int kMaxRank = 128;
constexpr int kCols = 512;       // columns of Y a block of the second launch

struct Params {
  const uint16_t *X, *A, *B;
  const float* scale;
  const int32_t* ids;
  float* Y;
  int32_t* head;     // [0]: tiles; from 64 on 32 words a tile: its 16 rows (-1: none), its adapter
  uint32_t* frag;    // [tile][16 of the rank][term][lane][4]: T as operands
  int64_t N, K, x_stride, y_stride;
  int M, n, rank;
  int32_t* status;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same place of shared memory in the cluster's block `rank`, read.
__device__ __forceinline__ float2 peer_load2(const float* p, uint32_t rank) {
  uint32_t at;
  float2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// What of x is left beside its bf16 part; nothing beside infinities and NaN.
__device__ __forceinline__ float rest_of(float x, float part) { return fabsf(part) < INFINITY ? x - part : 0.f; }

struct alignas(16) Tile {
  int id[kMaxM];
  int row[16];
  int count[kWarps];
  int key, rank;
};

// Block-wide: the rows of tile `t` into s.row, its adapter into s.key (-1: no such tile); the
// number of tiles. A tile begins at the first row of an adapter and at every 16th after it.
__device__ __forceinline__ int find_tile(const Params& p, Tile& s, int t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int key = -1;
  if (tid < p.M) {
    key = p.ids[tid];
    if (key < -1 || key >= p.n) {
      set_status(p.status, W12_ERR_ARG);
      key = -1;
    }
  }
  s.id[tid] = key;
  if (tid < 16) s.row[tid] = -1;
  if (tid == 0) s.key = -1;
  __syncthreads();
  int before = 0;
  const int4* all = reinterpret_cast<const int4*>(s.id);
  for (int i = 0; key >= 0 && i < (tid + 3) / 4; ++i) {
    const int4 v = all[i];
    before += (v.x == key) + (v.y == key && 4 * i + 1 < tid) + (v.z == key && 4 * i + 2 < tid) + (v.w == key && 4 * i + 3 < tid);
  }
  const bool first = key >= 0 && before % 16 == 0;
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
  if (lane == 0) s.count[warp] = __popc(firsts);
  __syncthreads();
  int at = __popc(firsts & ((1u << lane) - 1u)), total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    at += w < warp ? s.count[w] : 0;
    total += s.count[w];
  }
  if (first && at == t) {
    s.key = key;
    s.rank = before / 16;
  }
  __syncthreads();
  if (key >= 0 && key == s.key && before / 16 == s.rank) s.row[before % 16] = tid;
  __syncthreads();
  return total;
}

// kR: rank rounded up to the next of 16, 32, 64, 128.
template <int kR>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const __grid_constant__ Params p) {
  constexpr int kN = kR / 8;   // tiles of 8 of the rank
  constexpr int kParts = 4;
  __shared__ Tile s;
  __shared__ __align__(16) float part[kParts][16][kR];
  grid_dep_wait();
  grid_dep_launch();
  const int split = int(blockIdx.x), t = int(blockIdx.y);  // (the cluster is the grid's x)
  const int total = find_tile(p, s, t);
  if (split == 0 && t == 0 && threadIdx.x == 0) p.head[0] = total;
  if (t >= total) return;  // the same in all of the cluster
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int a = s.key;
  if (split == 0 && threadIdx.x < 17) p.head[64 + 32 * t + threadIdx.x] = threadIdx.x < 16 ? s.row[threadIdx.x] : a;
  const int r0 = s.row[g], r1 = s.row[g + 8];
  const uint16_t *x0 = p.X + int64_t(max(r0, 0)) * p.x_stride, *x1 = p.X + int64_t(max(r1, 0)) * p.x_stride;
  const uint16_t* Aa = p.A + int64_t(a) * p.rank * p.K;
  float acc[kN][4];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int64_t k = 32 * (split + kSplit * warp); k < p.K; k += 32 * kSplit * kWarps) {
    const int64_t at = k + 8 * q;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool in = at < p.K;  // K is a multiple of 8
    const uint4 u0 = in && r0 >= 0 ? *reinterpret_cast<const uint4*>(x0 + at) : zero;
    const uint4 u1 = in && r1 >= 0 ? *reinterpret_cast<const uint4*>(x1 + at) : zero;
    uint4 w[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i)
      w[i] = in && 8 * i + g < p.rank ? __ldg(reinterpret_cast<const uint4*>(Aa + int64_t(8 * i + g) * p.K + at)) : zero;
    const uint32_t m0[4] = {u0.x, u1.x, u0.y, u1.y}, m1[4] = {u0.z, u1.z, u0.w, u1.w};
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      mma16816(acc[i], m0, w[i].x, w[i].y);
      mma16816(acc[i], m1, w[i].z, w[i].w);
    }
  }
  // The warps' sums: those of the later four onto those of the first four, then these.
#pragma unroll
  for (int step = 1; step >= 0; --step) {
    if (warp / kParts == step) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float2* lo = reinterpret_cast<float2*>(&part[warp % kParts][g][8 * i + 2 * q]);
        float2* hi = reinterpret_cast<float2*>(&part[warp % kParts][g + 8][8 * i + 2 * q]);
        if (step == 1) {
          *lo = make_float2(acc[i][0], acc[i][1]);
          *hi = make_float2(acc[i][2], acc[i][3]);
        } else {
          *lo = make_float2(lo->x + acc[i][0], lo->y + acc[i][1]);
          *hi = make_float2(hi->x + acc[i][2], hi->y + acc[i][3]);
        }
      }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < 16 * kR; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) v += part[i][e / kR][e % kR];
    part[0][e / kR][e % kR] = v;
  }
  __syncwarp();
  cluster_sync();
  // The blocks' sums, a share of the pairs each: T, three bf16 parts, in the operands' order.
  const float scale = p.scale[a];
  for (int e = split * kThreads + threadIdx.x; e < 8 * kR; e += kSplit * kThreads) {
    const int row = e / (kR / 2), j = 2 * (e % (kR / 2));
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (uint32_t c = 0; c < kSplit; ++c) {
      const float2 o = peer_load2(&part[0][row][j], c);
      v.x += o.x;
      v.y += o.y;
    }
    v.x *= scale;
    v.y *= scale;
    uint32_t* out = p.frag + (int64_t(t) * (kR / 16) + j / 16) * 384 + ((row & 7) * 4 + (j % 16) / 4) * 4 + ((j & 2) ? 2 : 0) + (row >> 3);
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      const uint32_t b = pack_bf16x2(v.x, v.y);
      out[term * 128] = b;
      v.x = rest_of(v.x, __uint_as_float(b << 16));
      v.y = rest_of(v.y, __uint_as_float(b & 0xFFFF0000u));
    }
  }
  __syncwarp();
  cluster_sync();  // no block leaves while another reads its sums
}

template <int kR>
__global__ void __launch_bounds__(kThreads) expand_kernel(const __grid_constant__ Params p) {
  constexpr int kC = kR / 16;
  grid_dep_wait();
  grid_dep_launch();
  const int t = int(blockIdx.y);
  if (t >= p.head[0]) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int32_t* tile = p.head + 64 + 32 * t;
  const int r0 = tile[g], r1 = tile[g + 8], a = tile[16];
  uint32_t T[kC][3][4];
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      const uint4 v = *reinterpret_cast<const uint4*>(p.frag + ((int64_t(t) * kC + c) * 3 + term) * 128 + lane * 4);
      T[c][term][0] = v.x;
      T[c][term][1] = v.y;
      T[c][term][2] = v.z;
      T[c][term][3] = v.w;
    }
  const uint16_t* Ba = p.B + int64_t(a) * p.N * p.rank;
  float *y0 = p.Y + int64_t(max(r0, 0)) * p.y_stride, *y1 = p.Y + int64_t(max(r1, 0)) * p.y_stride;
  // 16 columns a step: column 4q + {0, 1} of them from the first product, 4q + {2, 3} from
  // the second, so that a lane holds four neighbours of a row.
  const int64_t end = min(int64_t(blockIdx.x + 1) * kCols, p.N);
  for (int64_t n = int64_t(blockIdx.x) * kCols + 16 * warp; n < end; n += 16 * kWarps) {
    const int64_t b0 = n + 4 * (g >> 1) + (g & 1);
    float4 u0 = make_float4(0.f, 0.f, 0.f, 0.f), u1 = u0;
    if (r0 >= 0) u0 = *reinterpret_cast<const float4*>(y0 + n + 4 * q);
    if (r1 >= 0) u1 = *reinterpret_cast<const float4*>(y1 + n + 4 * q);
    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
    uint2 w0[kC], w1[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int k = 16 * c + 4 * q;
      w0[c] = w1[c] = make_uint2(0, 0);
      if (k < p.rank) {  // (the rank is a multiple of 8)
        w0[c] = __ldg(reinterpret_cast<const uint2*>(Ba + b0 * p.rank + k));
        w1[c] = __ldg(reinterpret_cast<const uint2*>(Ba + (b0 + 2) * p.rank + k));
      }
    }
#pragma unroll
    for (int term = 2; term >= 0; --term)
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        mma16816(c0, T[c][term], w0[c].x, w0[c].y);
        mma16816(c1, T[c][term], w1[c].x, w1[c].y);
      }
    if (r0 >= 0) *reinterpret_cast<float4*>(y0 + n + 4 * q) = make_float4(u0.x + c0[0], u0.y + c0[1], u0.z + c1[0], u0.w + c1[1]);
    if (r1 >= 0) *reinterpret_cast<float4*>(y1 + n + 4 * q) = make_float4(u1.x + c0[2], u1.y + c0[3], u1.z + c1[2], u1.w + c1[3]);
  }
}

static bool shape_ok(int64_t M, int n, int rank) {
  return M >= 1 && M <= kMaxM && n >= 1 && n <= (1 << 24) && rank >= 8 && rank <= kMaxRank && rank % 8 == 0;
}

// Most tiles that M rows of n adapters can make.
static int64_t max_tiles(int64_t M, int n) {
  const int64_t used = M < n ? M : n;
  const int64_t t = used + M / 16;
  return t < M ? t : M;
}

static int padded_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

static size_t head_bytes(int64_t tiles) { return size_t(256 + 128 * tiles); }

template <int kR>
static cudaError_t launch(const Params& p, int64_t tiles, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSplit;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSplit, unsigned(tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, shrink_kernel<kR>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned((p.N + kCols - 1) / kCols), unsigned(tiles));
  cfg.attrs = attr + 1;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, expand_kernel<kR>, p);
}

}  // namespace lora
}  // namespace w12

using namespace w12;
using namespace w12::lora;

extern "C" {

size_t w12_lora_ws_bytes(int64_t M, int n_adapters, int rank) {
  if (!shape_ok(M, n_adapters, rank)) return 0;
  const int64_t tiles = max_tiles(M, n_adapters);
  return head_bytes(tiles) + size_t(tiles) * size_t(padded_rank(rank) / 16) * 1536;
}

int w12_lora(const uint16_t* X, int64_t x_stride, int64_t M, const w12_adapters* adapters, const int32_t* ids, float* Y,
             int64_t y_stride, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!X || !adapters || !ids || !Y || !adapters->A || !adapters->B || !adapters->scale) return W12_ERR_ARG;
  const w12_adapters& a = *adapters;
  if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(a.A, 16) || !aligned(a.B, 16)) return W12_ERR_ARG;
  if (!shape_ok(M, a.n, a.rank) || a.N < 16 || a.N % 16 || a.K < 8 || a.K % 8 || a.N >= (int64_t(1) << 30) || a.K >= (int64_t(1) << 30))
    return W12_ERR_SHAPE;
  if (M > 1 && (x_stride < a.K || x_stride % 8 || y_stride < a.N || y_stride % 4)) return W12_ERR_SHAPE;
  if (!ws || !aligned(ws, 16) || ws_bytes < w12_lora_ws_bytes(M, a.n, a.rank)) return W12_ERR_WORKSPACE;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  const int64_t tiles = max_tiles(M, a.n);
  Params p{};
  p.X = X;
  p.A = a.A;
  p.B = a.B;
  p.scale = a.scale;
  p.ids = ids;
  p.Y = Y;
  p.head = static_cast<int32_t*>(ws);
  p.frag = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + head_bytes(tiles));
  p.N = a.N;
  p.K = a.K;
  p.x_stride = x_stride;
  p.y_stride = y_stride;
  p.M = int(M);
  p.n = a.n;
  p.rank = a.rank;
  p.status = dev_status;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (padded_rank(a.rank)) {
    case 16: return cuda_status(launch<16>(p, tiles, s));
    case 32: return cuda_status(launch<32>(p, tiles, s));
    case 64: return cuda_status(launch<64>(p, tiles, s));
    default: return cuda_status(launch<128>(p, tiles, s));
  }
}

}  // extern "C"
