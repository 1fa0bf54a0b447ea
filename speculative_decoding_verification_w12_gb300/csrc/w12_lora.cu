// Low-rank adapters of many requests beside a shared projection:
//   Y[m, :] += scale_a B_a (A_a x_m),  a = ids[m],  m < M <= 256.
//
// Two launches. The first groups the rows by adapter into tiles of up to 16 (every block does
// that for itself from the ids: 256 numbers), multiplies a tile's rows by A_a and leaves
// T = scale (A x) for the second, which adds B_a T to the tile's rows of Y. So an adapter that
// several requests share is read once for each 16 of their rows, and a row without an adapter
// costs nothing. Up to 32 rows are grouped by one warp in a few instructions: then the second
// launch does so too, and starts beside the first; for more it takes the tiles that the first
// has written down (grouped by every block of it, 256 rows cost 13 of 47 us).
//
// Both are products of mma.sync m16n8k16 with 16 rows at a time: what is read decides, and a
// tensor-memory tile of 128 rows would be nearly empty. T is fp32; the second product takes
// it as the sum of three bf16 numbers (8 + 8 + 8 bits), since Y is fp32 and a T rounded to
// bf16 would leave 2^-9 of the adapter's part. The order of K within a product is free, so a
// lane's operands are 16 bytes of a row of memory (8 of B at rank 16 and below). The loads of a
// step are in flight before the step before it computes.
//
// The first launch splits K over a cluster of eight blocks (and their eight warps); the
// blocks' sums meet in distributed shared memory, in a fixed order. With more tiles than clusters a
// cluster takes 2, 4 or 8 of them at a time and splits K that much less: 256 rows of an adapter
// each had 47 us there when every tile went through a whole cluster, 21 so.
//
// The second gives every warp as many neighbouring units of 16 columns, over the tiles: warps that
// went over the tiles one behind the other waited for each one's rows, T and first columns (256
// rows of an adapter each, rank 16, 5120 -> 7168: both launches 84 us, now 42). B is marked as read once,
// which leaves the L2 cache to Y (64 rows of an adapter each, rank 16, 5120 -> 34,816: 36 us, without 39).
//
// 16 x 16 rows, rank 64, 5120 -> 34,816 take 36 us for 156 MB: 10 for the first launch's chain of
// loads and sums, 26 for the second's 142 MB at 5.5 TB/s. Few rows are two launches' latency: 16
// rows of one adapter of rank 16, 5120 -> 5120, 5.7 us. Many single rows of a small rank are bound
// by issue: those 64 rows' 100 MB at 2.8 TB/s. (All from HBM; 27, 5.5 and 33 us from L2.)
#include <algorithm>

#include "w12_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSplit = 8;        // blocks of a cluster, along K
constexpr int kMaxRank = 128;

struct Params {
  const uint16_t *X, *A, *B;
  const float* scale;
  const int32_t* ids;
  float* Y;
  uint32_t* frag;    // [tile][16 of the rank][term][lane][4]: T as operands
  int32_t* head;     // [0]: tiles; from 64 on 32 words a tile: its 16 rows (-1: none), its adapter
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

// Rows by adapter: a tile begins at the first row of an adapter and at every 16th after it.
struct Tiles {
  // Neighbours of one adapter: which, from where, how many; rows of it before.
  __align__(16) int run_key[kMaxM], run_len[kMaxM];
  int run_at[kMaxM + 1], run_before[kMaxM];
  int count[2][kWarps];
  int row[16];        // of the tile in hand; -1: none
  int key;            // its adapter
  int nth;            // its place among the adapter's tiles
};

// A thread's row: its adapter, the rows of the same before it, and the tile that begins with it (-1).
struct Mine {
  int key, before, begins;
};

// Threads of the block before this one for which `yes` holds; in `all`, how many do.
__device__ __forceinline__ int before_me(bool yes, int (&count)[kWarps], int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, yes);
  if (lane == 0) count[warp] = __popc(mask);
  __syncthreads();
  int at = __popc(mask & ((1u << lane) - 1u));
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    at += w < warp ? count[w] : 0;
    all += count[w];
  }
  return at;
}

// Block-wide: every thread's row (the row of its index); the number of tiles. Neighbours of one
// adapter (a request's rows) are taken together: runs are compared, not rows.
__device__ __forceinline__ int sort_rows(const Params& p, Tiles& s, Mine& m) {
  const int tid = threadIdx.x;
  auto id_of = [&](int row) {
    const int id = p.ids[row];
    return id >= -1 && id < p.n ? id : -2;
  };
  m.key = tid < p.M ? id_of(tid) : -1;
  if (m.key == -2) {
    set_status(p.status, W12_ERR_ARG);
    m.key = -1;
  }
  const int last = tid > 0 && tid < p.M ? max(id_of(tid - 1), -1) : -1;
  const bool begins = tid == 0 || m.key != last;
  int runs, total;
  const int run = before_me(begins, s.count[0], runs) + begins - 1;
  if (begins) {
    s.run_key[run] = m.key;
    s.run_at[run] = tid;
  }
  if (tid == 0) s.run_at[runs] = kThreads;
  __syncthreads();
  if (begins) s.run_len[run] = s.run_at[run + 1] - s.run_at[run];
  __syncthreads();
  if (begins) {
    int n = 0;
    for (int j = 0; m.key >= 0 && j < run; j += 4) {  // (runs from this one on are looked at and not counted)
      const int4 k = *reinterpret_cast<const int4*>(&s.run_key[j]), l = *reinterpret_cast<const int4*>(&s.run_len[j]);
      n += k.x == m.key ? l.x : 0;
      n += k.y == m.key && j + 1 < run ? l.y : 0;
      n += k.z == m.key && j + 2 < run ? l.z : 0;
      n += k.w == m.key && j + 3 < run ? l.w : 0;
    }
    s.run_before[run] = n;
  }
  __syncthreads();
  m.before = s.run_before[run] + tid - s.run_at[run];
  const bool first = m.key >= 0 && m.before % 16 == 0;
  const int at = before_me(first, s.count[1], total);
  m.begins = first ? at : -1;
  return total;
}

constexpr int kFew = 32;   // rows that one warp groups

// Of up to 32 rows, by every warp for itself: the rows g and g + 8 and the adapter of tile t; the
// number of tiles.
struct Few {
  uint32_t same, firsts;
  int key, before;
};
__device__ __forceinline__ int sort_few(const Params& p, Few& f) {
  const int lane = threadIdx.x & 31;
  f.key = lane < p.M ? p.ids[lane] : -1;
  if (f.key < -1 || f.key >= p.n) {
    set_status(p.status, W12_ERR_ARG);
    f.key = -1;
  }
  f.same = __match_any_sync(0xFFFFFFFFu, f.key);
  f.before = __popc(f.same & ((1u << lane) - 1u));
  f.firsts = __ballot_sync(0xFFFFFFFFu, f.key >= 0 && f.before % 16 == 0);
  return __popc(f.firsts);
}
__device__ __forceinline__ int nth_bit(uint32_t mask, int n) {  // n + 1 bits are set
  for (; n > 0; --n) mask &= mask - 1;
  return __ffs(mask) - 1;
}
__device__ __forceinline__ int few_tile(const Few& f, int t, int& r0, int& r1) {
  const int lane = threadIdx.x & 31, g = lane >> 2, from = nth_bit(f.firsts, t);
  const int key = __shfl_sync(0xFFFFFFFFu, f.key, from), at = __shfl_sync(0xFFFFFFFFu, f.before, from);
  const uint32_t same = __shfl_sync(0xFFFFFFFFu, f.same, from);
  const int n = __popc(same) - at;   // rows from the tile's first on
  r0 = g < n ? nth_bit(same, at + g) : -1;
  r1 = g + 8 < n ? nth_bit(same, at + g + 8) : -1;
  return key;
}

// Block-wide: the rows and the adapter of tile t (there is one) into s. Behind a barrier after
// the last use of the tile before.
__device__ __forceinline__ void take_tile(Tiles& s, const Mine& m, int t) {
  if (threadIdx.x < 16) s.row[threadIdx.x] = -1;
  if (m.begins == t) {
    s.key = m.key;
    s.nth = m.before / 16;
  }
  __syncthreads();
  if (m.key >= 0 && m.key == s.key && m.before / 16 == s.nth) s.row[m.before % 16] = threadIdx.x;
  __syncthreads();
}

// Blocks an SM of the two launches that a rank has registers for. (Rank 64 with one block of the first and
// three steps of loads ahead: 16 x 16 rows 31 us where two and one ahead take 27.)
constexpr int shrink_blocks(int rank) { return rank <= 64 ? 2 : 1; }
constexpr int expand_blocks(int rank) { return rank <= 16 ? 3 : rank <= 64 ? 2 : 1; }

// kR: rank rounded up to the next of 16, 32, 64, 128.
template <int kR, bool kSmall>
__global__ void __launch_bounds__(kThreads, shrink_blocks(kR)) shrink_kernel(const __grid_constant__ Params p) {
  constexpr int kN = kR / 8;   // tiles of 8 of the rank
  constexpr int kParts = 4;
  __shared__ Tiles s;
  __shared__ __align__(16) float part[kParts][16][kR];
  grid_dep_wait();
  grid_dep_launch();
  const int rank = int(blockIdx.x);  // (the cluster is the grid's x)
  Mine m;
  Few f;
  const int total = kSmall ? sort_few(p, f) : sort_rows(p, s, m);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  if (!kSmall && rank == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.head[0] = total;
  // A cluster takes as many tiles at a time (1, 2, 4, 8) as leaves few rounds; K is split over a
  // tile's blocks.
  int split = kSplit;
  while (split > 1 && total * split > int(gridDim.y) * kSplit) split >>= 1;
  const int group = rank / split, part_k = rank % split, groups = kSplit / split;
  for (int t0 = int(blockIdx.y) * groups; t0 < total; t0 += int(gridDim.y) * groups) {  // (the same in all of the cluster)
    const bool there = t0 + group < total;
    const int t = there ? t0 + group : t0;
    int a, r0, r1;
    if constexpr (kSmall) {
      a = few_tile(f, t, r0, r1);
    } else {
      take_tile(s, m, t);
      a = s.key;
      r0 = s.row[g];
      r1 = s.row[g + 8];
      if (part_k == 0 && there && threadIdx.x < 17) p.head[64 + 32 * t + threadIdx.x] = threadIdx.x < 16 ? s.row[threadIdx.x] : a;
    }
    const float scale = p.scale[a];
    const uint16_t *x0 = p.X + int64_t(max(r0, 0)) * p.x_stride, *x1 = p.X + int64_t(max(r1, 0)) * p.x_stride;
    const uint16_t* Aa = p.A + int64_t(a) * p.rank * p.K;
    float acc[kN][4];
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // Steps ahead that loads are in flight: as the registers allow.
    constexpr int kAhead = kR <= 16 ? 3 : kR <= 32 ? 2 : 1;
    const int step_k = 32 * split * kWarps;
    uint4 u0[kAhead], u1[kAhead], w[kAhead][kN];
    const int K = int(p.K);  // below 2^30
    auto load = [&](int i, int k) {
      const int at = k + 8 * q;
      const bool in = at < K;  // K is a multiple of 8
      u0[i] = in && r0 >= 0 ? *reinterpret_cast<const uint4*>(x0 + at) : zero;
      u1[i] = in && r1 >= 0 ? *reinterpret_cast<const uint4*>(x1 + at) : zero;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        w[i][j] = in && 8 * j + g < p.rank ? __ldg(reinterpret_cast<const uint4*>(Aa + int64_t(8 * j + g) * p.K + at)) : zero;
    };
    int k = there ? 32 * (part_k + split * warp) : K;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, k + i * step_k);
    while (k < K) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {  // (past K all operands are zero)
        const uint32_t m0[4] = {u0[i].x, u1[i].x, u0[i].y, u1[i].y}, m1[4] = {u0[i].z, u1[i].z, u0[i].w, u1[i].w};
        uint4 v[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] = w[i][j];
        load(i, k + kAhead * step_k);
        k += step_k;
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          mma16816(acc[j], m0, v[j].x, v[j].y);
          mma16816(acc[j], m1, v[j].z, v[j].w);
        }
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
    for (int e = there ? part_k * kThreads + threadIdx.x : 8 * kR; e < 8 * kR; e += split * kThreads) {
      const int row = e / (kR / 2), j = 2 * (e % (kR / 2));
      float2 v = make_float2(0.f, 0.f);
      for (int c = 0; c < split; ++c) {
        const float2 o = peer_load2(&part[0][row][j], uint32_t(group * split + c));
        v.x += o.x;
        v.y += o.y;
      }
      // (Columns past the rank: an infinity of X has met zeros there.)
      v.x = j < p.rank ? v.x * scale : 0.f;
      v.y = j + 1 < p.rank ? v.y * scale : 0.f;
      // At 32 and above a lane has 8 neighbours of 32, the first four of them in the first of two steps.
      const int step = kR >= 32 ? 2 * (j / 32) + ((j & 4) ? 1 : 0) : 0, lane_q = kR >= 32 ? (j % 32) / 8 : j / 4;
      uint32_t* out = p.frag + (int64_t(t) * (kR / 16) + step) * 384 + ((row & 7) * 4 + lane_q) * 4 + ((j & 2) ? 2 : 0) + (row >> 3);
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const uint32_t b = pack_bf16x2(v.x, v.y);
        out[term * 128] = b;
        v.x = rest_of(v.x, __uint_as_float(b << 16));
        v.y = rest_of(v.y, __uint_as_float(b & 0xFFFF0000u));
      }
    }
    __syncwarp();
    cluster_sync();  // no block goes on while another reads its sums
  }
}

template <int kR, bool kSmall>
__global__ void __launch_bounds__(kThreads, expand_blocks(kR)) expand_kernel(const __grid_constant__ Params p) {
  constexpr int kC = kR / 16;
  constexpr bool kWide = kR >= 32;
  constexpr int kAhead = kR <= 32 ? 2 : 1;   // units that loads are ahead: as the registers allow
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  // What the launch before writes of this is T alone where rows are few: their rows, Y and B are
  // there before it ends.
  Few f;
  int total;
  if constexpr (kSmall) {
    total = sort_few(p, f);
  } else {
    grid_dep_wait();
    total = p.head[0];
  }
  // Units of 16 columns of a tile, in order; every warp takes as many neighbours.
  const int64_t per = p.N / 16, units = total * per, warps = int64_t(gridDim.x) * kWarps, me = int64_t(blockIdx.x) * kWarps + warp;
  const int64_t from = units * me / warps;
  int left = int(units * (me + 1) / warps - from), to_load = left;
  // Where a warp is: its tile, the lane's places in the tile's rows (null: no row) and in B, and the
  // columns that are left of the tile.
  struct At {
    int t, cols;
    float *y0, *y1;
    const uint16_t* b;
  };
  auto enter = [&](At& at, int t, int col) {
    int r0, r1, a;
    if constexpr (kSmall) {
      a = few_tile(f, t, r0, r1);
    } else {
      const int32_t* tile = p.head + 64 + 32 * t;
      r0 = tile[g], r1 = tile[g + 8], a = tile[16];
    }
    at.t = t;
    at.cols = int(p.N) - col;
    at.y0 = r0 >= 0 ? p.Y + int64_t(r0) * p.y_stride + col + 4 * q : nullptr;
    at.y1 = r1 >= 0 ? p.Y + int64_t(r1) * p.y_stride + col + 4 * q : nullptr;
    at.b = p.B + (int64_t(a) * p.N + col + 4 * (g >> 1) + (g & 1)) * p.rank + (kWide ? 8 : 4) * q;
  };
  // To the next unit; more: there is one.
  auto advance = [&](At& at, bool more) -> bool {
    at.cols -= 16;
    if (more && at.cols == 0) {
      enter(at, at.t + 1, 0);
      return true;
    }
    at.b += 16 * p.rank;
    if (at.y0) at.y0 += 16;
    if (at.y1) at.y1 += 16;
    return false;
  };
  // 16 columns a step: column 4q + {0, 1} of them from the first product, 4q + {2, 3} from
  // the second, so that a lane holds four neighbours of a row.
  struct Cols {
    float4 u0, u1;
    uint32_t w0[2 * kC], w1[2 * kC];
  };
  At in{};
  auto load = [&](Cols& c) {   // the unit at `in`, which moves on
    const uint16_t *b0 = in.b, *b1 = in.b + 2 * p.rank;
    if constexpr (kWide) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        const bool is = 32 * i + 8 * q < p.rank;  // the rank is a multiple of 8
        const uint4 f = is ? __ldcs(reinterpret_cast<const uint4*>(b0 + 32 * i)) : zero, h = is ? __ldcs(reinterpret_cast<const uint4*>(b1 + 32 * i)) : zero;
        c.w0[4 * i] = f.x, c.w0[4 * i + 1] = f.y, c.w0[4 * i + 2] = f.z, c.w0[4 * i + 3] = f.w;
        c.w1[4 * i] = h.x, c.w1[4 * i + 1] = h.y, c.w1[4 * i + 2] = h.z, c.w1[4 * i + 3] = h.w;
      }
    } else {
      const bool is = 4 * q < p.rank;
      const uint2 f = is ? __ldcs(reinterpret_cast<const uint2*>(b0)) : make_uint2(0, 0);
      const uint2 h = is ? __ldcs(reinterpret_cast<const uint2*>(b1)) : make_uint2(0, 0);
      c.w0[0] = f.x, c.w0[1] = f.y, c.w1[0] = h.x, c.w1[1] = h.y;
    }
    c.u0 = c.u1 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in.y0) c.u0 = *reinterpret_cast<const float4*>(in.y0);
    if (in.y1) c.u1 = *reinterpret_cast<const float4*>(in.y1);
    advance(in, --to_load > 0);
  };
  Cols next[kAhead];
  if (left > 0) enter(in, int(from / per), 16 * int(from % per));
  At at = in;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (to_load > 0) load(next[i]);
  if (kSmall) grid_dep_wait();
  uint32_t T[kC][3][4];
  auto load_t = [&]() {
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const uint4 v = *reinterpret_cast<const uint4*>(p.frag + ((int64_t(at.t) * kC + c) * 3 + term) * 128 + lane * 4);
        T[c][term][0] = v.x, T[c][term][1] = v.y, T[c][term][2] = v.z, T[c][term][3] = v.w;
      }
  };
  if (left > 0) load_t();
  while (left > 0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (left == 0) break;
      const Cols c = next[i];
      if (to_load > 0) load(next[i]);
      float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int term = 2; term >= 0; --term)
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          mma16816(c0, T[j][term], c.w0[2 * j], c.w0[2 * j + 1]);
          mma16816(c1, T[j][term], c.w1[2 * j], c.w1[2 * j + 1]);
        }
      if (at.y0)
        *reinterpret_cast<float4*>(at.y0) = make_float4(c.u0.x + c0[0], c.u0.y + c0[1], c.u0.z + c1[0], c.u0.w + c1[1]);
      if (at.y1)
        *reinterpret_cast<float4*>(at.y1) = make_float4(c.u1.x + c0[2], c.u1.y + c0[3], c.u1.z + c1[2], c.u1.w + c1[3]);
      if (advance(at, --left > 0)) load_t();
    }
  }
  grid_dep_launch();
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

static size_t head_bytes(int64_t tiles) { return size_t(256 + 128 * tiles); }

static int padded_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

template <int kR, bool kSmall>
static cudaError_t launch(const Params& p, int64_t tiles, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSplit;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // Clusters that the GPU holds at a time take the tiles in turn.
  cfg.gridDim = dim3(kSplit, unsigned(std::min<int64_t>(tiles, shrink_blocks(kR) * device_sm_count() / kSplit)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, shrink_kernel<kR, kSmall>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned(std::min<int64_t>((tiles * (p.N / 16) + 2 * kWarps - 1) / (2 * kWarps), expand_blocks(kR) * int64_t(device_sm_count()))));
  cfg.attrs = attr + 1;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, expand_kernel<kR, kSmall>, p);
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
  const bool few = M <= kFew;
  switch (padded_rank(a.rank)) {
    case 16: return cuda_status(few ? launch<16, true>(p, tiles, s) : launch<16, false>(p, tiles, s));
    case 32: return cuda_status(few ? launch<32, true>(p, tiles, s) : launch<32, false>(p, tiles, s));
    case 64: return cuda_status(few ? launch<64, true>(p, tiles, s) : launch<64, false>(p, tiles, s));
    default: return cuda_status(few ? launch<128, true>(p, tiles, s) : launch<128, false>(p, tiles, s));
  }
}

}  // extern "C"
