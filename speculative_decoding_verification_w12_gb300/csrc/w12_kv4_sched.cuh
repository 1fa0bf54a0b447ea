// Work split of the 4-bit cache's attention kernels (stream-K over requests of
// any length), planned on the GPU from the lengths there.
//
// An entry is one (request, row tile); an item is an entry with one kv head; a
// unit is one block of 128 keys of an item. Units are numbered entry by entry,
// kv head by kv head, block by block, over the blocks that the entry's tokens
// see, so requests shorter than the planned bound cost nothing. CTA c of n takes
// units [c U / n, (c + 1) U / n): its run is the tail of one item, whole items
// and the head of another. A segment of a run that is a whole item writes its
// output; otherwise it leaves a partial result in the CTA's slot (0 for the
// run's first segment, 1 for its last) and counts its units in; the segment that
// completes the item's count joins its partials. Which CTAs hold parts of an
// item follows from the same formula, in a fixed order, so results do not
// depend on which CTA is last.
#pragma once

#include "w12_kv4.cuh"

namespace w12 {
namespace kv4_attn {

using namespace kv4;

constexpr int kKeys = 128;     // keys of a unit
constexpr int kMaxTree = 128;  // nodes of a draft tree

struct Params {
  const uint16_t* Q;
  int64_t q_b, q_t, q_h;  // strides in elements
  uint16_t* O;            // [B, T, Hq, d]
  const uint8_t* pool;
  int64_t n_pages, block;
  const int32_t *table, *prefix_len, *q_len, *parents;
  int32_t* status;
  float* part_o;   // [grid][2 slots][rows][d]
  float2* part_ml; // [grid][2 slots][rows]
  int32_t* cnt;    // [grid]: units done of the item that begins in the CTA's run and ends in another's (zero between calls)
  int B, T, Hq, Hkv, G, P, p_shift, max_pages, max_len, ntile, rows_per_tile;
  float c;         // scale * log2(e)
  uint64_t limit_ns;
  uint32_t sleep_ns;
};

// Request b's cached and new tokens, clamped into range when they are not.
struct Lens {
  int prefix, n;
};

__device__ __forceinline__ Lens lens_of(const Params& p, int b) {
  int n = p.q_len ? p.q_len[b] : p.T, a = p.prefix_len[b];
  if (n < 0 || n > p.T || a < 0 || a > p.max_len - n) {
    set_status(p.status, W12_ERR_ARG);
    n = min(min(max(n, 0), p.T), p.max_len);
    a = min(max(a, 0), p.max_len - n);
  }
  return {a, n};
}

// Keys that the tokens of row tile `tile` see (rows are (token, head of the
// group), token-major): all of the request's in a tree, those up to the tile's
// last token otherwise. 0 when the tile holds no token.
__device__ __forceinline__ int keys_of(const Params& p, const Lens& l, int tile) {
  const int r0 = tile * p.rows_per_tile;
  if (r0 >= l.n * p.G) return 0;
  if (p.parents) return l.prefix + l.n;
  return l.prefix + min(l.n, (r0 + p.rows_per_tile - 1) / p.G + 1);
}

__device__ __forceinline__ int blocks_of(const Params& p, int entry) {
  const int b = entry / p.ntile;
  return (keys_of(p, lens_of(p, b), entry - b * p.ntile) + kKeys - 1) / kKeys;
}

// A CTA's place in the split.
struct Run {
  int64_t U;           // units of the call
  int64_t begin, end;  // this CTA's units
  int64_t entry_base;  // first unit of `entry`
  int entry;           // the entry that holds unit `begin`
  int n;               // CTAs with a run
};

struct RunSmem {
  long long warp_sum[32];
  Run run;
};

// Every thread of the CTA calls it (kN threads, a multiple of 32). E entries:
// thread i sums entries [i C, (i + 1) C); the thread whose entries hold the
// run's first unit walks to it.
template <int kN>
__device__ __forceinline__ const Run& plan_run(const Params& p, RunSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.B * p.ntile, C = (E + kN - 1) / kN;
  const int e0 = min(E, tid * C), e1 = min(E, e0 + C);
  long long mine = 0;
  for (int e = e0; e < e1; ++e) mine += blocks_of(p, e);
  mine *= p.Hkv;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sm.warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0, U = 0;
  for (int w = 0; w < kN / 32; ++w) {
    const long long s = sm.warp_sum[w];
    if (w < warp) before += s;
    U += s;
  }
  inc += before;
  const int n = int(U < (long long)gridDim.x ? U : (long long)gridDim.x);
  const long long begin = n ? (long long)blockIdx.x * U / n : 0;
  const bool has = int(blockIdx.x) < n;
  if (tid == 0 && !has) sm.run = {U, 0, 0, 0, 0, n};
  if (has && begin >= inc - mine && begin < inc) {
    long long base = inc - mine;
    int e = e0;
    for (; e < e1; ++e) {
      const long long u = (long long)blocks_of(p, e) * p.Hkv;
      if (begin < base + u) break;
      base += u;
    }
    sm.run = {U, begin, (long long)(blockIdx.x + 1) * U / n, base, e, n};
  }
  __syncthreads();
  return sm.run;
}

__device__ __forceinline__ int64_t run_start(const Run& r, int64_t c) { return c * r.U / r.n; }
// The CTA whose run holds unit x: the largest c with run_start(c) <= x.
__device__ __forceinline__ int run_of(const Run& r, int64_t x) { return int(((x + 1) * r.n - 1) / r.U); }

// One segment of a run.
struct Seg {
  int64_t x0;         // first unit of the item
  int b, tile, h;
  int nkb;            // blocks of the item
  int j0, j1;         // blocks of the segment
  int prefix, n;      // the request's tokens
  int keys;           // keys the item's rows see
  int slot;
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == nkb; }
};

// Walks a CTA's run segment by segment.
struct Walk {
  int64_t pos, base;  // next unit; first unit of `entry`
  int entry;

  Walk() = default;
  __device__ __forceinline__ explicit Walk(const Run& r) : pos(r.begin), base(r.entry_base), entry(r.entry) {}

  __device__ __forceinline__ bool next(const Params& p, const Run& r, Seg& s) {
    if (pos >= r.end) return false;
    for (;;) {
      s.b = entry / p.ntile;
      s.tile = entry - s.b * p.ntile;
      const Lens l = lens_of(p, s.b);
      s.prefix = l.prefix;
      s.n = l.n;
      s.keys = keys_of(p, l, s.tile);
      s.nkb = (s.keys + kKeys - 1) / kKeys;
      const int64_t units = int64_t(s.nkb) * p.Hkv;
      if (pos < base + units) break;
      base += units;
      ++entry;
    }
    s.h = int((pos - base) / s.nkb);
    s.x0 = base + int64_t(s.h) * s.nkb;
    s.j0 = int(pos - s.x0);
    s.j1 = int(min(int64_t(s.nkb), s.j0 + (r.end - pos)));
    s.slot = pos == r.begin ? 0 : 1;
    pos = s.x0 + s.j1;
    return true;
  }
};

// Rows t >= q_len[b] of the output are zero: shared out over all CTAs, in each of
// which one warp (all its lanes call it) looks at 32 (request, token) pairs at a
// time. Off the other warps' way: done by the whole CTA before its run, pair by pair,
// it held up a prompt chunk of 2 x 2048 tokens by 8 us.
template <int kD>
__device__ __forceinline__ void zero_idle_rows(const Params& p) {
  const int lane = threadIdx.x & 31;
  const int64_t pairs = int64_t(p.B) * p.T, step = gridDim.x;
  const int words = p.Hq * kD / 8;
  for (int64_t first = blockIdx.x; first < pairs; first += 32 * step) {
    const int64_t i = first + lane * step;
    bool idle = false;
    if (i < pairs) {
      const int b = int(i / p.T);
      idle = int(i - int64_t(b) * p.T) >= lens_of(p, b).n;
    }
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, idle); m; m &= m - 1) {
      uint4* o = reinterpret_cast<uint4*>(p.O + (first + (__ffs(m) - 1) * step) * p.Hq * kD);
      for (int w = lane; w < words; w += 32) o[w] = make_uint4(0, 0, 0, 0);
    }
  }
}

}  // namespace kv4_attn
}  // namespace w12
