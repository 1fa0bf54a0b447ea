// Page tables of a paged cache: pages handed out and taken back on the GPU.
//
// Request b holds used[b] pages, table[b][0 .. used[b]). A call brings every
// request to want = ceil((start + add) / P) pages. Requests that grow pop from
// the top of the free stack, in (request, page) order: the k-th page taken is
// free[n_free - 1 - k]. Requests that shrink push theirs so that the k-th page
// given back (in the same order) lands at free[n_free' + R - 1 - k], n_free'
// the count after the pops and R the pages given back: growing and then
// shrinking by the same amounts restores the stack.
//
// One thread-block cluster runs the call. Each CTA scans all B lengths itself
// (B loads from L2 and one block scan are cheaper than exchanging partial sums) and
// keeps them in shared memory; then the cluster's threads share the pages to pop and
// the slots to write. A slot on a page that the call takes is read from the free stack,
// not from the table entry that another CTA may be writing, so nothing waits for the
// pops but the pushes that reuse their stack entries. Latency-bound: a call is
// a few dependent L2 round trips (16 requests of 16 tokens: reserve and trim take
// 6.2 us on the device; 256 prompts of 1024 tokens, 1.2 MB of slots and pages: 16.7 us).
#include <cooperative_groups.h>

#include "w12_dev.cuh"
#include "w12_host.h"
#include "w12_kv4.cuh"

namespace w12 {
namespace pages_impl {

constexpr int kSmall = 256;   // threads of a small call's only CTA
constexpr int kLarge = 1024;  // threads of each CTA of a large call's cluster
constexpr int kCluster = 8;
constexpr int kSpan = 256;    // slots of one request that a warp writes at a time
constexpr int kMaxB = 8192;  // requests per call
constexpr int kPerRequest = 5 * 4;  // bytes of shared memory a request

struct PagesParams {
  int32_t *table, *used, *free_pages, *n_free;
  const int32_t *start, *add;
  int32_t* slots;
  int32_t* status;
  int B, max_pages, p_shift, n_pages, T;
};

struct Need {
  int have, want;
  bool ok;  // lengths and counts in range
};

__device__ __forceinline__ Need need_of(const PagesParams& p, int b) {
  const int start = p.start[b], add = p.add ? p.add[b] : 0, have = p.used[b];
  Need n;
  const int64_t want = (int64_t(start) + add + (1 << p.p_shift) - 1) >> p.p_shift;
  n.ok = start >= 0 && add >= 0 && add <= p.T && have >= 0 && have <= p.max_pages && want <= p.max_pages;
  n.have = n.ok ? have : 0;
  n.want = n.ok ? int(want) : 0;
  return n;
}

// Last index b in [0, n) with pre[b] <= k (pre ascending, pre[0] <= k).
__device__ __forceinline__ int last_le(const int* pre, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) pages_update_kernel(const __grid_constant__ PagesParams p) {
  extern __shared__ int smem[];
  int* gpre = smem;         // pages taken by the requests before b
  int* spre = gpre + p.B;   // pages given back by the requests before b
  int* base = spre + p.B;   // pages that request b holds before and after the call
  int* from = base + p.B;   // its start
  int* live = from + p.B;   // its new tokens, 0 where it is not served
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ int granted;   // pages taken by all requests that get theirs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto cluster = cooperative_groups::this_cluster();
  const int rank = int(blockIdx.x), all = int(gridDim.x) * kThreads, me = rank * kThreads + tid;

  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) granted = 0;
  const int n_free = min(max(*p.n_free, 0), p.n_pages);
  if (n_free != *p.n_free) set_status(p.status, W12_ERR_ARG);
  // Prefix sums, kThreads requests at a time; (grow, shrink) packed in one 64-bit sum.
  long long carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    long long v = 0;
    Need n{};
    if (b < p.B) {
      n = need_of(p, b);
      v = (static_cast<long long>(max(0, n.want - n.have)) << 32) | static_cast<long long>(max(0, n.have - n.want));
    }
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long before = carry, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long s = warp_sum[w];
      if (w < warp) before += s;
      total += s;
    }
    inc += before;
    if (b < p.B) {
      gpre[b] = int((inc - v) >> 32);
      spre[b] = int((inc - v) & 0xFFFFFFFFll);
      // Growing requests whose pages all lie within the free stack get them.
      const int upto = int(inc >> 32);
      const bool grows = (v >> 32) > 0, served = n.ok && (!grows || upto <= n_free);
      if (grows && served) atomicMax(&granted, upto);
      base[b] = min(n.have, n.want);
      from[b] = p.start[b];
      live[b] = served && p.add ? p.add[b] : 0;
    }
    carry += total;
    __syncthreads();
  }
  const int G = granted, R = int(carry & 0xFFFFFFFFll);
  cluster.barrier_arrive();  // this CTA has read the lengths and counts
  // Pops.
  for (int k = me; k < G; k += all) {
    const int b = last_le(gpre, p.B, k);
    p.table[int64_t(b) * p.max_pages + base[b] + (k - gpre[b])] = p.free_pages[n_free - 1 - k];
  }
  // Slots of the new tokens: a warp takes kSpan slots of one request at a time.
  if (p.T > 0) {
    const int spans = (p.T + kSpan - 1) / kSpan, units = p.B * spans;
    for (int u = me >> 5; u < units; u += all >> 5) {
      const int b = u / spans, i0 = (u - b * spans) * kSpan;
      const int start = from[b], n = live[b], held = base[b];
      const int32_t* tab = p.table + int64_t(b) * p.max_pages;
      const int32_t* taken = p.free_pages + (n_free - 1 - gpre[b]);
      int32_t* out = p.slots + int64_t(b) * p.T;
      // All loads of the span are in flight before the first store.
      int page[kSpan / 32];
#pragma unroll
      for (int x = 0; x < kSpan / 32; ++x) {
        const int i = i0 + 32 * x + lane, q = int((uint32_t(start) + uint32_t(i)) >> p.p_shift);  // (up to 2^31 + T)
        const int32_t* at = q < held ? tab + q : taken + (held - q);
        page[x] = 0;
        if (i < n) page[x] = *at;
      }
#pragma unroll
      for (int x = 0; x < kSpan / 32; ++x) {
        const int i = i0 + 32 * x + lane;
        if (i < p.T) out[i] = i < n ? (page[x] << p.p_shift) + int((uint32_t(start) + uint32_t(i)) & ((1u << p.p_shift) - 1u)) : -1;
      }
    }
  }
  cluster.barrier_wait();
  if (G > 0 && R > 0) cluster.sync();  // (the same in every CTA) pushes reuse the entries of pops
  // Pushes.
#pragma unroll 2
  for (int k = me; k < R; k += all) {
    const int b = last_le(spre, p.B, k);
    int32_t* e = p.table + int64_t(b) * p.max_pages + base[b] + (k - spre[b]);
    const int at = n_free - G + R - 1 - k;
    if (at < p.n_pages) p.free_pages[at] = *e;
    else set_status(p.status, W12_ERR_ARG);  // more pages than the pool has: counts that do not match
    *e = -1;
  }
  for (int b = me; b < p.B; b += all) {
    const Need n = need_of(p, b);
    const int grow = n.want - n.have;
    if (!n.ok) set_status(p.status, W12_ERR_ARG);
    else if (grow > 0 && gpre[b] + grow > n_free) set_status(p.status, W12_ERR_WORKSPACE);
    else p.used[b] = n.want;
  }
  if (me == 0) *p.n_free = min(n_free - G + R, p.n_pages);
}

}  // namespace pages_impl
}  // namespace w12

using namespace w12;
using namespace w12::pages_impl;

extern "C" int w12_pages_update(int32_t* table, int32_t* used, int32_t* free_pages, int32_t* n_free, int B,
                                int max_pages, int page_size, int64_t n_pages, const int32_t* start,
                                const int32_t* add, int T, int32_t* slots, int32_t* dev_status, void* stream) {
  if (!table || !used || !free_pages || !n_free || !start || T < 0 || (T > 0 && (!add || !slots))) return W12_ERR_ARG;
  if (B < 1 || B > kMaxB || max_pages < 1 || !kv4::page_ok(page_size) || n_pages < 1 ||
      n_pages > int64_t(0x7FFFFFFF) / page_size || int64_t(B) * max_pages > 0x7FFFFFFF ||
      int64_t(B) * T > 0x7FFFFFFF)
    return W12_ERR_SHAPE;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  PagesParams p{table, used, free_pages, n_free, start, add, slots, dev_status, B, max_pages,
                __builtin_ctz(unsigned(page_size)), int(n_pages), T};
  const size_t smem = size_t(B) * kPerRequest;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = overlap_enabled() ? attr : attr + 1;
  // A small call (a verify step's blocks) is one CTA: a cluster's launch and
  // barriers cost more than its threads bring (16 requests: 2.4 us a trim
  // instead of 5). A trim is small by the pages it may give back.
  const int64_t most = T > 0 ? int64_t(B) * T : int64_t(B) * max_pages / 2;
  if (most <= 4096 && B <= kSmall) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kSmall);
    cfg.numAttrs = overlap_enabled() ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, pages_update_kernel<kSmall>, p));
  }
  if (smem > 40 * 1024 && cudaFuncSetAttribute(pages_update_kernel<kLarge>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxB * kPerRequest) != cudaSuccess)
    return W12_ERR_CUDA;
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kLarge);
  cfg.numAttrs = overlap_enabled() ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, pages_update_kernel<kLarge>, p));
}
