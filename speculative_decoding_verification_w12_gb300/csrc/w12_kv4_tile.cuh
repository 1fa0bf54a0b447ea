// Attention over the 4-bit cache for many query rows a kv head (draft blocks and
// trees, prompt chunks): 128-row tiles on the tensor memory.
//
// Work unit: 128 query rows of one (request, kv head), token-major, against one
// block of 128 keys (the split is w12_kv4_sched.cuh's). Per block:
//   raw pages -> shared memory   one bulk copy a page (warp 0)
//   codes -> bf16 K and V tiles  four warps; thread i restores row i of the block:
//                                z + s (q - 8), one rounding to bf16
//   S = Q K^T                    tcgen05.mma, D in TMEM, two buffers (warp 1)
//   P = exp2(c S - m)            two warpgroups, one a 64-key half of the block; P
//                                over its half's first 32 S columns as bf16 pairs
//   O_h += P_h V_h               tcgen05.mma, A = P from TMEM, V MN-major (warp 2)
// Here the scale is applied when the codes are restored: with 128 rows a tile,
// one more packed operation on a restored pair costs less than scales and
// centres in the softmax of 128 scores a key. The restored values are rounded
// to bf16 (2^-8 relative), as the rows of a bf16 cache would be.
//
// A key whose V parameters are not finite gets V = 0 and K = NaN: its score is
// NaN for the rows that see it and masked for the others, which P = 0 times NaN
// would not leave alone. Rows of the block past the keys get V = 0.
//
// The softmax warpgroups keep separate maxima, sums and O accumulators for the
// two key halves, joined in the epilogue; a maximum moves only when exceeded by
// more than 8 (log2 units).
#pragma once

#include "w12_attn_dev.cuh"
#include "w12_kv4_sched.cuh"

namespace w12 {
namespace kv4_attn {

using attn_impl::block_max;
using attn_impl::exp_pack;
using attn_impl::fast_exp2;
using attn_impl::mask_block;
using attn_impl::rescale_row;
using attn_impl::sdesc_mn_sw128;
using attn_impl::tmem_ld_wait64;

template <int kD>
struct TileCfg {
  static constexpr int kThreads = 512;     // warps 0-3 copy and issue, 4-11 softmax, 12-15 restore
  static constexpr uint32_t kHalf = 128u * 128u;       // 128 rows x 64 bf16, 128-byte swizzle
  static constexpr uint32_t kTile = kHalf * (kD / 64);
  static constexpr uint32_t kRaw = uint32_t(kKeys) * (kD + 8);
  static constexpr int kRawStages = kD == 128 ? 3 : 6;
  static constexpr int kStages = 2;        // restored K and V tiles
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kKOff = kTile;
  static constexpr uint32_t kVOff = kKOff + kStages * kTile;
  static constexpr uint32_t kRawOff = kVOff + kStages * kTile;
  static constexpr uint32_t kXchOff = kRawOff + kRawStages * kRaw;  // (m, l) of the two halves
  static constexpr uint32_t kBarOff = kXchOff + 2 * 128 * 8;
  static constexpr uint32_t kRunOff = kBarOff + 320;
  static constexpr uint32_t kSmem = kRunOff + 512 + 1024;           // 1024: alignment slack
  // TMEM columns: S of even and odd blocks, O of the two key halves.
  static constexpr uint32_t kS0 = 0, kS1 = 128, kOA = 256, kOB = 256 + kD, kCols = 512;
};

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Eight dims of a code word as bf16 values z + s (q - 8): 128 + q in bf16 bits,
// less 136 (exact), then one rounding. s2 and z2 hold s and z in both halves.
__device__ __forceinline__ uint4 restore_word(uint32_t w, uint32_t s2, uint32_t z2) {
  uint4 o;
  const uint32_t k136 = 0x43084308u;
  o.x = hfma2(hsub2((w & 0x000F000Fu) | 0x43004300u, k136), s2, z2);
  o.y = hfma2(hsub2(((w >> 4) & 0x000F000Fu) | 0x43004300u, k136), s2, z2);
  o.z = hfma2(hsub2(((w >> 8) & 0x000F000Fu) | 0x43004300u, k136), s2, z2);
  o.w = hfma2(hsub2(((w >> 12) & 0x000F000Fu) | 0x43004300u, k136), s2, z2);
  return o;
}

// Thread i's row of the block: its codes (kD / 2 bytes at `src`, row r of its
// page) into row i of a 128-byte-swizzled tile. The 16-byte pieces are taken in
// an order that differs from row to row, so that the eight rows of a
// shared-memory phase read and write different banks.
template <int kD>
__device__ __forceinline__ void restore_row(uint8_t* tile, const uint8_t* src, int i, uint32_t par, bool zero,
                                            uint32_t poison) {
  constexpr int kPieces = kD / 32;
  uint32_t s2 = __byte_perm(par, par, 0x1010), z2 = __byte_perm(par, par, 0x3232);
  if (zero) s2 = z2 = 0u;
  z2 |= poison;
  const uint32_t flip = kD == 128 ? uint32_t(i) & 2u : 0u;  // halves swapped in rows with bit 1 set
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const uint32_t at = (kD == 128 ? (uint32_t(i) >> 1) + k : (uint32_t(i) >> 2) + k) & (kPieces - 1);
    const uint4 w = *reinterpret_cast<const uint4*>(src + at * 16);
    const uint32_t c = at ^ flip;  // dims 32 c .. 32 c + 31
    uint8_t* row = tile + (c >> 1) * 16384u + uint32_t(i) * 128u;
    const uint32_t c8 = (c & 1u) * 4u, x = uint32_t(i) & 7u;
    *reinterpret_cast<uint4*>(row + (((c8 + 0) ^ x) << 4)) = restore_word(w.x, s2, z2);
    *reinterpret_cast<uint4*>(row + (((c8 + 1) ^ x) << 4)) = restore_word(w.y, s2, z2);
    *reinterpret_cast<uint4*>(row + (((c8 + 2) ^ x) << 4)) = restore_word(w.z, s2, z2);
    *reinterpret_cast<uint4*>(row + (((c8 + 3) ^ x) << 4)) = restore_word(w.w, s2, z2);
  }
}

__device__ __forceinline__ bool not_finite(uint32_t par) {
  return (par & 0x7F80u) == 0x7F80u || (par & 0x7F800000u) == 0x7F800000u;
}

template <int kD>
__global__ void __launch_bounds__(TileCfg<kD>::kThreads, 1) kv4_attn_tile_kernel(const __grid_constant__ Params p) {
  using C = TileCfg<kD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // pages of a block landed
  uint64_t* raw_empty = raw_full + C::kRawStages;                       // and restored (one arrival a warp)
  uint64_t* k_full = raw_empty + C::kRawStages;                         // K tile restored
  uint64_t* k_empty = k_full + C::kStages;                              // S of its block done
  uint64_t* v_full = k_empty + C::kStages;
  uint64_t* v_empty = v_full + C::kStages;                              // P V of its block done
  uint64_t* s_full = v_empty + C::kStages;                              // [2] S of block i in buffer i % 2
  uint64_t* p_full = s_full + 2;                                        // [2][2] P of block i, key half h
  uint64_t* o_done = p_full + 4;                                        // [2] P V of block i (both halves) done
  uint64_t* o_final = o_done + 2;                                       // every MMA of the segment done
  uint64_t* q_ready = o_final + 1;                                      // the segment's Q stored, O free
  uint64_t* drained = q_ready + 1;                                      // [2]
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(drained + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* merge_here = abort_flag + 1;
  RunSmem& rs = *reinterpret_cast<RunSmem*>(smem + C::kRunOff);
  static_assert((2 * C::kRawStages + 4 * C::kStages + 12) * 8 + 16 <= 320 && sizeof(RunSmem) <= 512, "carve-up");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&s_full[k], 1);
      mbar_init(&o_done[k], 1);
      mbar_init(&drained[k], 1);
    }
    for (int k = 0; k < 4; ++k) mbar_init(&p_full[k], 128);
    mbar_init(o_final, 2);
    mbar_init(q_ready, 256);
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_dep_wait();
  const Run run = plan_run<C::kThreads>(p, rs);  // its barriers publish the mbarriers too
  zero_idle_rows<kD, C::kThreads>(p);
  if (run.begin >= run.end) return;
  if (warp == 1) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint64_t lim = p.limit_ns;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 0; i < 0x80000000u; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((i & 63u) == 63u) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > lim) break;
      }
    }
    set_status(p.status, W12_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
  };

  Walk walk(run);
  Seg s;
  if (warp == 0) {
    // ------------------------------------------------------------- copies
    const int per = kKeys >> p.p_shift;
    const uint32_t bytes = uint32_t(p.block);
    const uint64_t page_stride = uint64_t(p.Hkv) * uint64_t(p.block);
    int issued = 0;
    bool ok = true;
    while (ok && walk.next(p, run, s)) {
      const int32_t* tab = p.table + int64_t(s.b) * p.max_pages;
      const uint8_t* pool = p.pool + uint64_t(s.h) * uint64_t(p.block);
      auto page_of = [&](int j) -> int {
        const int i = j * per + lane;
        return lane < per && (int64_t(i) << p.p_shift) < s.keys ? tab[i] : -2;
      };
      int next = page_of(s.j0);
      for (int j = s.j0; j < s.j1; ++j) {
        int page = next;
        if (j + 1 < s.j1) next = page_of(j + 1);
        const bool need = page != -2;
        if (need && (page < 0 || page >= p.n_pages)) {
          set_status(p.status, W12_ERR_ARG);
          page = 0;
        }
        const int st = issued % C::kRawStages;
        if (issued >= C::kRawStages &&
            !__all_sync(0xFFFFFFFFu, wait(&raw_empty[st], uint32_t(issued / C::kRawStages - 1) & 1u))) {
          ok = false;
          break;
        }
        const int pages = __popc(__ballot_sync(0xFFFFFFFFu, need));
        if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], uint32_t(pages) * bytes);
        __syncwarp();
        if (need)
          bulk_load(smem + C::kRawOff + st * C::kRaw + lane * bytes, pool + uint64_t(page) * page_stride, bytes,
                    &raw_full[st]);
        ++issued;
      }
    }
    if (lane == 0) grid_dep_launch();
    if (*abort_flag)
      for (int i = issued > C::kRawStages ? issued - C::kRawStages : 0; i < issued; ++i)
        mbar_wait(&raw_full[i % C::kRawStages], uint32_t(i / C::kRawStages) & 1u, drain_limit_ns(lim));
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      const uint32_t sbase = smem_u32(smem);
      const bool is_s = warp == 1;
      const uint64_t qd = sdesc_k_sw128(sbase + C::kQOff);
      const uint64_t kd0 = sdesc_k_sw128(sbase + C::kKOff);
      const uint64_t vd0 = sdesc_mn_sw128(sbase + C::kVOff, C::kHalf);
      const uint32_t idesc_s = idesc_bf16(128, 128);
      const uint32_t idesc_o = idesc_bf16(128, kD) | (1u << 16);  // B (V) MN-major
      int base = 0, si = 0;
      bool ok = true;
      while (ok && walk.next(p, run, s)) {
        const int n = s.j1 - s.j0;
        if (!wait(q_ready, uint32_t(si) & 1u)) break;
        for (int j = 0; j < n; ++j) {
          const int gj = base + j;
          const int st = gj % C::kStages;
          const uint32_t sb = tmem + ((gj & 1) ? C::kS1 : C::kS0);
          if (is_s) {
            // P of block j - 2 sits in the buffer that S overwrites.
            if (!wait(&k_full[st], uint32_t(gj / C::kStages) & 1u) ||
                (gj >= 2 && !wait(&o_done[gj & 1], uint32_t((gj - 2) >> 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t kd = kd0 + uint64_t((uint32_t(st) * C::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
              const uint64_t off = uint64_t((uint32_t(ks >> 2) * C::kHalf + uint32_t(ks & 3) * 32u) >> 4);
              mma_bf16_ss(sb, qd + off, kd + off, idesc_s, ks > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[gj & 1]);
            tc_commit(&k_empty[st]);
          } else {
            if (!wait(&v_full[st], uint32_t(gj / C::kStages) & 1u)) {
              ok = false;
              break;
            }
            const uint64_t vd = vd0 + uint64_t((uint32_t(st) * C::kTile) >> 4);
            for (int h = 0; h < 2; ++h) {
              if (!wait(&p_full[(gj & 1) * 2 + h], uint32_t(gj >> 1) & 1u)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                const uint64_t off = uint64_t((uint32_t(h) * 8192u + uint32_t(ks) * 2048u) >> 4);
                mma_bf16_ts(tmem + (h ? C::kOB : C::kOA), sb + uint32_t(64 * h + 8 * ks), vd + off, idesc_o,
                            (j > 0 || ks > 0) ? 1u : 0u);
              }
            }
            if (!ok) break;
            tc_commit(&o_done[gj & 1]);
            tc_commit(&v_empty[st]);
          }
        }
        if (!ok) break;
        tc_commit(o_final);
        base += n;
        ++si;
      }
      tc_commit(&drained[is_s ? 0 : 1]);
      mbar_wait(&drained[is_s ? 0 : 1], 0, drain_limit_ns(lim));
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ restore
    const int i = tid - 384;  // row of the block
    int gj = 0;
    bool ok = true;
    while (ok && walk.next(p, run, s)) {
      for (int j = s.j0; j < s.j1; ++j, ++gj) {
        const int rst = gj % C::kRawStages, st = gj % C::kStages;
        const uint32_t use = uint32_t(gj / C::kStages);
        if (!__all_sync(0xFFFFFFFFu, wait(&raw_full[rst], uint32_t(gj / C::kRawStages) & 1u)) ||
            (gj >= C::kStages && !__all_sync(0xFFFFFFFFu, wait(&k_empty[st], (use - 1u) & 1u)))) {
          ok = false;
          break;
        }
        const uint8_t* pg = smem + C::kRawOff + rst * C::kRaw + (i >> p.p_shift) * int(p.block);
        const int r = i & (p.P - 1);
        const uint32_t* par = reinterpret_cast<const uint32_t*>(pg + p.P * kD) + r;
        const uint32_t kp = par[0], vp = par[p.P];
        const bool past = j * kKeys + i >= s.keys;
        const bool odd = !past && not_finite(vp);
        restore_row<kD>(smem + C::kKOff + st * C::kTile, pg + r * (kD / 2), i, kp, past, odd ? 0x7FC07FC0u : 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[st]);
        if (gj >= C::kStages && !__all_sync(0xFFFFFFFFu, wait(&v_empty[st], (use - 1u) & 1u))) {
          ok = false;
          break;
        }
        restore_row<kD>(smem + C::kVOff + st * C::kTile, pg + (p.P + r) * (kD / 2), i, vp, past || odd, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&v_full[st]);
          mbar_arrive(&raw_empty[rst]);
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    // Warps 4-7 take keys 0-63 of every block, warps 8-11 keys 64-127; thread
    // (warp w, lane) owns row 32 (w % 4) + lane.
    const int q = warp & 3, h = (warp - 4) >> 2, r = q * 32 + lane;
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    const uint32_t o_own = tmem + lane_off + (h ? C::kOB : C::kOA);
    float2* xch = reinterpret_cast<float2*>(smem + C::kXchOff);
    int base = 0, si = 0;
    bool more = walk.next(p, run, s);
    while (more) {
      const int R = s.n * p.G;
      const int rr = s.tile * 128 + r;
      const bool valid = rr < R;
      const bool warp_live = __any_sync(0xFFFFFFFFu, valid);
      const int tok = valid ? rr / p.G : 0, hh = valid ? rr - tok * p.G : 0;
      // Q rows into the swizzled Q tile: thread (h, r) takes half the row's pieces.
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + s.b * p.q_b + tok * p.q_t +
                                                          (int64_t(s.h) * p.G + hh) * p.q_h) + h * (kD / 16);
        uint4 v[kD / 16];
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) v[k] = valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          const uint32_t piece = uint32_t(h * (kD / 16) + k);  // 8 dims
          *reinterpret_cast<uint4*>(smem + C::kQOff + (piece >> 3) * C::kHalf + uint32_t(r) * 128u +
                                    (((piece & 7u) ^ (uint32_t(r) & 7u)) << 4)) = v[k];
        }
      }
      uint32_t anc[4] = {0u, 0u, 0u, 0u};
      int limit = 0;  // keys before it are seen
      if (p.parents) {
        int pr[4];
        attn_impl::parent_row(p.parents + int64_t(s.b) * p.T, p.T, pr);
        attn_impl::tree_ancestors(pr, tok, p.T, valid, anc, p.status);
        limit = s.prefix;
      } else {
        limit = s.prefix + tok + 1;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(q_ready);
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      const int n = s.j1 - s.j0;
      for (int i = 0; i < n; ++i) {
        const int gi = base + i;
        const int kb = (s.j0 + i) * kKeys + 64 * h;
        if (!__all_sync(0xFFFFFFFFu, wait(&s_full[gi & 1], uint32_t(gi >> 1) & 1u))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (warp_live) {
          const uint32_t sc = tmem + lane_off + ((gi & 1) ? C::kS1 : C::kS0) + uint32_t(64 * h);
          uint32_t v[64];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_ld16(sc + uint32_t(ch * 16), *reinterpret_cast<uint32_t(*)[16]>(&v[ch * 16]));
          tmem_ld_wait64(v);
          if (kb + 64 > limit || !valid) mask_block<64>(v, kb, limit, anc, valid);
          const float mx = block_max<64>(v) * p.c;
          float factor = 1.f;
          if (mx > m_ref + 8.f) {
            factor = fast_exp2(m_ref - mx);  // 0 while m_ref = -inf
            m_ref = mx;
          }
          const float psum = exp_pack<64>(v, p.c, m_ref == -INFINITY ? 0.f : -m_ref);
          const bool resc = i > 0 && factor < 1.f && l > 0.f;
          if (__any_sync(0xFFFFFFFFu, resc)) {
            if (!__all_sync(0xFFFFFFFFu, wait(&o_done[(gi - 1) & 1], uint32_t((gi - 1) >> 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            rescale_row<kD>(o_own, resc ? factor : 1.f);
          }
          l = l * factor + psum;
          tmem_st16(sc, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
          tmem_st16(sc + 16u, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&p_full[(gi & 1) * 2 + h]);
      }
      // Epilogue: thread (h, r) joins the halves for dims (kD / 2) h .. of its row.
      const bool fin = __all_sync(0xFFFFFFFFu, ok && wait(o_final, uint32_t(si) & 1u));
      if (named_bar_any(1, 256, !fin)) break;
      tc_fence_after();
      xch[h * 128 + r] = make_float2(m_ref, l);
      named_bar_sync(1, 256);
      const float2 other = xch[(1 - h) * 128 + r];
      const float ma = h ? other.x : m_ref, la = h ? other.y : l;
      const float mb = h ? m_ref : other.x, lb = h ? l : other.y;
      const float M = fmaxf(ma, mb);
      const float wa = ma == M ? 1.f : fast_exp2(ma - M), wb = mb == M ? 1.f : fast_exp2(mb - M);
      const float den = wa * la + wb * lb;
      const bool whole = s.whole();
      const float inv = !whole ? 1.f : den == 0.f ? 0.f : 1.f / den;
      uint32_t* out = reinterpret_cast<uint32_t*>(
          p.O + ((int64_t(s.b) * p.T + tok) * p.Hq + int64_t(s.h) * p.G + hh) * kD + h * (kD / 2));
      float4* po = reinterpret_cast<float4*>(p.part_o) + (int64_t(blockIdx.x) * 2 + s.slot) * (kD / 4) * 128 + r;
      if (warp_live) {
#pragma unroll
        for (int ch = 0; ch < kD / 32; ++ch) {
          uint32_t a[16], b[16];
          tmem_ld16(tmem + lane_off + C::kOA + uint32_t(h * (kD / 2) + ch * 16), a);
          tmem_ld16(tmem + lane_off + C::kOB + uint32_t(h * (kD / 2) + ch * 16), b);
          tmem_ld_wait(a);
          tmem_ld_wait(b);
          float o[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = (wa * __uint_as_float(a[k]) + wb * __uint_as_float(b[k])) * inv;
          if (valid && whole) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint4 w;
              w.x = kv4::pack_bf16x2(o[8 * k], o[8 * k + 1]);
              w.y = kv4::pack_bf16x2(o[8 * k + 2], o[8 * k + 3]);
              w.z = kv4::pack_bf16x2(o[8 * k + 4], o[8 * k + 5]);
              w.w = kv4::pack_bf16x2(o[8 * k + 6], o[8 * k + 7]);
              reinterpret_cast<uint4*>(out)[ch * 2 + k] = w;
            }
          } else if (valid) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              po[(h * (kD / 8) + ch * 4 + k) * 128] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        if (h == 0 && valid) p.part_ml[(int64_t(blockIdx.x) * 2 + s.slot) * 128 + r] = make_float2(M, den);
        const int item = s.entry * p.Hkv + s.h;
        fence_acq_rel_gpu();
        named_bar_sync(1, 256);
        if (tid == 128) {
          const int add = s.j1 - s.j0;
          *merge_here = atomic_add_acq_rel_gpu(p.cnt + item, add) + add == s.nkb;
          if (*merge_here) p.cnt[item] = 0;
        }
        named_bar_sync(1, 256);
        if (*merge_here && valid) {
          fence_acq_rel_gpu();
          const int c0 = run_of(run, s.x0), c1 = run_of(run, s.x0 + s.nkb - 1);
          const int first = run_start(run, c0) >= s.x0 ? 0 : 1;
          float Mx = -INFINITY, L = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = __ldcg(p.part_ml + (int64_t(c) * 2 + (c == c0 ? first : 0)) * 128 + r);
            const float mn = fmaxf(Mx, ml.x);
            L = L * (Mx == mn ? 1.f : fast_exp2(Mx - mn)) + ml.y * (ml.x == mn ? 1.f : fast_exp2(ml.x - mn));
            Mx = mn;
          }
          const float scale = L == 0.f ? 0.f : 1.f / L;
          for (int ch = 0; ch < kD / 32; ++ch) {  // 16 dims at a time
            float o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const int64_t slot = int64_t(c) * 2 + (c == c0 ? first : 0);
              const float mx = __ldcg(p.part_ml + slot * 128 + r).x;
              const float f = mx == Mx ? 1.f : fast_exp2(mx - Mx);
              const float4* src = reinterpret_cast<const float4*>(p.part_o) + (slot * (kD / 4) + h * (kD / 8) + ch * 4) * 128 + r;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 v = __ldcg(src + k * 128);
                o[4 * k] = fmaf(f, v.x, o[4 * k]);
                o[4 * k + 1] = fmaf(f, v.y, o[4 * k + 1]);
                o[4 * k + 2] = fmaf(f, v.z, o[4 * k + 2]);
                o[4 * k + 3] = fmaf(f, v.w, o[4 * k + 3]);
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) out[ch * 8 + k] = kv4::pack_bf16x2(o[2 * k] * scale, o[2 * k + 1] * scale);
          }
        }
      }
      base += n;
      ++si;
      more = walk.next(p, run, s);
    }
  }

  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

}  // namespace kv4_attn
}  // namespace w12
