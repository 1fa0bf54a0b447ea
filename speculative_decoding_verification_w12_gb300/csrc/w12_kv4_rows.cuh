// Attention over the 4-bit cache for few query rows a kv head (single tokens,
// short blocks): streams the codes and multiplies them in registers.
//
// The floor is HBM: d + 8 bytes a (key, kv head) against at most 16 rows of work.
// 64 requests of 2048 to 8192 tokens (40 q / 8 kv heads x 128, 332 MB): 102 us, 3.3
// TB/s, 48 % of a copy's rate. What bounds it is the issue of about 380 instructions a
// 16-key group by seven warps a CTA, two CTAs an SM (59 % of the issue slots, the logic
// pipe 51 % busy): registers (128 a thread) allow no more warps, and nine a CTA at 96
// registers spill and take 106 us. (Two 8-row tiles at d = 128 run eleven warps at 168
// registers and spill 100 bytes.)
// A copy warp brings 128 keys at a time (their pages' blocks, one bulk copy
// each) into a ring in shared memory; each of the other warps takes groups of
// 16 keys. With few rows, a tensor-memory tile of 128 rows would be nearly
// empty and the restored operands would have to pass through shared memory;
// here a code word is restored straight into the registers of an
// mma.m16n8k16 operand, keys (or dims) on the 16-wide side and the rows on the
// 8-wide side:
//   S^T[16 keys, rows]  = K Q^T:  A = K codes, B = Q
//   O^T[16 dims, rows] += V^T P^T: A = V codes, B = P
// Codes are never scaled. A nibble of K, masked into place, is the fp16 subnormal q 2^-24
// (or q 2^-20, the nibble above it) as it stands; one of V is made q - 8. With
// z + s (q - 8) = (z - 8 s) + s q
//   score = c 2^a (s (q^.q) + (z - 8 s) sum(q^)),   c = scale log2(e)
//   o     = sum p~ (q - 8) + sum p~ z/s,            p~ = fp16(p s)
// with operands exact but for p~, which stands for the weight p~/s of the whole value (2^-11
// relative; with p z in place of p~ z/s the rounding would show where the two cancel). What is
// left are the sums: those of p~ (q - 8) and of p~ z/s round apart, in fp32, so next to a key
// with nearly all of the weight an output is off by up to a few 2^-24 of that key's 8 s; and the
// tensor cores sum products of subnormals with fewer bits (see key_codes). The powers of two of the K nibbles' places are made up for in Q (even
// pairs of dims times 16). A row of Q is held as q^ = q / 2^a, a power of two that keeps
// it in the fp16 range.
//
// Layout of the 16-key group: lane (g, t) = (lane / 4, lane % 4). K: key phi(g)
// (and 8 + phi(g)), dims (d/4) t ..: one 16-byte load per key gives all its A
// fragments. V: keys phi(2t), phi(2t+1) (and + 8), dims (d/8) g ..: the two
// keys' nibbles are paired by byte permutes. phi is the permutation
// 0 5 2 7 1 4 3 6, chosen with the layout's swapped halves so that both kinds of
// loads are free of bank conflicts.
//
// Weights are p = 2^(score - M). M follows the maximum of score + f - 8, 2^f a power of
// two that bounds the key's V row, so that p~ stays inside fp16 (2^5 where it is
// largest) and what it rounds to zero is below 2^-28 of what counts in o. It moves only
// when a p~ passes 2^14 (or p itself 2^112, which V rows of zeros allow): one vote a
// group, rescaling is rare.
#pragma once

#include "w12_attn_dev.cuh"
#include "w12_kv4_sched.cuh"

namespace w12 {
namespace kv4_attn {

using attn_impl::pack_f16x2;
using attn_impl::scaled_down;
using attn_impl::mbar_wait_asleep;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements spread over the warp (lane
// (g, t) holds row g, columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The four nibbles of both 16-bit halves of a K word as fp16 pairs: q 2^-24 in o[0]
// and o[2], q 2^-20 in o[1] and o[3]. Five operations a word. (The products of
// subnormal operands are summed with up to 10 bits less than others: 2^-13 of a step of
// the row's scale, far inside what a score's operands are rounded by.)
__device__ __forceinline__ void key_codes(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t v = w >> 8;
  o[0] = w & 0x000F000Fu;
  o[1] = w & 0x00F000F0u;
  o[2] = v & 0x000F000Fu;
  o[3] = v & 0x00F000F0u;
}

// Those of a V word as q - 8, exactly: masked into place, a nibble is 1024 + q or
// 1024 + 16 q. Nine operations a word; as subnormals the values of V came out up to
// 2^-13 of a step off, which shows in an output that is 0 where one key has the weight.
__device__ __forceinline__ void value_codes(uint32_t w, uint32_t (&o)[4]) {
  constexpr uint32_t k1024 = 0x64006400u, kM1032 = 0xE408E408u, kSixteenth = 0x2C002C00u, kM72 = 0xD480D480u;
  const uint32_t v = w >> 8;
  o[0] = hadd2(and_or(w, 0x000F000Fu, k1024), kM1032);
  o[1] = hfma2(and_or(w, 0x00F000F0u, k1024), kSixteenth, kM72);
  o[2] = hadd2(and_or(v, 0x000F000Fu, k1024), kM1032);
  o[3] = hfma2(and_or(v, 0x00F000F0u, k1024), kSixteenth, kM72);
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  float2 r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(r.x), "=f"(r.y) : "r"(v));
  return r;
}

// f of a row of V with the given parameters: |z| + 8 s < 2^f, at least -100 (rows
// of zeros; values that are not finite, whose weights are NaN all the same).
__device__ __forceinline__ float row_bound(uint32_t par) {
  const float half = fmaf(4.f, bf16_lo(par), 0.5f * fabsf(bf16_hi(par)));  // (the whole may pass the fp32 range)
  const int e = int((__float_as_uint(half) >> 23) & 255u) - 125;
  return float(e > 129 ? -100 : max(e, -100));
}

template <int kD, int kNT>
struct RowsCfg {
  static constexpr int kWarps = kNT == 1 ? 7 : 11;      // warps that compute (a multiple of 4 with the copy warp)
  static constexpr int kCtas = kNT == 1 ? 2 : 1;        // CTAs an SM
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kRows = 8 * kNT;
  static constexpr int kStage = kKeys * (kD + 8);
  static constexpr int kStages = kNT == 1 ? 4 : 6;
  static constexpr int kPitch = kD + 8;                 // floats of an output row in shared memory
  static constexpr int kOOff = kStages * kStage;
  static constexpr int kMlOff = kOOff + kWarps * kRows * kPitch * 4;
  static constexpr int kBarOff = kMlOff + kWarps * kRows * 8;
  static constexpr int kRunOff = kBarOff + 128;
  static constexpr int kSmem = kRunOff + 512;
};

template <int kD, int kNT>
__global__ void __launch_bounds__(RowsCfg<kD, kNT>::kThreads, RowsCfg<kD, kNT>::kCtas)
    kv4_attn_rows_kernel(const __grid_constant__ Params p) {
  using C = RowsCfg<kD, kNT>;
  constexpr int kComp = C::kWarps * 32;   // computing threads
  constexpr int kKW = kD / 32;            // code words of a key a lane reads (K)
  constexpr int kVW = kD / 64;            // and (V)
  constexpr int kMT = kD / 16;            // 16-dim tiles
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
  volatile int* merge_here = abort_flag + 1;
  RunSmem& rs = *reinterpret_cast<RunSmem*>(smem + C::kRunOff);
  static_assert(sizeof(RunSmem) <= 512 && C::kStages * 16 + 8 <= 128, "shared memory carve-up");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 8);  // one arrival per 16-key group
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_dep_wait();
  const Run run = plan_run<C::kThreads>(p, rs);  // its barriers publish the mbarriers too
  if (run.begin >= run.end) {
    if (warp == 0) zero_idle_rows<kD>(p);
    return;
  }
  const uint64_t lim = p.limit_ns;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait_asleep(bar, parity, lim, p.sleep_ns, abort_flag)) return true;
    if (*abort_flag) return false;
    set_status(p.status, W12_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
  };

  if (warp == C::kWarps) {
    // ------------------------------------------------------------- copies
    // Lane i brings the i-th page of a block; page ids are read one block ahead.
    const int per = kKeys >> p.p_shift;               // pages of a block (1 to 8)
    const uint32_t bytes = uint32_t(p.block);
    const uint64_t page_stride = uint64_t(p.Hkv) * uint64_t(p.block);
    int issued = 0;
    bool ok = true;
    Walk walk(run);
    Seg s;
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
        const int st = issued % C::kStages;
        if (issued >= C::kStages &&
            !__all_sync(0xFFFFFFFFu, wait(&empty[st], uint32_t(issued / C::kStages - 1) & 1u))) {
          ok = false;
          break;
        }
        const int pages = __popc(__ballot_sync(0xFFFFFFFFu, need));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], uint32_t(pages) * bytes);
        __syncwarp();
        if (need) bulk_load(smem + st * C::kStage + lane * bytes, pool + uint64_t(page) * page_stride, bytes, &full[st]);
        ++issued;
      }
    }
    grid_dep_launch();
    zero_idle_rows<kD>(p);
    // The CTA ends only with every copy landed, whatever the computing warps do: one of their
    // waits may still expire. (They need all copies, so this costs a call nothing.)
    for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
      mbar_wait(&full[i % C::kStages], uint32_t(i / C::kStages) & 1u, drain_limit_ns(lim));
    return;
  }

  // ---------------------------------------------------------------- compute
  const int g = lane >> 2, t = lane & 3;
  float* osm = reinterpret_cast<float*>(smem + C::kOOff);
  float2* mlsm = reinterpret_cast<float2*>(smem + C::kMlOff);
  const int phi_g = ((g >> 2) & 1) | (((g >> 1) & 1) << 1), row_k = phi_g ^ ((g & 1) ? 5 : 0);
  const int row_v = ((t >> 1) & 1) | ((t & 1) << 1);  // phi(2t); phi(2t + 1) = row_v ^ 5
  const int P = p.P;
  int group = 0;  // 16-key groups of the run before this segment
  Walk walk(run);
  Seg s;
  bool ok = true;
  while (walk.next(p, run, s)) {
    const int R = s.n * p.G;  // rows of the item
    // Q fragments: row 8 nt + g, dims (d/4) t .. + d/4 - 1, over 2^a.
    uint32_t q[kNT][kD / 8];
    float sq[kNT][2];           // sums of the rows 8 nt + 2t, + 1
    float cr[kNT][2];           // c 2^a of those rows
    uint32_t see[kNT][2];       // draft tokens those rows see (bit i: token i)
    // Scores come in units of 2^9 c 2^a, so that no product with a key passes the fp32
    // range, or of c 2^a where a row of Q is so large that 2^9 c 2^a might.
    float unit = 1.f;
    int ra[kNT];                // |q| < 2^ra in row 8 nt + g
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int r = 8 * nt + g;
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) q[nt][i] = 0u;
      if (r < R) {
        const int tok = r / p.G;
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + s.b * p.q_b + tok * p.q_t +
                                                          (int64_t(s.h) * p.G + (r - tok * p.G)) * p.q_h + t * (kD / 4));
#pragma unroll
        for (int i = 0; i < kD / 32; ++i) *reinterpret_cast<uint4*>(&q[nt][4 * i]) = __ldg(src + i);
      }
      uint32_t big = 0u;
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) big = max(big, max((q[nt][i] << 16) & 0x7FFFFFFFu, q[nt][i] & 0x7FFF0000u));
      big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
      big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
      ra[nt] = min(max(int(big >> 23) - 126, -100), 127);  // (a row with NaN or infinities stays one)
      if (__any_sync(0xFFFFFFFFu, ra[nt] > 100)) unit = 512.f;
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      // q^ = q 2^(11 - a), 16 times that where the codes are 2^-24 units: just inside fp16.
      const float down = __uint_as_float(uint32_t(127 + 11 - ra[nt]) << 23);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) {
        const float lo = bf16_lo(q[nt][i]) * down, hi = bf16_hi(q[nt][i]) * down;
        sum += lo + hi;
        q[nt][i] = (i & 1) ? pack_f16x2(lo, hi) : pack_f16x2(lo * 16.f, hi * 16.f);
      }
      sum *= 0x1p-20f * unit;
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      sq[nt][0] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t);
      sq[nt][1] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t + 4);
      const float cs = fmaxf(p.c * __uint_as_float(uint32_t(127 + ra[nt] + (unit == 1.f ? 9 : 0)) << 23), 1.2e-38f);
      cr[nt][0] = __shfl_sync(0xFFFFFFFFu, cs, 8 * t);
      cr[nt][1] = __shfl_sync(0xFFFFFFFFu, cs, 8 * t + 4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 8 * nt + 2 * t + e;
        uint32_t m = 0;
        if (rr < R) {
          const int tok = rr / p.G;
          if (!p.parents) {
            m = (2u << tok) - 1u;
          } else {
            const int32_t* par = p.parents + int64_t(s.b) * p.T;
            bool bad = false;
            for (int i = 0; i < p.T; ++i) bad |= i == 0 ? par[0] != -1 : (par[i] < 0 || par[i] >= i);
            if (bad) set_status(p.status, W12_ERR_BAD_TREE);
            for (int i = tok; i >= 0; i = bad ? -1 : par[i]) m |= 1u << i;
          }
        }
        see[nt][e] = m;
      }
    }
    float o[kNT][kMT][4], m[kNT][2], l[kNT][2], zs[kNT][2];
    float neg[kNT][2];  // -M, 0 while there is none
    bool fresh = true;  // some row has no M yet (the same in the whole warp)
    // Weights are held as 2^(score - M + lift), parameters of V over 2^lift: 0, or 40
    // once M has met value rows so large that 2^(score - M) might leave the fp32 range.
    float lift = 0.f, low = 1.f;  // low: 2^-lift
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int i = 0; i < kMT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = -INFINITY, l[nt][e] = zs[nt][e] = neg[nt][e] = 0.f;
    }
    const int group_end = group + (s.j1 - s.j0) * 8;
    // This warp's groups: those whose number is its own modulo kWarps.
    int gi = group + (C::kWarps + warp - group % C::kWarps) % C::kWarps;
    for (; gi < group_end; gi += C::kWarps) {
      const int blk = gi >> 3;
      const int st = blk % C::kStages;
      if (!__all_sync(0xFFFFFFFFu, wait(&full[st], uint32_t(blk / C::kStages) & 1u))) {
        ok = false;
        break;
      }
      const int sub = gi & 7;                                         // 16-key group of the block
      const int key0 = (s.j0 + blk - (group >> 3)) * kKeys + sub * 16;  // its first position
      if (key0 < s.keys) {
        const int r0 = (sub * 16) & (P - 1);
        const uint8_t* pg = smem + st * C::kStage + ((sub * 16) >> p.p_shift) * int(p.block);
        const uint8_t* kc = pg + (r0 + row_k) * (kD / 2);
        const uint32_t* par = reinterpret_cast<const uint32_t*>(pg + P * kD) + r0 + row_k;
        uint32_t ka[kKW], kb[kKW];
        if constexpr (kD == 128) {
          const int off = (t ^ (row_k & 2)) * 16;
          *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(kc + off);
          *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(kc + 8 * (kD / 2) + off);
        } else {
          *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(kc + t * 8);
          *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(kc + 8 * (kD / 2) + t * 8);
        }
        const uint32_t kpa = par[0], kpb = par[8], vpa = par[P], vpb = par[P + 8];
        float x[kNT][4], x2[kNT][4];  // two accumulators: half the chain of dependent products
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
          x2[nt][0] = x2[nt][1] = x2[nt][2] = x2[nt][3] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kKW; ++i) {
          uint32_t a[4], b[4];
          key_codes(ka[i], a);
          key_codes(kb[i], b);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma16816(x[nt], a[0], b[0], a[1], b[1], q[nt][4 * i], q[nt][4 * i + 1]);
            mma16816(x2[nt], a[2], b[2], a[3], b[3], q[nt][4 * i + 2], q[nt][4 * i + 3]);
          }
        }
        // x: scores without c 2^a, -inf where masked.
        const float ksa = bf16_lo(kpa), ksb = bf16_lo(kpb);
        const float kza = fmaf(-8.f, ksa, bf16_hi(kpa)), kzb = fmaf(-8.f, ksb, bf16_hi(kpb));
        const float kua = ksa * unit, kub = ksb * unit;
        const bool edge = key0 + 16 > s.prefix;
        uint32_t hidden = 0;  // bit 4 nt + i: element i is masked
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          x[nt][0] = fmaf(x[nt][0] + x2[nt][0], kua, sq[nt][0] * kza);
          x[nt][1] = fmaf(x[nt][1] + x2[nt][1], kua, sq[nt][1] * kza);
          x[nt][2] = fmaf(x[nt][2] + x2[nt][2], kub, sq[nt][0] * kzb);
          x[nt][3] = fmaf(x[nt][3] + x2[nt][3], kub, sq[nt][1] * kzb);
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rel = key0 + row_k + (i >= 2 ? 8 : 0) - s.prefix;  // draft token of the key
              const bool vis = rel < 0 ? see[nt][i & 1] != 0 : rel < 32 && ((see[nt][i & 1] >> rel) & 1u);
              if (!vis) {
                x[nt][i] = -INFINITY;
                hidden |= 1u << (4 * nt + i);
              }
            }
          }
        }
        float e[kNT][4], w[kNT][4], l2[kNT][2], vsa, vsb;
        bool move = fresh;
#pragma unroll 1
        for (;;) {
          if (move) {
            float fa = row_bound(vpa), fb = row_bound(vpb);
            float up = 1.f;
            if (lift == 0.f && __any_sync(0xFFFFFFFFu, fmaxf(fa, fb) > 86.f)) {
              lift = 40.f;
              up = 0x1p40f;
              low = 0x1p-40f;
            }
            fa = fmaxf(fa, lift - 100.f) - 8.f;
            fb = fmaxf(fb, lift - 100.f) - 8.f;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaf(x[nt][r], cr[nt][r], fa), fmaf(x[nt][2 + r], cr[nt][r], fb));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
                mx = fmaxf(mx, m[nt][r]);
                const float m_old = m[nt][r], f = m_old == mx ? 1.f : ex2(m_old - mx);  // 0 while m = -inf
                m[nt][r] = mx;
                l[nt][r] = scaled_down(l[nt][r], m_old == mx ? 0.f : m_old - mx) * up;
                zs[nt][r] *= f;
#pragma unroll
                for (int i = 0; i < kMT; ++i) {
                  o[nt][i][r] *= f;
                  o[nt][i][2 + r] *= f;
                }
                neg[nt][r] = mx == -INFINITY ? 0.f : lift - mx;
              }
            bool none = false;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) none |= m[nt][0] == -INFINITY || m[nt][1] == -INFINITY;
            fresh = __any_sync(0xFFFFFFFFu, none);
          }
          vsa = bf16_lo(vpa) * low, vsb = bf16_lo(vpb) * low;
          float most = 0.f, sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            e[nt][0] = ex2(fmaf(x[nt][0], cr[nt][0], neg[nt][0]));
            e[nt][1] = ex2(fmaf(x[nt][1], cr[nt][1], neg[nt][1]));
            e[nt][2] = ex2(fmaf(x[nt][2], cr[nt][0], neg[nt][0]));
            e[nt][3] = ex2(fmaf(x[nt][3], cr[nt][1], neg[nt][1]));
            w[nt][0] = e[nt][0] * vsa;
            w[nt][1] = e[nt][1] * vsa;
            w[nt][2] = e[nt][2] * vsb;
            w[nt][3] = e[nt][3] * vsb;
            most = fmaxf(most, fmaxf(fmaxf(w[nt][0], w[nt][1]), fmaxf(w[nt][2], w[nt][3])));
            l2[nt][0] = e[nt][0] + e[nt][2];
            l2[nt][1] = e[nt][1] + e[nt][3];
            sum += l2[nt][0] + l2[nt][1];
          }
          if (move || !__any_sync(0xFFFFFFFFu, most > 16384.f || sum > 0x1p112f)) break;
          move = true;
        }
        // A key adds p~ z/s, or p z where |z| >= 16 s (z/s may not be there).
        const float ta = bf16_hi(vpa) * rcp(bf16_lo(vpa)), tb = bf16_hi(vpb) * rcp(bf16_lo(vpb));
        const bool ina = fabsf(ta) < 16.f, inb = fabsf(tb) < 16.f;
        const float k1a = ina ? ta : 0.f, k2a = ina ? 0.f : bf16_hi(vpa) * low;
        const float k1b = inb ? tb : 0.f, k2b = inb ? 0.f : bf16_hi(vpb) * low;
        uint32_t pb[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          const uint32_t hd = edge ? hidden >> (4 * nt) : 0u;
          if (edge) {  // parameters in masked places may be anything
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((hd >> i) & 1u) w[nt][i] = 0.f;
          }
          l[nt][0] += l2[nt][0];
          l[nt][1] += l2[nt][1];
          const uint32_t ra = pack_f16x2(w[nt][0], w[nt][1]), rb = pack_f16x2(w[nt][2], w[nt][3]);
          pb[nt][0] = transpose8x8(ra);
          pb[nt][1] = transpose8x8(rb);
          const float2 fa = unpack_f16x2(ra), fb = unpack_f16x2(rb);  // the weights as they are multiplied
          float z[4] = {fmaf(fa.x, k1a, e[nt][0] * k2a), fmaf(fa.y, k1a, e[nt][1] * k2a),
                        fmaf(fb.x, k1b, e[nt][2] * k2b), fmaf(fb.y, k1b, e[nt][3] * k2b)};
          if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((hd >> i) & 1u) z[i] = 0.f;
          }
          zs[nt][0] += z[0] + z[2];
          zs[nt][1] += z[1] + z[3];
        }
        // V: keys phi(2t), phi(2t + 1) and 8 further, dims (d/8) g ..
        const uint8_t* vc = pg + P * (kD / 2) + r0 * (kD / 2);
        uint32_t v[4][kVW];  // keys: 2t, 2t + 1, 2t + 8, 2t + 9 of the group's order
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = ((k & 1) ? row_v ^ 5 : row_v) + ((k & 2) ? 8 : 0);
          if constexpr (kD == 128)
            *reinterpret_cast<uint2*>(v[k]) =
                *reinterpret_cast<const uint2*>(vc + r * (kD / 2) + ((g * 8) ^ ((r & 2) << 4)));
          else
            v[k][0] = *reinterpret_cast<const uint32_t*>(vc + r * (kD / 2) + g * 4);
        }
#pragma unroll
        for (int e = 0; e < kVW; ++e) {
          const uint32_t lo0 = __byte_perm(v[0][e], v[1][e], 0x5410), hi0 = __byte_perm(v[0][e], v[1][e], 0x7632);
          const uint32_t lo1 = __byte_perm(v[2][e], v[3][e], 0x5410), hi1 = __byte_perm(v[2][e], v[3][e], 0x7632);
          uint32_t a0[4], a1[4], a2[4], a3[4];
          value_codes(lo0, a0);
          value_codes(hi0, a1);
          value_codes(lo1, a2);
          value_codes(hi1, a3);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
              mma16816(o[nt][4 * e + j], a0[j], a1[j], a2[j], a3[j], pb[nt][0], pb[nt][1]);
        }
      }
      fence_proxy_async_smem();  // these reads come before the copy that refills the stage
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    group = group_end;
    // ------------------------------------------------------------ epilogue
    // The warps' results meet in shared memory: o (dims 2j of word e at
    // ((4 e + j) 8 + g) 2), then every row's sum over the warps.
    if (named_bar_any(1, kComp, !ok)) break;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float ls = l[nt][e], z = zs[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          ls += __shfl_xor_sync(0xFFFFFFFFu, ls, x);
          z += __shfl_xor_sync(0xFFFFFFFFu, z, x);
        }
        const int r = 8 * nt + 2 * t + e;
        if (g == 0) mlsm[warp * C::kRows + r] = make_float2(m[nt][e], ls * low);
        float* dst = osm + (warp * C::kRows + r) * C::kPitch + g * 2;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
          *reinterpret_cast<float2*>(dst + i * 16) =
              make_float2(o[nt][i][e] + z, o[nt][i][2 + e] + z);
      }
    named_bar_sync(1, kComp);
    const bool whole = s.whole();
    float* po = p.part_o + (int64_t(blockIdx.x) * 2 + s.slot) * C::kRows * kD;
    float2* pml = p.part_ml + (int64_t(blockIdx.x) * 2 + s.slot) * C::kRows;
    // Output pairs of dims: pair pd is dims 2 pd, 2 pd + 1.
    auto out_row = [&](int r) -> uint32_t* {
      const int tok = r / p.G;
      return reinterpret_cast<uint32_t*>(p.O + ((int64_t(s.b) * p.T + tok) * p.Hq + int64_t(s.h) * p.G + (r - tok * p.G)) * kD);
    };
    for (int i = tid; i < R * (kD / 2); i += kComp) {
      const int r = i / (kD / 2), pd = i - r * (kD / 2);
      const int at = kD == 128 ? ((((pd >> 2) & 1) * 4 + (pd & 3)) * 8 + (pd >> 3)) * 2 : ((pd & 3) * 8 + (pd >> 2)) * 2;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, mlsm[w * C::kRows + r].x);
      float L = 0.f, a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 ml = mlsm[w * C::kRows + r];
        const float d = ml.x == M ? 0.f : ml.x - M, f = ex2(d);
        const float2 v = *reinterpret_cast<const float2*>(osm + (w * C::kRows + r) * C::kPitch + at);
        L += scaled_down(ml.y, d);
        a = fmaf(f, v.x, a);
        b = fmaf(f, v.y, b);
      }
      if (whole) {
        out_row(r)[pd] = L == 0.f ? 0u : pack_bf16x2(a / L, b / L);  // (1 / L may pass the fp32 range)
      } else {
        *reinterpret_cast<float2*>(po + r * kD + 2 * pd) = make_float2(a, b);
        if (pd == 0) pml[r] = make_float2(M, L);
      }
    }
    if (!whole) {
      // (The barrier orders the CTA's stores before the one release, and its acquire before all loads.)
      named_bar_sync(1, kComp);
      if (tid == 0) {
        const int add = s.j1 - s.j0;
        int32_t* cnt = p.cnt + run_of(run, s.x0);
        *merge_here = atomic_add_acq_rel_gpu(cnt, add) + add == s.nkb;
        if (*merge_here) *cnt = 0;
      }
      named_bar_sync(1, kComp);
      if (*merge_here) {
        // Only the first of the item's CTAs can have begun its run before the item.
        const int c0 = run_of(run, s.x0), c1 = run_of(run, s.x0 + s.nkb - 1);
        const int first = run_start(run, c0) >= s.x0 ? 0 : 1;
        for (int i = tid; i < R * (kD / 2); i += kComp) {
          const int r = i / (kD / 2), pd = i - r * (kD / 2);
          float M = -INFINITY, L = 0.f, a = 0.f, b = 0.f;
          for (int c = c0; c <= c1; c += 4) {  // four partials' loads in flight
            float2 ml[4], v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int64_t slot = int64_t(c + u) * 2 + (c + u == c0 ? first : 0);
              ml[u] = make_float2(-INFINITY, 0.f);
              v[u] = make_float2(0.f, 0.f);
              if (c + u <= c1) {
                ml[u] = __ldcg(p.part_ml + slot * C::kRows + r);
                v[u] = __ldcg(reinterpret_cast<const float2*>(p.part_o + (slot * C::kRows + r) * kD) + pd);
              }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float mn = fmaxf(M, ml[u].x);
              const float da = M == mn ? 0.f : M - mn, db = ml[u].x == mn ? 0.f : ml[u].x - mn;
              const float fa = ex2(da), fb = ex2(db);
              L = scaled_down(L, da) + scaled_down(ml[u].y, db);
              a = a * fa + fb * v[u].x;
              b = b * fa + fb * v[u].y;
              M = mn;
            }
          }
          out_row(r)[pd] = L == 0.f ? 0u : pack_bf16x2(a / L, b / L);
        }
      }
    }
    named_bar_sync(1, kComp);  // shared memory is free for the next segment
  }
}

}  // namespace kv4_attn
}  // namespace w12
