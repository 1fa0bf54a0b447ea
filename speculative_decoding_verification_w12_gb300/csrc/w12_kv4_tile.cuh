// Attention over the 4-bit cache for many query rows a kv head (draft blocks and
// trees, prompt chunks): 128-row tiles on the tensor memory.
//
// The floor is the tensor pipe (1024 cycles a tile and block at d = 128), or HBM for a
// single tile of rows. 4 trees of 64 nodes over 32768 tokens: 211 us, 0.81 PFLOP/s of
// the 320 rows, 42 % of the measured bf16 rate; 16 blocks of 16 over 8192: 86 us, 26 % of
// either bound; prompt chunk 2 x 2048 (d 64): 142 us. A block takes 2400 cycles of a
// CTA: the softmax and restore warps (two of each a scheduler) issue 48 to 50 % of the
// slots (60 % at d = 64) and wait on one another's and on tensor-memory latencies for the
// rest.
//
// Work unit: 128 query rows of one (request, kv head), token-major, against one
// block of 128 keys (the split is w12_kv4_sched.cuh's). Per block:
//   segments, tree ancestors     ahead of their use (warp 3)
//   raw pages -> shared memory   one bulk copy a page (warp 0)
//   codes -> fp16 K and V tiles  eight warps, four for each; a thread restores one row
//   S = Q K^T                    tcgen05.mma, D in TMEM, two buffers (warp 1)
//   P = exp2(S - M)              two warpgroups, one a 64-key part of the block; P
//                                over its part's first 32 S columns as fp16 pairs
//   O_h += P_h V_h               tcgen05.mma, A = P from TMEM, V MN-major (warp 2)
//
// Operands are fp16 (2^-11 relative) rather than bf16 (2^-8): restored values
// z + s (q - 8) and P then add little that shows next to the output's own
// rounding to bf16. Their range is kept by powers of two, which are exact: every
// 32 keys (one restore warp) have an exponent e for K and f + 8 for V, the largest
// of their rows', as long as no row's own is more than 8 below it (of K: no row but
// zeros); otherwise each of the 32 keys has its own. So a row keeps its values to 2^-11
// relative or 2^-16 of its own bound, whatever stands beside it: a key of another
// size, seen or masked, does not coarsen it. (Exponents a key for all would cost the
// softmax two loads and three operations more for each pair of scores. As it is, trees
// take 211 us where one exponent for any 32 rows took 205, blocks 86 for 82, the prompt
// chunk 142 for 140.)
// The tile holds K / 2^e and V / 2^(f + 8), and a row of Q is held over its own power
// of two 2^a. With
//   y_ij = c 2^(a_i + e_j) S_ij + f_j,       c = scale log2(e)
// the weight that meets the scaled V is P = 2^(y - M), M a running maximum of y less
// kTop: the largest weight was 2^8 when M was set, so weights are rounded to 2^-11
// relative down to 2^-22 of it, and below that to 2^-33 of it (a key with nearly all of
// the weight may add little, as the first of a long cache often does: the others keep
// theirs). The denominator sum of 2^(y - M) / 2^f_j is kept in fp32, and the output is
// 2^8 times their quotient.
//
// The softmax takes 32 scores at a time and does not look for a block's maximum: it
// uses the running M, and only if the 32 weights sum to more than kMost (the first
// block, or scores that grow along the keys) does it find the maximum and do the
// block again (S is still in TMEM). Weights then stay inside fp16. The two
// warpgroups keep separate maxima, sums and O accumulators, joined in the epilogue.
//
// A key whose V parameters are not finite gets V = 0 and K = NaN: its score is
// NaN for the rows that see it and masked for the others, which P = 0 times NaN
// would not leave alone. Rows of the block past the keys get K = V = 0.
#pragma once

#include "w12_attn_dev.cuh"
#include "w12_kv4_sched.cuh"

namespace w12 {
namespace kv4_attn {

using attn_impl::block_max;
using attn_impl::add2;
using attn_impl::fma2;
using attn_impl::pack_f16x2;
using attn_impl::fast_exp2;
using attn_impl::mask_block;
using attn_impl::rescale_row;
using attn_impl::scaled_down;
using attn_impl::mbar_wait_asleep;
using attn_impl::sdesc_mn_sw128;

// True for one lane of the (converged) warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Registers of the calling warp's threads, from here on; all warps of its warpgroup call it.
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// idesc_bf16 with fp16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

constexpr int kSpread = 8;               // rows of a 32-key group may be this much smaller, as powers of two
// Least exponents of rows: the smallest ones still keep 2^-16 of their bound (2^-97 with
// the smallest scale), and 2^24 keys of value rows of zeros their sum of weights 2^(8 - f).
constexpr int kLeastK = -92, kLeastV = -88;
// Exponent of a row of V below which keys have their own: 2^(score + f - M) may then be below
// the fp32 range where 2^(score - M) is not (M may be of rows 2^134 larger).
constexpr int kSmallV = -44;
constexpr float kTop = 8.f;              // the largest weight when the running maximum was set, as a power of two
constexpr float kMost = 61440.f;         // sum of 32 weights above which it moves (fp16 ends at 65504)

template <int kD>
struct TileCfg {
  // Parts of a block's keys with softmax warps, a maximum and an O of their own. (Four at
  // d = 64, where O has room: 16 softmax warps at 72 registers, prompt chunk 146 us for 134.)
  static constexpr int kParts = 2;
  static constexpr int kPart = 128 / kParts;              // keys of a part
  static constexpr int kSoft = 4 * kParts;                // softmax warps, from warp 4 on
  static constexpr int kRest = 4 + kSoft;                 // eight restore warps from here; 0-3 copy, issue, plan
  static constexpr int kThreads = (kRest + 8) * 32;
  // Registers a thread from the role's start on, of the 96 that the launch has for each
  // (checked there): the softmax, with code of its own for keys that have exponents of
  // their own, spills at 96 (blocks 89 us for 85, trees 217 for 210.5). A warpgroup changes
  // its registers by one instruction that all its warps meet.
  static constexpr int kLaunchRegs = 96, kPlainRegs = 88, kSoftRegs = 112, kRestRegs = 80;
  static_assert(kPlainRegs * 4 + kSoftRegs * kSoft + kRestRegs * 8 <= kLaunchRegs * (kThreads / 32),
                "the launch's registers");
  static constexpr uint32_t kHalf = 128u * 128u;       // 128 rows x 64 fp16, 128-byte swizzle
  static constexpr uint32_t kTile = kHalf * (kD / 64);
  static constexpr uint32_t kRaw = uint32_t(kKeys) * (kD + 8);
  static constexpr int kRawStages = kD == 128 ? 3 : 6;
  static constexpr int kStages = 2;        // restored K and V tiles
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kKOff = kTile;
  static constexpr uint32_t kVOff = kKOff + kStages * kTile;
  static constexpr uint32_t kRawOff = kVOff + kStages * kTile;
  static constexpr uint32_t kXchOff = kRawOff + kRawStages * kRaw;  // (m, l) of the parts
  static constexpr uint32_t kQxOff = kXchOff + kParts * 128 * 8;         // [2][128] powers of two of Q rows
  // Exponents of the restored tiles, by block modulo 4 and 32 keys: (c 2^(e - 8), f, 2^-f,
  // whether the keys have their own), and those of the keys, (c 2^(e - 8), f), where they do.
  // Four deep: K of block j + 2 may be restored while the softmax of block j still reads.
  static constexpr int kExpRing = 4;
  static constexpr uint32_t kExpOff = kQxOff + 2 * 128 * 4;
  static constexpr uint32_t kKeyOff = kExpOff + kExpRing * 4 * 16;
  static constexpr uint32_t kBarOff = kKeyOff + kExpRing * 128 * 8;
  static constexpr uint32_t kRunOff = kBarOff + 384;
  static constexpr uint32_t kSegOff = kRunOff + 512;
  static constexpr uint32_t kAncOff = kSegOff + 256;                // [2][128] sets, then 128 words
  static constexpr uint32_t kSmem = kAncOff + 2 * 128 * 16 + 512 + 1024;  // 1024: alignment slack
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  // TMEM columns: S of even and odd blocks, O of the parts (kD columns each).
  static constexpr uint32_t kS0 = 0, kS1 = 128, kO = 256, kCols = 512;
  static_assert(kO + kParts * kD <= kCols, "tensor memory");
};

// Eight dims of a code word as fp16 values z + s (q - 8), s2 and z2 holding s and
// z in both halves. A nibble in the lowest bits of fp16 1024 is 1024 + q, in the
// next four 1024 + 16 q; both become q - 8 exactly, then one rounding. Two operations
// instead of three would give (z - 8 s) + s q with z - 8 s rounded first (trees 189 us
// for 204, blocks 77 for 82), but that shifts a whole row by up to 2^-11 of its largest
// value: where one key has most of the weight, outputs near 0 came out 2 % off. For K
// alone, as code of its own beside V's, it gains nothing (200, 88).
__device__ __forceinline__ uint4 restore_word(uint32_t w, uint32_t s2, uint32_t z2) {
  constexpr uint32_t k1024 = 0x64006400u, kM1032 = 0xE408E408u, kSixteenth = 0x2C002C00u, kM72 = 0xD480D480u;
  const uint32_t v = w >> 8;
  uint4 o;
  o.x = hfma2(hadd2(and_or(w, 0x000F000Fu, k1024), kM1032), s2, z2);
  o.y = hfma2(hfma2(and_or(w, 0x00F000F0u, k1024), kSixteenth, kM72), s2, z2);
  o.z = hfma2(hadd2(and_or(v, 0x000F000Fu, k1024), kM1032), s2, z2);
  o.w = hfma2(hfma2(and_or(v, 0x00F000F0u, k1024), kSixteenth, kM72), s2, z2);
  return o;
}

// Exponent of a power of two that no value of a row passes: |z| + 8 s < 2^e, at least
// `least`; that, too, for rows of zeros and of values that are not finite. At most 129.
__device__ __forceinline__ int row_exponent(uint32_t par, int least) {
  const float half = fmaf(4.f, bf16_lo(par), 0.5f * fabsf(bf16_hi(par)));  // (the whole may pass the fp32 range)
  const int e = int((__float_as_uint(half) >> 23) & 255u) - 125;
  return e > 129 ? least : max(e, least);  // 130: inf or NaN
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Where thread i of a block restores its row: the 16-byte pieces of its codes are
// taken in an order that differs from row to row, so that the eight rows of a
// shared-memory phase read and write different banks. Piece k is at byte 16 at(k)
// of the row's codes and holds dims 32 c .. 32 c + 31; its word m goes to
// dst(k) + word(m) of the row's 128-byte-swizzled tile.
template <int kD>
struct RowPlace {
  static constexpr int kPieces = kD / 32;
  uint32_t at[kPieces], dst[kPieces], word[4];
  __device__ __forceinline__ explicit RowPlace(int i) {
    const uint32_t x = uint32_t(i) & 7u;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const uint32_t a = (kD == 128 ? (uint32_t(i) >> 1) + k : (uint32_t(i) >> 2) + k) & (kPieces - 1);
      const uint32_t c = a ^ (kD == 128 ? uint32_t(i) & 2u : 0u);  // halves swapped in rows with bit 1 set
      at[k] = a * 16u;
      dst[k] = (c >> 1) * 16384u + uint32_t(i) * 128u + ((((c & 1u) * 4u) ^ (x & 4u)) << 4);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) word[m] = (uint32_t(m) ^ (x & 3u)) << 4;
  }
};

__device__ __forceinline__ bool not_finite(uint32_t par) {
  return (par & 0x7F80u) == 0x7F80u || (par & 0x7F800000u) == 0x7F800000u;
}

// Each thread of the warp reads 32 consecutive 32-bit columns of its own lane;
// valid after tmem_ld_wait32, which ties the values to the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : W12_TIE8(v, 0), W12_TIE8(v, 8), W12_TIE8(v, 16), W12_TIE8(v, 24)
               :
               : "memory");
}

// 2^(c v + b) of 32 scores: fp16 pairs into out[0 .. 16), returns the fp32 sum.
__device__ __forceinline__ float exp_pack_f16(const uint32_t (&v)[32], float c, float b, uint32_t* out) {
  float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 c2 = make_float2(c, c), b2 = make_float2(b, b);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 y = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2, b2);
    const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
    sum[k & 3] = add2(sum[k & 3], e);
    out[k] = pack_f16x2(e.x, e.y);
  }
  const float2 s = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  return s.x + s.y;
}

// Scores of 32 keys with exponents of their own, (c 2^(e - 8), f) each in key: v becomes
// y = score + f. Returns the sum of the keys' 2^(score - ref).
__device__ __forceinline__ float key_scores(uint32_t (&v)[32], const float2* key, float up, float ref) {
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float4 x = reinterpret_cast<const float4*>(key)[k];
    const float s0 = __uint_as_float(v[2 * k]) * fmaxf(x.x * up, 1.2e-38f);
    const float s1 = __uint_as_float(v[2 * k + 1]) * fmaxf(x.z * up, 1.2e-38f);
    sum += fast_exp2(s0 - ref) + fast_exp2(s1 - ref);
    v[2 * k] = __float_as_uint(s0 + x.y);
    v[2 * k + 1] = __float_as_uint(s1 + x.w);
  }
  return sum;
}

// A segment as warp 3 hands it to the softmax warps, two ahead at most.
struct SegSlot {
  Seg seg;
  int more;  // 0: the run is over
};
static_assert(sizeof(SegSlot) <= 128, "shared memory carve-up");

// Ancestors of a draft tree's nodes, themselves included, as 128-bit sets in anc[0 .. T),
// by one warp, four nodes a lane: each round a node joins the set of the node that its
// pointer has reached and moves on to that node's pointer, so paths double in length.
// at: 128 words of shared memory. A malformed tree is flagged and every node then sees
// itself alone.
__device__ __forceinline__ void ancestors_of(const int32_t* parents, int T, uint4* anc, int* at, int32_t* status) {
  const int lane = threadIdx.x & 31;
  int to[4];
  uint4 a[4];
  attn_impl::parent_row(parents, T, to);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    if (i < T) bad |= i == 0 ? to[k] != -1 : (to[k] < 0 || to[k] >= i);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (bad && lane == 0) set_status(status, W12_ERR_BAD_TREE);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t own = 1u << lane;
    a[k] = make_uint4(k == 0 ? own : 0u, k == 1 ? own : 0u, k == 2 ? own : 0u, k == 3 ? own : 0u);
    if (bad) to[k] = -1;
    anc[lane + 32 * k] = a[k];
    at[lane + 32 * k] = to[k];
  }
  __syncwarp();
  for (int round = 0; round < 7; ++round) {
    bool on = false;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (to[k] >= 0) {
        const uint4 x = anc[to[k]];
        a[k] = make_uint4(a[k].x | x.x, a[k].y | x.y, a[k].z | x.z, a[k].w | x.w);
        to[k] = at[to[k]];
        on = true;
      }
    if (!__any_sync(0xFFFFFFFFu, on)) break;  // (the vote also keeps these reads before the writes)
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      anc[lane + 32 * k] = a[k];
      at[lane + 32 * k] = to[k];
    }
    __syncwarp();
  }
}

// A softmax warp's share of a segment's Q rows into the swizzled fp16 Q tile: each over a
// power of two 2^ra[row] that brings it below 2^10, so that c 2^(e - 8) and 2^(ra + 8) have
// room up to the largest values. A row with NaN or infinities stays one.
template <int kD>
__device__ __forceinline__ void load_q(const Params& p, const Seg& s, int share, uint8_t* tile, int* ra) {
  constexpr int kRows = 128 / TileCfg<kD>::kSoft;
  constexpr int kLanes = kD / 8, kStep = 32 / kLanes, kN = kRows / kStep;  // lanes a row, rows a load, loads
  const int lane = threadIdx.x & 31, c = lane % kLanes, r0 = share * kRows + lane / kLanes;
  const int R = s.n * p.G;
  const uint16_t* q = p.Q + s.b * p.q_b + int64_t(s.h) * p.G * p.q_h + c * 8;
  int rr = s.tile * 128 + r0, tok = rr / p.G, hh = rr - tok * p.G;
  uint4 v[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    v[k] = rr < R ? __ldg(reinterpret_cast<const uint4*>(q + tok * p.q_t + hh * p.q_h)) : make_uint4(0, 0, 0, 0);
    rr += kStep;
    for (hh += kStep; hh >= p.G; hh -= p.G) ++tok;
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t big = 0u;
#pragma unroll
    for (int x = 0; x < 4; ++x) big = max(big, max((w[x] << 16) & 0x7FFFFFFFu, w[x] & 0x7FFF0000u));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
    const int a = min(max(int(big >> 23) - 126, -100), 128) - 10, r = r0 + k * kStep;
    const float down = pow2(-a);
    uint4 o;
    o.x = pack_f16x2(bf16_lo(w[0]) * down, bf16_hi(w[0]) * down);
    o.y = pack_f16x2(bf16_lo(w[1]) * down, bf16_hi(w[1]) * down);
    o.z = pack_f16x2(bf16_lo(w[2]) * down, bf16_hi(w[2]) * down);
    o.w = pack_f16x2(bf16_lo(w[3]) * down, bf16_hi(w[3]) * down);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * TileCfg<kD>::kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = o;
    if (c == 0) ra[r] = a;
  }
}

template <int kD>
__global__ void __launch_bounds__(TileCfg<kD>::kThreads, 1) kv4_attn_tile_kernel(const __grid_constant__ Params p) {
  using C = TileCfg<kD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (An offset, not a rounded pointer: the compiler then still knows that it is shared memory.)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // pages of a block landed
  uint64_t* raw_empty = raw_full + C::kRawStages;                       // and restored (one arrival a warp)
  uint64_t* k_full = raw_empty + C::kRawStages;                         // K tile restored
  uint64_t* k_empty = k_full + C::kStages;                              // S of its block done
  uint64_t* v_full = k_empty + C::kStages;
  uint64_t* v_empty = v_full + C::kStages;                              // P V of its block done
  uint64_t* s_full = v_empty + C::kStages;                              // [2] S of block i in buffer i % 2
  uint64_t* p_full = s_full + 2;                                        // [2][parts] P of block i, part h
  uint64_t* o_done = p_full + 2 * C::kParts;                            // [2] P V of block i (all parts) done
  uint64_t* o_final = o_done + 2;                                       // P V of the segment's last block done
  uint64_t* o_free = o_final + 1;                                       // O of the segment read (one arrival a warp)
  uint64_t* q_full = o_free + 1;                                        // its Q stored (one arrival a warp)
  uint64_t* drained = q_full + 1;                                      // [2]
  uint64_t* seg_full = drained + 2;                                     // [2] segment i found, in slot i % 2
  uint64_t* seg_empty = seg_full + 2;                                   // [2] and done with (one arrival a warp)
  uint64_t* anc_full = seg_empty + 2;                                   // [2] its tree's ancestors found
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(anc_full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* merge_here = abort_flag + 1;
  RunSmem& rs = *reinterpret_cast<RunSmem*>(smem + C::kRunOff);
  float4* exps = reinterpret_cast<float4*>(smem + C::kExpOff);
  float2* key_exps = reinterpret_cast<float2*>(smem + C::kKeyOff);
  SegSlot* segs = reinterpret_cast<SegSlot*>(smem + C::kSegOff);
  uint4* ancs = reinterpret_cast<uint4*>(smem + C::kAncOff);
  int* qx = reinterpret_cast<int*>(smem + C::kQxOff);
  static_assert((2 * C::kRawStages + 4 * C::kStages + 15 + 2 * C::kParts) * 8 + 16 <= 384 && sizeof(RunSmem) <= 512, "carve-up");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 8);
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
      mbar_init(&seg_full[k], 1);
      mbar_init(&seg_empty[k], C::kSoft);
      mbar_init(&anc_full[k], 1);
    }
    for (int k = 0; k < 2 * C::kParts; ++k) mbar_init(&p_full[k], 128);
    mbar_init(o_final, 1);
    mbar_init(o_free, C::kSoft);
    mbar_init(q_full, C::kSoft);
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_dep_wait();
  plan_run<C::kThreads>(p, rs);  // its barriers publish the mbarriers too
  const Run& run = rs.run;       // read where it is used: registers are short
  if (run.begin >= run.end) {
    if (warp == 0) zero_idle_rows<kD>(p);
    return;
  }
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
    if (mbar_wait_asleep(bar, parity, lim, p.sleep_ns, abort_flag)) return true;
    if (*abort_flag) return false;
    set_status(p.status, W12_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
  };

  if (warp < 4) {
    fewer_registers<C::kPlainRegs>();
    if (warp == 0) {
      // ------------------------------------------------------------- copies
      Walk walk(run);
      Seg s;
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
      // The CTA ends only with every copy landed, whatever the other warps do: one of their waits
      // may still expire. (They need all copies, so this costs a call nothing.)
      for (int i = issued > C::kRawStages ? issued - C::kRawStages : 0; i < issued; ++i)
        mbar_wait(&raw_full[i % C::kRawStages], uint32_t(i / C::kRawStages) & 1u, drain_limit_ns(lim));
    } else if (warp == 1 || warp == 2) {
      // ---------------------------------------------------------------- MMA
      // The whole warp waits; one elected lane issues. (With the loop under one
      // lane, descriptors pass from vector to uniform registers product by product.)
      const uint32_t sbase = smem_u32(smem);
      const bool is_s = warp == 1;
      const uint64_t qd = sdesc_k_sw128(sbase + C::kQOff);
      const uint64_t kd0 = sdesc_k_sw128(sbase + C::kKOff);
      const uint64_t vd0 = sdesc_mn_sw128(sbase + C::kVOff, C::kHalf);
      constexpr uint32_t idesc_s = idesc_f16(128, 128);
      constexpr uint32_t idesc_o = idesc_f16(128, kD) | (1u << 16);  // B (V) MN-major
      auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
      Walk walk(run);
      Seg s;
      int base = 0, si = 0;
      bool ok = true;
      while (ok && walk.next(p, run, s)) {
        const int n = s.j1 - s.j0;
        if (is_s) {
          if (!wait_all(q_full, uint32_t(si) & 1u)) break;
        } else if (si >= 1 && !wait_all(o_free, uint32_t(si - 1) & 1u)) {
          break;
        }
        for (int j = 0; j < n; ++j) {
          const int gj = base + j;
          const int st = gj % C::kStages;
          const uint32_t sb = tmem + ((gj & 1) ? C::kS1 : C::kS0);
          if (is_s) {
            // P of block j - 2 sits in the buffer that S overwrites.
            if (!wait_all(&k_full[st], uint32_t(gj / C::kStages) & 1u) ||
                (gj >= 2 && !wait_all(&o_done[gj & 1], uint32_t((gj - 2) >> 1) & 1u))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t kd = kd0 + uint64_t((uint32_t(st) * C::kTile) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < kD / 16; ++ks) {
                const uint64_t off = uint64_t((uint32_t(ks >> 2) * C::kHalf + uint32_t(ks & 3) * 32u) >> 4);
                mma_bf16_ss(sb, qd + off, kd + off, idesc_s, ks > 0 ? 1u : 0u);
              }
              tc_commit(&s_full[gj & 1]);
              tc_commit(&k_empty[st]);
            }
            __syncwarp();
          } else {
            if (!wait_all(&v_full[st], uint32_t(gj / C::kStages) & 1u)) {
              ok = false;
              break;
            }
            const uint64_t vd = vd0 + uint64_t((uint32_t(st) * C::kTile) >> 4);
            for (int h = 0; h < C::kParts; ++h) {
              if (!wait_all(&p_full[(gj & 1) * C::kParts + h], uint32_t(gj >> 1) & 1u)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < C::kPart / 16; ++ks) {
                  const uint64_t off = uint64_t((uint32_t(h * C::kPart) * 128u + uint32_t(ks) * 2048u) >> 4);
                  mma_bf16_ts(tmem + C::kO + uint32_t(h * kD), sb + uint32_t(C::kPart * h + 8 * ks), vd + off, idesc_o,
                              (j > 0 || ks > 0) ? 1u : 0u);
                }
                if (h == C::kParts - 1) {
                  tc_commit(&o_done[gj & 1]);
                  tc_commit(&v_empty[st]);
                }
              }
              __syncwarp();
            }
            if (!ok) break;
          }
        }
        if (!ok) break;
        if (!is_s && elect_one()) tc_commit(o_final);
        __syncwarp();
        base += n;
        ++si;
      }
      if (elect_one()) tc_commit(&drained[is_s ? 0 : 1]);
      __syncwarp();
      mbar_wait(&drained[is_s ? 0 : 1], 0, drain_limit_ns(lim));
    } else if (warp == 3) {
      // ----------------------------------------------------------- segments
      // Finds the run's segments for the softmax warps, up to two ahead, with the
      // ancestors of their trees (7000 cycles a segment when every softmax warp walked
      // the paths of its rows), and brings their Q rows to the L2 cache.
      Walk walk(run);
      for (int si = 0;; ++si) {
        const int sl = si & 1;
        if (si >= 2 && !__all_sync(0xFFFFFFFFu, wait(&seg_empty[sl], uint32_t((si >> 1) - 1) & 1u))) break;
        Seg s;
        const bool more = walk.next(p, run, s);
        if (lane == 0) {
          if (more) segs[sl].seg = s;
          segs[sl].more = more;
          mbar_arrive(&seg_full[sl]);
        }
        if (more) {
          for (int x = lane; x < 128; x += 32) {
            const int rr = s.tile * 128 + x;
            if (rr < s.n * p.G) {
              const int tok = rr / p.G;
              const uint16_t* row = p.Q + s.b * p.q_b + tok * p.q_t + (int64_t(s.h) * p.G + rr - tok * p.G) * p.q_h;
              asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
              if (kD == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 64));
            }
          }
          if (p.parents) {
            ancestors_of(p.parents + int64_t(s.b) * p.T, p.T, ancs + sl * 128, reinterpret_cast<int*>(ancs + 256), p.status);
            __syncwarp();
            if (lane == 0) mbar_arrive(&anc_full[sl]);
          }
        }
        if (si == 0) zero_idle_rows<kD>(p);
        if (!more) break;
      }
    }
  } else if (warp >= C::kRest) {
    fewer_registers<C::kRestRegs>();
    // ------------------------------------------------------------ restore
    // Four warps restore K, four V; thread i of each four has row i of the block.
    const bool is_k = warp < C::kRest + 4;
    const int i = tid & 127;
    uint64_t* fullb = is_k ? k_full : v_full;
    uint64_t* emptyb = is_k ? k_empty : v_empty;
    uint8_t* tiles = smem + (is_k ? C::kKOff : C::kVOff);
    const RowPlace<kD> place(i);
    Walk walk(run);
    Seg s;
    int rst = 0, gj = 0;
    uint32_t rph = 0u;
    bool ok = true;
    while (ok && walk.next(p, run, s)) {
      for (int j = s.j0; j < s.j1; ++j, ++gj) {
        const int st = gj & 1;
        if (!__all_sync(0xFFFFFFFFu, wait(&raw_full[rst], rph))) {
          ok = false;
          break;
        }
        const uint8_t* pg = smem + C::kRawOff + rst * C::kRaw + (i >> p.p_shift) * int(p.block);
        const int r = i & (p.P - 1);
        const uint32_t* par = reinterpret_cast<const uint32_t*>(pg + p.P * kD) + r;
        const uint8_t* src = pg + (is_k ? r : p.P + r) * (kD / 2);
        const uint32_t vp = par[p.P], mine = is_k ? par[0] : vp;
        uint4 w[kD / 32];
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) w[k] = *reinterpret_cast<const uint4*>(src + place.at[k]);
        const bool past = j * kKeys + i >= s.keys;
        const bool odd = not_finite(vp);
        // Exponents of this thread's row: its warp's, or its own where the warp's rows differ.
        // (A row that does not count has none: past the keys, not finite, zeros of K.)
        int e = row_exponent(mine, is_k ? kLeastK : kLeastV), f = is_k ? row_exponent(vp, kLeastV) : e;
        const int top = __reduce_max_sync(0xFFFFFFFFu, past ? kLeastK : e);
        const bool apart = __any_sync(0xFFFFFFFFu, !past && e < (is_k ? top - kSpread : max(top - kSpread, kSmallV)) &&
                                                       !not_finite(mine) && (!is_k || (mine & 0x7FFF7FFFu)));
        bool key_apart = apart;  // in K or in V (K warps)
        if (!apart) e = top;
        if (is_k) {
          const int top_v = __reduce_max_sync(0xFFFFFFFFu, past ? kLeastV : f);
          const bool apart_v = __any_sync(0xFFFFFFFFu, !past && f < max(top_v - kSpread, kSmallV) && !odd);
          if (!apart_v) f = top_v;
          key_apart |= apart_v;
        }
        f -= 8;
        const float down = pow2(8 - e) * 0x1p-8f;
        uint32_t s2 = 0u, z2 = 0u;
        if (!past && (is_k || !odd)) {
          s2 = pack_f16x2(bf16_lo(mine) * down, bf16_lo(mine) * down);
          z2 = is_k && odd ? 0x7E007E00u : pack_f16x2(bf16_hi(mine) * down, bf16_hi(mine) * down);
        }
        if (gj >= C::kStages && !__all_sync(0xFFFFFFFFu, wait(&emptyb[st], uint32_t((gj >> 1) - 1) & 1u))) {
          ok = false;
          break;
        }
        // The K warps publish both exponents: the softmax then waits for K alone.
        if (is_k && lane == 0)
          exps[(gj % C::kExpRing) * 4 + (i >> 5)] =
              make_float4(p.c * pow2(e - 8), float(f), pow2(-f), key_apart ? 1.f : 0.f);
        if (is_k && key_apart) key_exps[(gj % C::kExpRing) * 128 + i] = make_float2(p.c * pow2(e - 8), float(f));
        uint8_t* tile = tiles + st * C::kTile;
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) {
          uint8_t* dst = tile + place.dst[k];
          *reinterpret_cast<uint4*>(dst + place.word[0]) = restore_word(w[k].x, s2, z2);
          *reinterpret_cast<uint4*>(dst + place.word[1]) = restore_word(w[k].y, s2, z2);
          *reinterpret_cast<uint4*>(dst + place.word[2]) = restore_word(w[k].z, s2, z2);
          *reinterpret_cast<uint4*>(dst + place.word[3]) = restore_word(w[k].w, s2, z2);
        }
        fence_proxy_async_smem();  // the tile before the MMAs read it, the raw stage before it is refilled
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&fullb[st]);
          mbar_arrive(&raw_empty[rst]);
        }
        if (++rst == C::kRawStages) {
          rst = 0;
          rph ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    more_registers<C::kSoftRegs>();
    // ------------------------------------------------------------ softmax
    // Each four warps take a part of every block's keys; thread (warp w, lane) owns
    // row 32 (w % 4) + lane.
    const int q = warp & 3, h = (warp - 4) >> 2, r = q * 32 + lane;
    const uint32_t lane_off = uint32_t(q * 32) << 16;
    const uint32_t o_own = tmem + lane_off + C::kO + uint32_t(h * kD);
    constexpr int kSoftThreads = C::kSoft * 32;
    float2* xch = reinterpret_cast<float2*>(smem + C::kXchOff);
    int base = 0, si = 0;
    auto store_q = [&](int slot) {
      load_q<kD>(p, segs[slot].seg, warp - 4, smem + C::kQOff, qx + slot * 128);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };
    for (;;) {
      const int sl = si & 1;
      const Seg& s = segs[sl].seg;  // read where it is used: registers are short
      const bool got = wait(&seg_full[sl], uint32_t(si >> 1) & 1u);
      if (named_bar_any(1, kSoftThreads, !got)) break;
      if (!segs[sl].more) break;
      const int R = s.n * p.G;
      const int rr = s.tile * 128 + r;
      const bool valid = rr < R;
      const bool warp_live = __any_sync(0xFFFFFFFFu, valid);
      const int tok = valid ? rr / p.G : 0, hh = valid ? rr - tok * p.G : 0;
      if (si == 0) store_q(0);
      bool ok = __all_sync(0xFFFFFFFFu, wait(q_full, uint32_t(si) & 1u));
      const float up = pow2(qx[sl * 128 + r] + 8);  // the row's power of two, times 2^8
      uint32_t anc[4] = {0u, 0u, 0u, 0u};
      int limit = 0x7FFFFFFF;  // keys before it are seen (idle rows mask nothing: their results are not stored)
      if (p.parents) {
        ok &= __all_sync(0xFFFFFFFFu, wait(&anc_full[sl], uint32_t(si >> 1) & 1u));
        const uint4 x = ancs[sl * 128 + tok];
        anc[0] = x.x, anc[1] = x.y, anc[2] = x.z, anc[3] = x.w;
        if (valid) limit = s.prefix;
      } else if (valid) {
        limit = s.prefix + tok + 1;
      }
      float M = -INFINITY, l = 0.f;
      const int n = s.j1 - s.j0, key0 = s.j0 * kKeys + C::kPart * h;
      for (int i = 0; i < n && ok; ++i) {
        const int gi = base + i;
        const int kb = key0 + i * kKeys;
        if (!__all_sync(0xFFFFFFFFu, wait(&s_full[gi & 1], uint32_t(gi >> 1) & 1u))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (warp_live) {
          const uint32_t sc = tmem + lane_off + ((gi & 1) ? C::kS1 : C::kS0) + uint32_t(C::kPart * h);
          const bool edge = limit - kb < C::kPart;
          uint32_t pk[C::kPart / 2];
          float psum;
          const float4* own = exps + (gi % C::kExpRing) * 4 + C::kPart / 32 * h;
          // Rows that have seen nothing yet have no maximum to go by.
          bool look = __any_sync(0xFFFFFFFFu, M == -INFINITY);
          if (!look) {
            psum = 0.f;
#pragma unroll
            for (int ch = 0; ch < C::kPart / 32; ++ch) {
              uint32_t v[32];
              tmem_ld32(sc + uint32_t(ch * 32), v);
              const float4 ex = own[ch];
              tmem_ld_wait32(v);
              if (edge) mask_block<32>(v, kb + 32 * ch, limit, anc, true);
              const float sum = exp_pack_f16(v, fmaxf(ex.x * up, 1.2e-38f), ex.y - M, pk + 16 * ch);
              look |= sum > kMost || ex.w != 0.f;
              psum = fmaf(sum, ex.z, psum);
            }
            look = __any_sync(0xFFFFFFFFu, look);
          }
          if (look) {
            const float2* key = key_exps + (gi % C::kExpRing) * 128 + C::kPart * h;
            // The maximum moves to this block's where that is larger; O and the sum follow.
            float mx = -INFINITY;
#pragma unroll 1
            for (int ch = 0; ch < C::kPart / 32; ++ch) {
              uint32_t v[32];
              tmem_ld32(sc + uint32_t(ch * 32), v);
              tmem_ld_wait32(v);
              const float4 ex = own[ch];
              if (edge) mask_block<32>(v, kb + 32 * ch, limit, anc, true);
              float c = fmaxf(ex.x * up, 1.2e-38f), f = ex.y;
              if (ex.w != 0.f) {
                key_scores(v, key + 32 * ch, up, 0.f);
                c = 1.f, f = 0.f;
              }
              mx = fmaxf(mx, fmaf(block_max<32>(v), c, f));
            }
            mx -= kTop;
            const float down = mx > M ? M - mx : 0.f, factor = fast_exp2(down);  // 0 while M = -inf
            M = fmaxf(M, mx);
            l = scaled_down(l, down);
            if (i > 0) {
              if (!__all_sync(0xFFFFFFFFu, wait(&o_done[(gi - 1) & 1], uint32_t((gi - 1) >> 1) & 1u))) {
                ok = false;
                break;
              }
              tc_fence_after();
              rescale_row<kD>(o_own, factor);
            }
            const float ref = M == -INFINITY ? 0.f : M;
            psum = 0.f;
#pragma unroll
            for (int ch = 0; ch < C::kPart / 32; ++ch) {
              uint32_t v[32];
              tmem_ld32(sc + uint32_t(ch * 32), v);
              const float4 ex = own[ch];
              tmem_ld_wait32(v);
              if (edge) mask_block<32>(v, kb + 32 * ch, limit, anc, true);
              float c = fmaxf(ex.x * up, 1.2e-38f), f = ex.y, w = ex.z;
              if (ex.w != 0.f) {
                psum += key_scores(v, key + 32 * ch, up, ref);
                c = 1.f, f = w = 0.f;
              }
              psum = fmaf(exp_pack_f16(v, c, f - ref, pk + 16 * ch), w, psum);
            }
          }
          l += psum;
#pragma unroll
          for (int ch = 0; ch < C::kPart / 32; ++ch)
            tmem_st16(sc + uint32_t(16 * ch), *reinterpret_cast<uint32_t(*)[16]>(&pk[16 * ch]));
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&p_full[(gi & 1) * C::kParts + h]);
      }
      // The last S of the segment is done, so Q makes room for the next segment's: its S
      // goes on under this epilogue.
      if (ok && __all_sync(0xFFFFFFFFu, wait(&seg_full[sl ^ 1], uint32_t((si + 1) >> 1) & 1u)) && segs[sl ^ 1].more)
        store_q(sl ^ 1);
      // Epilogue: thread (h, r) joins the parts for its share of its row's dims.
      const bool fin = __all_sync(0xFFFFFFFFu, ok && wait(o_final, uint32_t(si) & 1u));
      if (named_bar_any(1, kSoftThreads, !fin)) break;
      tc_fence_after();
      xch[h * 128 + r] = make_float2(M, l);
      named_bar_sync(1, kSoftThreads);
      M = -INFINITY;
#pragma unroll
      for (int k = 0; k < C::kParts; ++k) M = fmaxf(M, xch[k * 128 + r].x);
      float den = 0.f, wt[C::kParts];
#pragma unroll
      for (int k = 0; k < C::kParts; ++k) {
        const float2 ml = xch[k * 128 + r];
        const float d = ml.x == M ? 0.f : ml.x - M;
        den += scaled_down(ml.y, d);
        wt[k] = 256.f * fast_exp2(d);  // V is held over 2^(f + 8)
      }
      constexpr int kDims = kD / C::kParts;
      const bool whole = s.whole();
      const float inv = !whole ? 1.f : den == 0.f ? 0.f : 1.f / den;
      uint32_t* out = reinterpret_cast<uint32_t*>(
          p.O + ((int64_t(s.b) * p.T + tok) * p.Hq + int64_t(s.h) * p.G + hh) * kD + h * kDims);
      float4* po = reinterpret_cast<float4*>(p.part_o) + (int64_t(blockIdx.x) * 2 + s.slot) * (kD / 4) * 128 + r;
      if (warp_live) {
#pragma unroll
        for (int ch = 0; ch < kDims / 16; ++ch) {
          float o[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0.f;
#pragma unroll
          for (int part = 0; part < C::kParts; ++part) {
            uint32_t a[16];
            tmem_ld16(tmem + lane_off + C::kO + uint32_t(part * kD + h * kDims + ch * 16), a);
            tmem_ld_wait(a);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(wt[part], __uint_as_float(a[k]), o[k]);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] *= inv;
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
              po[(h * (kDims / 4) + ch * 4 + k) * 128] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      if (!whole) {
        if (h == 0 && valid) p.part_ml[(int64_t(blockIdx.x) * 2 + s.slot) * 128 + r] = make_float2(M, den);
        // (The barrier orders the CTA's stores before the one release, and its acquire before all loads.)
        named_bar_sync(1, kSoftThreads);
        if (tid == 128) {
          const int add = s.j1 - s.j0;
          int32_t* cnt = p.cnt + run_of(run, s.x0);
          *merge_here = atomic_add_acq_rel_gpu(cnt, add) + add == s.nkb;
          if (*merge_here) *cnt = 0;
        }
        named_bar_sync(1, kSoftThreads);
        if (*merge_here && valid) {
          const int c0 = run_of(run, s.x0), c1 = run_of(run, s.x0 + s.nkb - 1);
          const int first = run_start(run, c0) >= s.x0 ? 0 : 1;
          // Three partials' loads are in flight at a time (an item has two or three as
          // a rule; one after the other they took 15000 cycles, 80 rows of 128 dims).
          auto slot_of = [&](int c) { return int64_t(c) * 2 + (c == c0 ? first : 0); };
          float Mx = -INFINITY, L = 0.f;
          for (int c = c0; c <= c1; c += 3) {
            float2 ml[3];
#pragma unroll
            for (int u = 0; u < 3; ++u)
              ml[u] = c + u <= c1 ? __ldcg(p.part_ml + slot_of(c + u) * 128 + r) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int u = 0; u < 3; ++u) {
              const float mn = fmaxf(Mx, ml[u].x);
              L = scaled_down(L, Mx == mn ? 0.f : Mx - mn) + scaled_down(ml[u].y, ml[u].x == mn ? 0.f : ml[u].x - mn);
              Mx = mn;
            }
          }
          const float scale = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
          for (int ch = 0; ch < kDims / 16; ++ch) {  // 16 dims at a time
            float o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
            for (int c = c0; c <= c1; c += 3) {
              float4 v[3][4];
              float mx[3];
#pragma unroll
              for (int u = 0; u < 3; ++u) {
                const int64_t slot = slot_of(c + u);
                const float4* src = reinterpret_cast<const float4*>(p.part_o) + (slot * (kD / 4) + h * (kDims / 4) + ch * 4) * 128 + r;
                mx[u] = c + u <= c1 ? __ldcg(p.part_ml + slot * 128 + r).x : -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[u][k] = c + u <= c1 ? __ldcg(src + k * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int u = 0; u < 3; ++u) {
                const float f = mx[u] == Mx ? 1.f : fast_exp2(mx[u] - Mx);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  o[4 * k] = fmaf(f, v[u][k].x, o[4 * k]);
                  o[4 * k + 1] = fmaf(f, v[u][k].y, o[4 * k + 1]);
                  o[4 * k + 2] = fmaf(f, v[u][k].z, o[4 * k + 2]);
                  o[4 * k + 3] = fmaf(f, v[u][k].w, o[4 * k + 3]);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint4 w;
              w.x = kv4::pack_bf16x2(o[8 * k] * scale, o[8 * k + 1] * scale);
              w.y = kv4::pack_bf16x2(o[8 * k + 2] * scale, o[8 * k + 3] * scale);
              w.z = kv4::pack_bf16x2(o[8 * k + 4] * scale, o[8 * k + 5] * scale);
              w.w = kv4::pack_bf16x2(o[8 * k + 6] * scale, o[8 * k + 7] * scale);
              reinterpret_cast<uint4*>(out)[ch * 2 + k] = w;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[sl]);
      base += n;
      ++si;
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
