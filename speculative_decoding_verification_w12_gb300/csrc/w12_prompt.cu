// Causal attention over whole prompts, packed one behind the other:
//   O[i, h] = sum_{j <= i} softmax_j(scale Q[i, h] . K[j, h / G]) V[j, h / G],
// i and j tokens of one sequence, G = Hq / Hkv query heads for each kv head.
//
// Rows of a tile are (token, head of the group), token-major, 128 / G tokens: a key block is
// read once for the whole group, and few of a tile's keys are cut by the diagonal. An item is
// two such tiles (few rows: one), one behind the other, of one (sequence, kv head), with all keys
// that they see in blocks. The kernel is persistent; the items of some sequences go out longest first
// (Walk), in rounds of the grid that alternate in direction, so every block gets about the same
// work and nothing is counted in memory. Per key block and tile:
//   S = Q K^T         tcgen05.mma, both from shared memory, S in TMEM;
//   P = 2^(c S - m)   a warpgroup for each tile, a row a thread: the running maximum moves only
//                     when a block's passes it by 2^8, so O is rescaled rarely;
//   O += P V          tcgen05.mma, P from TMEM, V from shared memory (MN-major).
// P has columns of its own, so the next block's S is under way as soon as the softmax has read
// this one's: products run about 430 cycles from issue to the waiting thread (measured, eight
// in a row), which a P over S would add twice a block to the softmax. At d = 128 the columns
// (512: S, P and O of both tiles) leave room for blocks of 80 keys, at d = 64 for 128.
//
// Long prompts are bound by the products: 8192 tokens of 40 / 8 heads of 128 take 381 us, 1800
// TFLOP/s. At d = 64 a block of both tiles has 1024 cycles of products, 1024 of exponentials (4 a
// warp's instruction) and about as many issue slots a scheduler, and takes 1950: 8192 tokens of 32 / 8
// heads 226 us (1210 TFLOP/s; all of these from L2). Short prompts are bound by the steps of an item (first scores,
// masks, last products, outputs), 7,000 to 9,000 cycles for 2 to 4 blocks: 64 of up to 300 57 us.
//
// P enters O rounded to the type of V (bf16: 2^-8 of itself; fp16: 2^-11, or 2^-25 of the
// largest weight), its sum is of the unrounded P; scores, maxima, sums and O are fp32.
//
// Masked places may hold anything. Masked scores are replaced, not added to. A value that is
// not finite would turn the zero weights of rows that do not see it into NaN: two warps look
// through the V blocks that the diagonal cuts, take such values out of shared memory and
// note their keys, and rows that see one add it at the end. (They pass on every V block, which P V waits
// for, so that no warp can fall a turn of the ring behind.)
//
// Warps: 0-3 and 4-7 softmax and epilogue of the two tiles; 8 and 9 issue S, 10 and 11 P V of the
// two tiles; 12 copies; 13 and 14 look through V; 15 finds the items. Each of the four
// series of products has a warp on a scheduler of its own: what a thread waits for comes back
// behind the products it has issued before (285 idle cycles a wait where one thread issues all,
// measured), so only other warps' products fill that time. The issuing warps run whole and elect
// a lane at the instruction: the operands are then known to be the same for the warp (an
// N = 64 product 32 cycles instead of 46).
#include <atomic>

#include "w12_attn_dev.cuh"
#include "w12_host.h"

namespace w12 {
namespace prompt_impl {

using namespace attn_impl;

constexpr int kThreads = 512;
constexpr float kRescale = 8.0f;   // log2 growth of the maximum that triggers a rescale
// Keys and values of a group of sequences whose items are under way together: a third of the L2
// cache, which Q and O pass through too. All sequences at once read them again for every place:
// 64 prompts of up to 1000 (40 / 8 heads of 128) took 324 us instead of 284, 8 of 8192 3350
// instead of 3150 (16 to 64 MB: alike).
constexpr int kGroupBytes = 43 << 20;
constexpr int kItems = 4;          // items handed out ahead
constexpr int kItemReaders = 15;   // warps that read an item
constexpr int kBadItems = 8;       // items whose cut blocks are noted (no warp is more than kItems ahead of another)
static_assert(kBadItems > kItems, "notes");
constexpr int kMostCut = 5;        // blocks that the diagonal cuts in an item: 256 tokens of blocks of 80 or more

// Registers: a warpgroup changes its share by one instruction that all its warps meet.
constexpr int kLaunchRegs = 128, kSoftRegs = 184, kRestRegs = 72;
static_assert(8 * kSoftRegs + 8 * kRestRegs <= (kThreads / 32) * kLaunchRegs, "the launch's registers");

// Whether this lane is the one that the warp, all of it here, has chosen.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kD>
struct Cfg {
  static constexpr int kKeys = kD == 128 ? 80 : 128;           // of a block
  static constexpr int kHalves = kD / 64;                      // 128-byte pieces of a row
  static constexpr uint32_t kQHalf = 128u * 128u;              // 128 rows of one piece of Q
  static constexpr uint32_t kQTile = kHalves * kQHalf;
  static constexpr uint32_t kHalf = 128u * kKeys;              // a key block's rows of one piece
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr int kStages = kD == 128 ? 8 : 10;           // K and V blocks in turn
  static constexpr uint32_t kRing = 2 * kQTile;                // behind the two tiles' Q
  static constexpr uint32_t kBar = kRing + kStages * kTile;
  static constexpr uint32_t kSmem = kBar + 1280 + 1024;        // barriers, items; alignment
  // TMEM columns of the first tile, and how far on the second's are.
  static constexpr uint32_t kColS = 0, kNextS = 128;
  static constexpr uint32_t kColP = kD == 128 ? kKeys : 256, kNextP = kD == 128 ? 128 : 64;
  static constexpr uint32_t kColO = kD == 128 ? 256 : 384, kNextO = kD;
  static_assert(kColP + kKeys / 2 <= (kD == 128 ? kNextS : kColP + kNextP) && kColO + 2 * kNextO <= 512, "columns");
};

struct Item {
  int first;   // token of the buffer that the first tile begins with
  int t0;      // its place in the sequence
  int len;     // tokens of the sequence
  int head;    // kv head; kSecond in it: the one tile is the second of a pair; -1: no more items
  static constexpr int kSecond = 1 << 16;
  __device__ __forceinline__ int kv() const { return head & (kSecond - 1); }
};

struct Params {
  const void* V;               // for values that are not finite
  int64_t v_tok, v_head;       // strides in elements
  void* O;                     // [total, Hq, kD]
  const int32_t* cu;           // [B + 1]
  int32_t* status;
  int64_t total;
  int B, Hq, Hkv, G, tpt;      // tpt: tokens a tile
  int room;                    // tokens of a group of sequences
  int step;                    // tokens of an item: two tiles or one
  uint32_t inv_g;              // a row's token is row inv_g / 2^16
  float c;                     // scale log2(e)
  uint64_t limit_ns;
  uint32_t sleep_ns;           // longest sleep of a wait between looks at its bound
};

// A box of (dims from x on, head y, token z on) rows; the maps' fourth extent is 1.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(0), "r"(smem_u32(bar))
      : "memory");
}

// Key blocks of a tile that begins at token t0 (none past the sequence's end), and the first
// of them that some row of the item or, of an item of one tile, of its pair of tiles does not see whole: what
// is taken out of V then hangs on the sequence alone.
template <int kKeys>
__device__ __forceinline__ int blocks_of(int t0, int tpt, int len) {
  return t0 >= len ? 0 : (min(t0 + tpt, len) + kKeys - 1) / kKeys;
}
template <int kKeys>
__device__ __forceinline__ int first_cut(const Item& it, int tpt) {
  return (it.t0 + 1 - ((it.head & Item::kSecond) ? tpt : 0)) / kKeys;
}

// Walks the items in their order: groups of sequences, whose keys and values stay in the L2 cache
// while their items are under way; in a group by place in the sequence (in items), then
// sequence, then kv head. Groups run alternately up and down the places, the last one down, so that
// neighbours in the order are alike in size and the smallest come last. Warp-collective.
struct Walk {
  const int32_t* cu;
  int B, Hkv, step, room;   // room: tokens of a group
  int64_t total;
  int chunk;        // of 32 sequences; past the last one: no more items
  uint32_t firsts;  // sequences of the chunk that a group begins with, those to come
  bool member;      // this lane's sequence is of the current group
  bool down;
  int level, top;   // items before the current ones in their sequences, and the most of the group
  uint32_t left;    // sequences of the group that are still to come at this level
  int head;         // next kv head of the first of them
  int n, start, len, group;  // of this lane's sequence of the chunk: items, first token, tokens, group

  __device__ __forceinline__ int chunks() const { return (B + 31) / 32; }
  __device__ __forceinline__ void load(int32_t* status) {
    const int lane = threadIdx.x & 31, b = chunk * 32 + lane;
    start = len = 0;
    if (b < B) {
      const int a = cu[b], e = cu[b + 1];
      if (a < 0 || e < a || e > total) {
        if (status) set_status(status, W12_ERR_ARG);
      } else {
        start = a;
        len = e - a;
      }
    }
    n = (len + step - 1) / step;
    // A group for every `room` tokens, by where a sequence begins among the chunk's.
    const int mine = min(len, room);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, n > 0);
    group = n > 0 ? 0 : -1;
    firsts = some & (0u - some);
    if (int(__reduce_add_sync(0xFFFFFFFFu, unsigned(mine))) > room) {
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += v;
      }
      if (n > 0) group = (before - mine) / room;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, group);
      firsts = __ballot_sync(0xFFFFFFFFu, n > 0 && !(same & ((1u << lane) - 1u)));
    }
  }
  __device__ __forceinline__ void begin(int32_t* status) {
    int groups = 0;
    for (chunk = chunks() - 1; chunk >= 0; --chunk) {
      load(status);
      groups += __popc(firsts);
    }
    chunk = 0;
    if (chunks() > 1) load(nullptr);
    down = !(groups & 1);
    member = false;
    level = top = -1;
    left = 0;
    head = 0;
  }
  // To the next level that has items; false: there is none.
  __device__ __forceinline__ bool advance() {
    head = 0;
    level += down ? -1 : 1;
    if (level < 0 || level > top) {
      while (!firsts) {
        if (++chunk >= chunks()) return false;
        load(nullptr);
      }
      const int first = __ffs(firsts) - 1;
      firsts &= firsts - 1;
      down = !down;
      member = group == __shfl_sync(0xFFFFFFFFu, group, first);
      top = int(__reduce_max_sync(0xFFFFFFFFu, member ? unsigned(n) : 0u)) - 1;
      level = down ? top : 0;
    }
    left = __ballot_sync(0xFFFFFFFFu, member && n > level);
    return true;
  }
  // The item `skip` places on.
  __device__ __forceinline__ Item next(int skip) {
    Item it{0, 0, 0, -1};
    while (chunk < chunks()) {
      const int here = __popc(left) * Hkv - head;
      if (skip < here) {
        const int at = head + skip;
        for (int k = at / Hkv; k > 0; --k) left &= left - 1;
        head = at % Hkv;
        const int src = __ffs(left) - 1;
        it.t0 = level * step;
        it.first = __shfl_sync(0xFFFFFFFFu, start, src) + it.t0;
        it.len = min(__shfl_sync(0xFFFFFFFFu, len, src), it.t0 + step);
        it.head = head;
        return it;
      }
      skip -= here;
      if (!advance()) break;
    }
    return it;
  }
};

#define W12_R8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
#define W12_W8(v, o) \
  "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])

// Each thread reads (valid after the wait for loads) columns of its own lane and their largest
// value (NaN aside), or writes some.
__device__ __forceinline__ void tmem_ld_max32(uint32_t taddr, uint32_t* v, float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : W12_W8(v, 0), W12_W8(v, 8), W12_W8(v, 16), W12_W8(v, 24), "=f"(top)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : W12_W8(v, 0), W12_W8(v, 8), W12_W8(v, 16), W12_W8(v, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_max16(uint32_t taddr, uint32_t* v, float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, %16, "
      "[%17];"
      : W12_W8(v, 0), W12_W8(v, 8), "=f"(top)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::W12_R8(v, 0),
      W12_R8(v, 8), W12_R8(v, 16), W12_R8(v, 24), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::W12_R8(v, 0), "r"(taddr) : "memory");
}

// 16 rows of 32 columns: a lane gets column 4 k + lane % 4 of row lane / 4 as v[k], of row lane / 4 + 8
// as v[8 + k].
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %8, %1, %9, %2, %10, %3, %11, %4, %12, %5, %13, %6, %14, %7, %15}, [%16];"
      : W12_W8(v, 0), W12_W8(v, 8)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(v[k]));  // (no use of a value moves before the wait)
}

// 32 bytes of memory of this thread's: a whole sector.
__device__ __forceinline__ void st_global32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), W12_R8(w, 0) : "memory");
}

// The largest of N scores, three at a time (the two-operand maximum runs at the same rate).
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
template <int N>
__device__ __forceinline__ float largest(const uint32_t (&v)[N]) {
  float m[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) m[a] = __uint_as_float(v[a]);
#pragma unroll
  for (int k = 4; k + 1 < N; k += 2) m[(k >> 1) & 3] = max3(m[(k >> 1) & 3], v[k], v[k + 1]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBf16) return pack_bf16x2(lo, hi);
  else return pack_f16x2(lo, hi);
}

// P_k = 2^(c s_k + negm) of N scores, packed as pairs into v[0 .. N/2 - 1] in place (pair k
// over v[k], which pair k/2 has read); returns the fp32 sum.
template <bool kBf16, int N>
__device__ __forceinline__ float weights(uint32_t (&v)[N], float c, float negm) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 c2 = make_float2(c, c), m2 = make_float2(negm, negm);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    const float2 x = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2, m2);
    const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    sum[k & 1] = add2(sum[k & 1], p);
    v[k] = pack2<kBf16>(p.x, p.y);
  }
  const float2 s = add2(sum[0], sum[1]);
  return s.x + s.y;
}

// A row's scores from TMEM, ready to use, and the largest of them (found by the load).
template <int N>
__device__ __forceinline__ float load_scores(uint32_t taddr, uint32_t (&v)[N]) {
  constexpr int kParts = (N + 31) / 32;
  float top[kParts];
#pragma unroll
  for (int ch = 0; ch < N / 32; ++ch) tmem_ld_max32(taddr + uint32_t(32 * ch), &v[32 * ch], top[ch]);
  if constexpr (N % 32) tmem_ld_max16(taddr + uint32_t(N - 16), &v[N - 16], top[kParts - 1]);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(v[k]));  // (no use of a value moves before the wait)
  float m = -INFINITY;
#pragma unroll
  for (int ch = 0; ch < kParts; ++ch) {
    asm volatile("" : "+f"(top[ch]));
    m = fmaxf(m, top[ch]);
  }
  return m;
}

// N columns of weights to TMEM, done when it returns.
template <int N>
__device__ __forceinline__ void store_weights(uint32_t taddr, uint32_t* v) {
#pragma unroll
  for (int ch = 0; ch < N / 32; ++ch) tmem_st32(taddr + uint32_t(32 * ch), v + 32 * ch);
  if constexpr (N % 32 != 0) {
    static_assert(N % 32 == 8, "one more piece");
    tmem_st8(taddr + uint32_t(N - 8), v + N - 8);
  }
  tmem_st_wait();
}

// A value of V's type is finite: all exponent bits set otherwise.
template <bool kBf16>
__device__ __forceinline__ bool finite16(uint32_t h) {
  constexpr uint32_t kExp = kBf16 ? 0x7F80u : 0x7C00u;
  return (h & kExp) != kExp;
}

// x with its elements that are not finite replaced by zeros.
template <bool kBf16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
  return (finite16<kBf16>(x) ? x & 0xFFFFu : 0u) | (finite16<kBf16>(x >> 16) ? x & 0xFFFF0000u : 0u);
}

// acc + 0 x, as pairs: NaN in either half once an element of x is not finite.
template <bool kBf16>
__device__ __forceinline__ uint32_t spot(uint32_t x, uint32_t acc) {
  uint32_t r;
  if constexpr (kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}

// Adds to a row's outputs the values that were taken out of V, of the keys that the row sees, as
// they are: infinities and NaN.
template <int kKeys, int kD, bool kBf16>
__device__ __noinline__ void add_taken_out(const Params& P, uint16_t* out, uint32_t odd, int cut, int t, int seq, int head) {
  for (int b = 0; b < kMostCut; ++b) {
    if (!((odd >> b) & 1u)) continue;
    const int key0 = (cut + b) * kKeys;
    for (int key = key0; key < key0 + kKeys && key <= t; ++key) {
      const uint16_t* src = static_cast<const uint16_t*>(P.V) + int64_t(seq + key) * P.v_tok + int64_t(head) * P.v_head;
#pragma unroll 1
      for (int x = 0; x < kD; ++x) {
        const uint32_t u = src[x];
        if (finite16<kBf16>(u)) continue;
        const uint32_t before = out[x];
        const float f = kBf16 ? __uint_as_float(before << 16) + __uint_as_float(u << 16) : unpack_f16x2(before).x + unpack_f16x2(u).x;
        out[x] = uint16_t(pack2<kBf16>(f, f));
      }
    }
  }
}

template <int kD, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params P) {
  using C = Cfg<kD>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (An offset, not a rounded pointer: the compiler then still knows that it is shared memory.)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // [kBadItems][kMostCut]: keys of an item's cut blocks with values taken out of V
  uint4* bad = reinterpret_cast<uint4*>(smem + C::kBar);
  uint64_t* full = reinterpret_cast<uint64_t*>(bad + kBadItems * kMostCut);  // [kStages]: block landed
  uint64_t* empty = full + kStages;       // [kStages]: products of the stage's block done
  uint64_t* clean = empty + kStages;      // [kStages]: V block passed on, looked through where the diagonal cuts it
  uint64_t* q_full = clean + kStages;     // [2]: tile's Q landed
  uint64_t* q_empty = q_full + 2;         // [2]: the item's last S of the tile done
  uint64_t* s_full = q_empty + 2;         // [2]: S of the tile's block
  uint64_t* s_read = s_full + 2;          // [2]: and read
  uint64_t* p_full = s_read + 2;          // [2]: P of the tile's block
  uint64_t* o_done = p_full + 2;          // [2]: P V of the tile's block done
  uint64_t* o_free = o_done + 2;          // [2]: the item's O read
  uint64_t* drained = o_free + 2;         // [4]: all products of an issuing warp done
  uint64_t* it_full = drained + 4;        // [kItems]
  uint64_t* it_empty = it_full + kItems;  // [kItems]
  Item* items = reinterpret_cast<Item*>(it_empty + kItems);       // [kItems]
  uint32_t* misc = reinterpret_cast<uint32_t*>(items + kItems);
  volatile uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* copied = reinterpret_cast<volatile int*>(misc + 2);  // blocks requested
  volatile int* q_copied = reinterpret_cast<volatile int*>(misc + 3);  // [2]: Q tiles requested
  static_assert(16 * kBadItems * kMostCut + (3 * kStages + 18 + 2 * kItems) * 8 + 16 * kItems + 20 <= 1280, "barriers");

  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);   // one arrival a tile
      mbar_init(&clean[s], 2);   // two warps, half of the keys each
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_read[i], 4);       // one arrival a warp
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_free[i], 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&drained[i], 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], kItemReaders);
    }
    *abort_flag = 0;
    copied[0] = q_copied[0] = q_copied[1] = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 8) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const uint64_t lim = P.limit_ns;
  // Everything below reads what the previous kernel on the stream wrote.
  grid_dep_wait();

  // (Asleep for no longer than its bound at a time, as in mbar_wait_asleep: 64 x 300 57.3 us, with that one 57.9.)
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait_hint(bar, parity, P.sleep_ns)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 0; i < 0x80000000u; ++i) {
      if (mbar_try_wait_hint(bar, parity, P.sleep_ns)) return true;
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > lim) break;
    }
    set_status(P.status, W12_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
  };
  // One decision for the warp: what follows is warp-collective.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait(bar, parity)); };
  // The k-th item of this block, for a whole warp.
  auto get_item = [&](int k, Item& it) -> bool {
    if (!wait_all(&it_full[k % kItems], uint32_t(k / kItems) & 1u)) return false;
    it = items[k % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_empty[k % kItems]);
    return it.head >= 0;
  };

  if (warp >= 8) {
    fewer_registers<kRestRegs>();
  if (warp == 12) {
    // --------------------------------------------------------- items, copies
    int issued = 0, q_issued[2] = {0, 0};
    bool ok = true;
    Item it;
    auto stage = [&](const CUtensorMap* map, int head, int token) -> bool {
      const int s = issued % kStages;
      if (issued >= kStages && !wait(&empty[s], uint32_t(issued / kStages - 1) & 1u)) return false;
      uint8_t* at = smem + C::kRing + uint32_t(s) * C::kTile;
      mbar_arrive_expect_tx(&full[s], C::kTile);
      for (int h = 0; h < C::kHalves; ++h) load_box(at + h * C::kHalf, map, 64 * h, head, token, &full[s]);
      ++issued;
      return true;
    };
    for (int k = 0; ok && get_item(k, it); ++k) {
      if (lane == 0) {
        const int seq = it.first - it.t0;
        const int n0 = blocks_of<C::kKeys>(it.t0, P.tpt, it.len), n1 = blocks_of<C::kKeys>(it.t0 + P.tpt, P.tpt, it.len);
        const int n = max(n0, n1);
        for (int j = 0; ok && j < n; ++j) {
          ok = stage(&tm_k, it.kv(), seq + j * C::kKeys);
          if (j == 0) {
            for (int i = 0; ok && i < (n1 ? 2 : 1); ++i) {
              if (q_issued[i] > 0) ok = wait(&q_empty[i], uint32_t(q_issued[i] - 1) & 1u);
              if (!ok) break;
              mbar_arrive_expect_tx(&q_full[i], uint32_t(kD * 2 * P.G * P.tpt));
              for (int h = 0; h < C::kHalves; ++h)
                load_box(smem + uint32_t(i) * C::kQTile + h * C::kQHalf, &tm_q, 64 * h, it.kv() * P.G, it.first + i * P.tpt,
                         &q_full[i]);
              ++q_issued[i];
            }
          }
          if (ok) ok = stage(&tm_v, it.kv(), seq + j * C::kKeys);
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, int(ok), 0);
    }
    grid_dep_launch();
    if (lane == 0) {
      copied[0] = issued;
      q_copied[0] = q_issued[0];
      q_copied[1] = q_issued[1];
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------- products
    // Block j of the item is K in ring place 2j and V in 2j + 1 from the item's first.
    const int i = warp & 1;
    const bool is_s = warp < 10;
    const uint32_t sbase = smem_u32(smem);
    const uint64_t qd = sdesc_k_sw128(sbase + uint32_t(i) * C::kQTile);
    const uint64_t kd0 = sdesc_k_sw128(sbase + C::kRing);
    const uint64_t vd0 = sdesc_mn_sw128(sbase + C::kRing, C::kHalf);
    constexpr uint32_t kTypes = kBf16 ? 0u : (1u << 7) | (1u << 10);  // fp16 operands: the formats' bits clear
    const uint32_t idesc_s = idesc_bf16(128, C::kKeys) & ~kTypes;
    const uint32_t idesc_o = (idesc_bf16(128, kD) & ~kTypes) | (1u << 16);  // V is MN-major
    const uint32_t s_at = tmem + C::kColS + C::kNextS * i, p_at = tmem + C::kColP + C::kNextP * i, o_at = tmem + C::kColO + C::kNextO * i;
    int place = is_s ? 0 : 1;   // in the ring, of the next block
    int blocks = 0;             // blocks of this tile so far
    int mine = 0;               // items of this tile before this one
    bool ok = true;
    Item it;
    for (int k = 0; ok && get_item(k, it); ++k) {
      const int n0 = blocks_of<C::kKeys>(it.t0, P.tpt, it.len), n1 = blocks_of<C::kKeys>(it.t0 + P.tpt, P.tpt, it.len);
      const int all = max(n0, n1), n = i ? n1 : n0;
      if (n > 0 && is_s) ok = wait_all(&q_full[i], uint32_t(mine) & 1u);
      if (n > 0 && !is_s && mine > 0) ok = wait_all(&o_free[i], uint32_t(mine - 1) & 1u);
      for (int j = 0; ok && j < all; ++j, place += 2) {
        const int s = place % kStages;
        // V is waited for as looked through in every block, cut or not: a wait names a parity alone, and
        // were some turns of `clean` not waited for, the ring could pass the two warps that look.
        const uint32_t turn = uint32_t(place / kStages) & 1u;
        ok = wait_all(&full[s], turn) && (is_s || wait_all(&clean[s], turn));
        if (!ok) break;
        if (j >= n) {  // a block that only the other tile has
          if (lane == 0) mbar_arrive(&empty[s]);
          continue;
        }
        if (is_s) {
          // The softmax has read the block before.
          if (blocks > 0 && !(ok = wait_all(&s_read[i], uint32_t(blocks - 1) & 1u))) break;
          tc_fence_after();
          const uint64_t kd = kd0 + uint64_t((uint32_t(s) * C::kTile) >> 4);
          if (elected()) {
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
              const uint32_t in = uint32_t(ks & 3) * 32u;
              mma_bf16_ss(s_at, qd + uint64_t((uint32_t(ks >> 2) * C::kQHalf + in) >> 4),
                          kd + uint64_t((uint32_t(ks >> 2) * C::kHalf + in) >> 4), idesc_s, ks > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[i]);
            tc_commit(&empty[s]);
            if (j == n - 1) tc_commit(&q_empty[i]);
          }
        } else {
          if (!(ok = wait_all(&p_full[i], uint32_t(blocks) & 1u))) break;
          tc_fence_after();
          const uint64_t vd = vd0 + uint64_t((uint32_t(s) * C::kTile) >> 4);
          if (elected()) {
#pragma unroll
            for (int ks = 0; ks < C::kKeys / 16; ++ks)
              mma_bf16_ts(o_at, p_at + uint32_t(8 * ks), vd + uint64_t((uint32_t(ks) * 2048u) >> 4), idesc_o, (j > 0 || ks > 0) ? 1u : 0u);
            tc_commit(&o_done[i]);
            tc_commit(&empty[s]);
          }
        }
        __syncwarp();
        ++blocks;
      }
      mine += n > 0;
    }
    // The products are done before the block leaves: after a failed wait they may not be.
    if (elected()) {
      tc_commit(&drained[warp - 8]);
      mbar_wait(&drained[warp - 8], 0, drain_limit_ns(lim));
    }
    __syncwarp();
  } else if (warp == 15) {
    // ---------------------------------------------------------------- items
    Walk walk{P.cu, P.B, P.Hkv, P.step, P.room, P.total};
    walk.begin(blockIdx.x == 0 ? P.status : nullptr);
    const int grid = int(gridDim.x), me = int(blockIdx.x);
    int skip = me;
    for (int k = 0;; ++k) {
      Item it = walk.next(skip);
      if (P.step == P.tpt && it.head >= 0 && (walk.level & 1)) it.head |= Item::kSecond;
      // Rounds alternate in direction: place `me` of even rounds, `grid - 1 - me` of odd ones.
      // (walk.next leaves the walk on the item: the next one is one place more on.)
      skip = ((k & 1) ? 2 * me : 2 * (grid - 1 - me)) + 1;
      if (k >= kItems && !wait_all(&it_empty[k % kItems], uint32_t(k / kItems - 1) & 1u)) break;
      if (lane == 0) {
        items[k % kItems] = it;
        mbar_arrive(&it_full[k % kItems]);
      }
      if (it.head < 0) break;
    }
  } else if (warp == 13 || warp == 14) {
    // ------------------------------------------------- values that are not finite
    int place = 1;   // in the ring, of the next V block
    bool ok = true;
    Item it;
    for (int k = 0; ok && get_item(k, it); ++k) {
      const int all = max(blocks_of<C::kKeys>(it.t0, P.tpt, it.len), blocks_of<C::kKeys>(it.t0 + P.tpt, P.tpt, it.len));
      const int cut = first_cut<C::kKeys>(it, P.tpt);
      uint4* notes = bad + (k % kBadItems) * kMostCut;
      // (V blocks that the diagonal does not cut are waited for and passed on too: the ring cannot pass these warps.)
      for (int j = 0; ok && j < all; ++j, place += 2) {
        const int s = place % kStages;
        if (!(ok = wait_all(&full[s], uint32_t(place / kStages) & 1u))) break;
        if (j < cut) {
          if (lane == 0) mbar_arrive(&clean[s]);
          continue;
        }
        uint8_t* v = smem + C::kRing + uint32_t(s) * C::kTile;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int word = 2 * w + warp - 13, row = 32 * word + lane;   // 32 keys at a time
          const bool there = row < C::kKeys;
          uint32_t acc = 0u;
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
            for (int c = 0; there && c < 8; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(v + h * C::kHalf + row * 128 + ((c ^ (row & 7)) << 4));
              acc = spot<kBf16>(x.w, spot<kBf16>(x.z, spot<kBf16>(x.y, spot<kBf16>(x.x, acc))));
            }
          const bool odd = !(finite16<kBf16>(acc) && finite16<kBf16>(acc >> 16));
          if (odd) {
            for (int c = 0; c < 8 * C::kHalves; ++c) {
              uint4* at = reinterpret_cast<uint4*>(v + (c >> 3) * C::kHalf + row * 128 + ((c & 7) << 4));
              const uint4 x = *at;
              *at = make_uint4(finite_pair<kBf16>(x.x), finite_pair<kBf16>(x.y), finite_pair<kBf16>(x.z), finite_pair<kBf16>(x.w));
            }
          }
          const uint32_t keys = __ballot_sync(0xFFFFFFFFu, odd);
          if (lane == 0) reinterpret_cast<uint32_t*>(&notes[j - cut])[word] = keys;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[s]);
      }
    }
  }
  } else {
    more_registers<kSoftRegs>();
    // -------------------------------------------------------------- softmax
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;          // row of the tile = TMEM lane
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_off + C::kColS + C::kNextS * i, p_at = tmem + lane_off + C::kColP + C::kNextP * i;
    const uint32_t o_at = tmem + lane_off + C::kColO + C::kNextO * i;
    const float c = P.c;
    const int row_t = r / P.G, row_h = r - row_t * P.G;  // the row's token of the tile and head of the group
    int blocks = 0;
    Item it;
    for (int k = 0; get_item(k, it); ++k) {
      const int t0 = it.t0 + i * P.tpt;
      const int n0 = blocks_of<C::kKeys>(it.t0, P.tpt, it.len), n1 = blocks_of<C::kKeys>(it.t0 + P.tpt, P.tpt, it.len);
      const int n = i ? n1 : n0;
      const int t = t0 + row_t;                     // the row's token, in its sequence
      const bool valid = row_t < P.tpt && t < it.len;
      const int cut = first_cut<C::kKeys>(it, P.tpt);   // (from here on values may have been taken out)
      const int masked = (it.t0 + 1) / C::kKeys;    // (and from here on the item's first rows do not see all keys)
      float m = -INFINITY, l = 0.f;
      // A wait is one vote of the warp a block (what follows is warp-collective): barriers are
      // looked at early, and waited for only where that has not shown them complete.
      bool ok = true, come = false;                 // come: the block's scores are there
      for (int j = 0; j < n; ++j) {
        if (!come) ok = wait(&s_full[i], uint32_t(blocks + j) & 1u);
        __syncwarp();
        tc_fence_after();
        const bool used = j == 0 || mbar_try_wait(&o_done[i], uint32_t(blocks + j - 1) & 1u);  // P of the block before
        uint32_t v[C::kKeys];
        float top = load_scores<C::kKeys>(s_at, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_read[i]);
        if (j >= masked) {
          const int see = t - j * C::kKeys + 1;     // keys of the block that the row sees
#pragma unroll
          for (int x = 0; x < C::kKeys; ++x)
            if (x >= see) v[x] = __float_as_uint(-INFINITY);
          top = largest(v);
        }
        const float mx = top * c;
        float factor = 1.f;
        if (mx > m + kRescale) {
          factor = fast_exp2(m - mx);               // 0 while m = -inf
          m = mx;
        }
        const bool resc = j > 0 && factor < 1.f && l > 0.f;
        if (__any_sync(0xFFFFFFFFu, resc || !used || !ok)) {
          if (!used && ok) ok = wait(&o_done[i], uint32_t(blocks + j - 1) & 1u);
          if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
          if (__any_sync(0xFFFFFFFFu, resc)) {
            tc_fence_after();
            rescale_row<kD>(o_at, resc ? factor : 1.f);
            tmem_st_wait();
          }
        }
        const float negm = m == -INFINITY ? 0.f : -m;
        l = l * factor + weights<kBf16>(v, c, negm);
        come = j + 1 < n && mbar_try_wait(&s_full[i], uint32_t(blocks + j + 1) & 1u);
        tc_fence_after();
        store_weights<C::kKeys / 2>(p_at, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      if (!ok) break;
      if (n > 0) {
        if (!wait_all(&o_done[i], uint32_t(blocks + n - 1) & 1u)) break;
        tc_fence_after();
        // Bit b: the row sees a value of block cut + b that is not finite. (The products waited for the notes.)
        uint32_t odd = 0;
        const uint4* notes = bad + (k % kBadItems) * kMostCut;
#pragma unroll
        for (int b = 0; b < kMostCut; ++b) {
          const uint4 keys = b < n - cut ? notes[b] : make_uint4(0, 0, 0, 0);
          if (keys.x | keys.y | keys.z | keys.w) {
            const uint32_t word[4] = {keys.x, keys.y, keys.z, keys.w};
            const int see = t - (cut + b) * C::kKeys + 1;
#pragma unroll
            for (int w = 0; w < (C::kKeys + 31) / 32; ++w) {
              const int lim_w = see - 32 * w;
              const uint32_t seen = lim_w >= 32 ? ~0u : lim_w <= 0 ? 0u : (1u << lim_w) - 1u;
              if (word[w] & seen) odd |= 1u << b;
            }
          }
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
        // Of its own row a lane would store 32 bytes at a time, a line each; the lines are what the
        // stores take. So half rows change lanes on the way, through P's columns: four lanes have a
        // line of a row then, an instruction eight lines (2,400 -> 1,700 cycles an item of short prompts).
        uint16_t* tile = static_cast<uint16_t*>(P.O) + (int64_t(it.first - it.t0 + t0) * P.Hq + it.kv() * P.G) * kD;
        const int end = min(P.tpt, it.len - t0);      // tokens
#pragma unroll
        for (int ch = 0; ch < kD / 64; ++ch) {
          uint32_t o[64], w[32];
          tmem_ld32(o_at + uint32_t(64 * ch), &o[0]);
          tmem_ld32(o_at + uint32_t(64 * ch + 32), &o[32]);
          tmem_ld_wait64(o);
          if (ch == kD / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[i]);
          }
          // Column 4 k + q has word 8 q + k: lane q of four gets eight neighbours.
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int y = 8 * (x & 3) + (x >> 2);
            w[x] = pack2<kBf16>(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
          }
          tmem_st32(p_at, w);
          tmem_st_wait();
          tmem_ld_quads(p_at, &w[0]);
          tmem_ld_quads(p_at + (16u << 16), &w[16]);
          tmem_ld_wait32(w);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t row = (warp & 3) * 32 + 8 * x + (lane >> 2), tok = (row * P.inv_g) >> 16;
            if (int(tok) < end)
              st_global32(tile + int64_t(tok * P.Hq + row - tok * P.G) * kD + 64 * ch + 16 * (lane & 3), &w[8 * x]);
          }
        }
        if (__any_sync(0xFFFFFFFFu, odd && valid)) {
          __syncwarp();
          uint16_t* out = tile + int64_t(row_t * P.Hq + row_h) * kD;
          if (odd && valid) add_taken_out<C::kKeys, kD, kBf16>(P, out, odd, cut, t, it.first - it.t0, it.kv());
        }
      }
      blocks += n;
    }
  }

  tc_fence_before();
  cta_sync();
  // Only now is no wait left that could expire: after one, copies may be in flight still.
  if (*abort_flag && warp == 12 && lane == 0) {
    for (int k = copied[0] > kStages ? copied[0] - kStages : 0; k < copied[0]; ++k)
      mbar_wait(&full[k % kStages], uint32_t(k / kStages) & 1u, drain_limit_ns(lim));
    for (int i = 0; i < 2; ++i)
      if (q_copied[i] > 0) mbar_wait(&q_full[i], uint32_t(q_copied[i] - 1) & 1u, drain_limit_ns(lim));
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kD, bool kBf16>
static cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Params& P, unsigned grid,
                          cudaStream_t stream) {
  auto kernel = prompt_kernel<kD, kBf16>;
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!((ready.load() >> dev) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Cfg<kD>::kSmem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(uint64_t(1) << dev);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<kD>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, q, k, v, P);
}

// Rows [total, H, d] with element strides as boxes of `tokens` tokens of `heads` heads, 64 dims each.
static bool row_map(CUtensorMap* map, const void* x, bool bf16, int d, int H, int64_t total, int64_t tok, int64_t head, int heads,
                    int tokens) {
  const uint64_t dims[4] = {uint64_t(d), uint64_t(H), uint64_t(total), 1};
  const uint64_t strides[3] = {uint64_t(head) * 2, uint64_t(tok) * 2, 16};
  const uint32_t box[4] = {64, uint32_t(heads), uint32_t(tokens), 1};
  return encode_tmap_4d(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, const_cast<void*>(x), dims,
                        strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Strides that a tensor map takes: positive multiples of 16 bytes below 2^40.
static bool stride_ok(int64_t elements) { return elements > 0 && elements % 8 == 0 && elements < (int64_t(1) << 38); }

}  // namespace prompt_impl
}  // namespace w12

using namespace w12;
using namespace w12::prompt_impl;

extern "C" {

int w12_prompt_attention(const void* Q, int64_t q_token_stride, int64_t q_head_stride, const void* K, int64_t k_token_stride,
                         int64_t k_head_stride, const void* V, int64_t v_token_stride, int64_t v_head_stride, int dtype,
                         int64_t total, const int32_t* cu_seqlens, int B, int Hq, int Hkv, int head_dim, float scale, void* O,
                         int32_t* dev_status, void* stream) {
  if (dtype != W12_BF16 && dtype != W12_F16) return W12_ERR_ARG;
  if (!cu_seqlens || !(scale > 0.f) || scale > 1e30f) return W12_ERR_ARG;
  if (B < 0 || B > 65535 || total < 0 || total > 0x7FFFFFFF - 256 || Hkv < 1 || Hkv > 1024 || Hq < Hkv || Hq % Hkv ||
      Hq / Hkv > 128 || (head_dim != 64 && head_dim != 128))
    return W12_ERR_SHAPE;
  if (total == 0 || B == 0) return device_supported() ? W12_OK : W12_ERR_UNSUPPORTED;
  if (!Q || !K || !V || !O || !aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 32)) return W12_ERR_ARG;
  if (!stride_ok(q_token_stride) || !stride_ok(q_head_stride) || !stride_ok(k_token_stride) || !stride_ok(k_head_stride) ||
      !stride_ok(v_token_stride) || !stride_ok(v_head_stride))
    return W12_ERR_ARG;
  if (!device_supported()) return W12_ERR_UNSUPPORTED;
  Params P{};
  P.V = V;
  P.v_tok = v_token_stride;
  P.v_head = v_head_stride;
  P.O = O;
  P.cu = cu_seqlens;
  P.status = dev_status;
  P.total = total;
  P.B = B;
  P.Hq = Hq;
  P.Hkv = Hkv;
  P.G = Hq / Hkv;
  P.tpt = 128 / P.G;
  P.inv_g = 65536u / P.G + 1;  // (exact for 128 rows)
  P.room = kGroupBytes / (4 * Hkv * head_dim) + 1;
  P.c = float(double(scale) * 1.4426950408889634);
  P.limit_ns = wait_limit_ns();
  P.sleep_ns = sleep_ns(P.limit_ns);
  const bool bf16 = dtype == W12_BF16;
  CUtensorMap q, k, v;
  const int keys = head_dim == 128 ? Cfg<128>::kKeys : Cfg<64>::kKeys;
  if (!row_map(&q, Q, bf16, head_dim, Hq, total, q_token_stride, q_head_stride, P.G, P.tpt) ||
      !row_map(&k, K, bf16, head_dim, Hkv, total, k_token_stride, k_head_stride, 1, keys) ||
      !row_map(&v, V, bf16, head_dim, Hkv, total, v_token_stride, v_head_stride, 1, keys))
    return W12_ERR_CUDA;
  const int sms = device_sm_count();
  const int64_t pairs = (total / (2 * P.tpt) + B) * Hkv;
  // One tile an item where that leaves no block with two: tiles then do not share a block's schedulers
  // (400 tokens, 40 / 8 heads of 128: 8.8 us, pairs 10.4; 777, where blocks would have two: 15.2, pairs 14.3).
  P.step = pairs <= sms / 2 ? P.tpt : 2 * P.tpt;
  const int64_t most = (total / P.step + B) * Hkv;
  const unsigned grid = unsigned(most < sms ? most : sms);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(head_dim == 128 ? (bf16 ? launch<128, true>(q, k, v, P, grid, s) : launch<128, false>(q, k, v, P, grid, s))
                                     : (bf16 ? launch<64, true>(q, k, v, P, grid, s) : launch<64, false>(q, k, v, P, grid, s)));
}

}  // extern "C"
