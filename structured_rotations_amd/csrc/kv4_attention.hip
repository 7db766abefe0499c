// Attention over a cache in 4 bits.
//
// For one key head, the rows of a sequence are its call's tokens times the
// query heads that share the key head.  With S = K Q^T (keys by rows), the matrix
// instructions' layouts fit one another: what a lane holds of S, for one row of Q
// and some keys, is what it has to give of P to the product with V, so the
// softmax needs no exchange but the maximum.  The order of keys within a step is
// free; it is the one in which S comes out.
//
// K's and V's codes become bf16 exactly (E2M1 times a power of two) by one
// conversion instruction for two values, scale included.  A lane's piece of K
// is as it is in memory; two neighbours of V belong to one key and two columns,
// where a product wants two keys of one column.  The kernel for few rows lets
// the instruction pick them (mfma_pairs), the one for many pairs them by byte
// permutations when it puts them into LDS.
//
// Scores, weights, maxima, sums and accumulators are fp32.  The product with V
// takes the weights as bf16.  Rounding them once is off by up to 2^-8 of each, of
// the heaviest too, since a row's weights go by a reference that its largest score
// may pass.
// - Tiles of 16 rows: what the rounding left off goes into a second product, which
//   leaves 2^-16 of a weight, and the result off by its own rounding only (1.57e-3
//   in relative l2 against 64 bits; with one product 1.7e-3).  Bytes bound this kernel:
//   64 x 1 over 50 .. 8192 keys, 32/8 x 128, 71.5 us, with one product 69.8.
// - Tiles of 32 and 128 rows: products and vector work count, and a second product
//   costs more (64 x 8 over 4096, 64/8 x 128: 150 us, one 134; 4 x 2048 over 8192, 32/8 x
//   128: 832, one 640).  There is one, and what divides it is the sum of the weights as
//   they were rounded (138 and 656 us): rounding then moves a result by up to 2^-8 of the
//   values' distances from it, not of the values, and a row with one heavy key not at
//   all.  (4 x 2048 over 2048 .. 8192: off by 1.69e-3, by the result's rounding alone 1.57e-3.)
//   lse takes the sum of the weights as they were.
#include <algorithm>
#include <climits>
#include <cmath>

#include "kv4.h"
#include "q8.h"

namespace harp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16_t __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ bf16x8_t as_frag(const uint32_t (&w)[4]) {
  bf16x8_t r;
  __builtin_memcpy(&r, w, 16);
  return r;
}
__device__ __forceinline__ f32x4 mfma16(const bf16x8_t& a, const bf16x8_t& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Adds the product of P and of one column of every pair in V.  An instruction for
// matrices of which two of four values are zero takes only the two, and the
// places (a bit pair each) that they have: of V's values (key 0, column 0), (key
// 0, column 1), (key 1, column 0), (key 1, column 1) the places 0 and 2 or 1 and
// 3 are one column's keys, at the price of a product without the other.
template <int kOdd>
__device__ __forceinline__ f32x4 mfma_pairs(const bf16x8_t& p, const bf16x16_t& v, const f32x4& c) {
  return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(p, v, c, kOdd ? 0xdddd : 0x8888, 0, 0);
}
// Byte kByte's two codes, times 2^(e - 127), e in the exponent's place.
template <int kByte>
__device__ __forceinline__ uint32_t widen4(uint32_t codes, uint32_t e) {
  const bf16x2_t v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __uint_as_float(e), kByte);
  uint32_t w;
  __builtin_memcpy(&w, &v, 4);
  return w;
}
// One factor for each of two weights rounded to bf16 (w), and an fp32 number added
// to the products.  (Exact where the result has no more than 24 bits.)
template <uint32_t kFactors>
__device__ __forceinline__ float dot_weights(uint32_t w, float c) {
  uint32_t factors = kFactors;
  asm("" : "+s"(factors));  // in a register: -1 in the lower half would become the instruction's own -1.0, which is in the upper
  bf16x2_t x, y;
  __builtin_memcpy(&x, &w, 4);
  __builtin_memcpy(&y, &factors, 4);
  return __builtin_amdgcn_fdot2_f32_bf16(x, y, c, false);
}
// What their rounding left off two weights, as bf16.
__device__ __forceinline__ uint32_t left_off(uint32_t w, float a, float b) {
  return pack_bf16x2_hw(dot_weights<0x0000bf80u>(w, a), dot_weights<0xbf800000u>(w, b));  // -1, 0; 0, -1
}
// Largest over the lanes that are 16 and 32 apart, in every one of them.
__device__ __forceinline__ float max_of_groups(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_of_groups(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float max_of_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_of_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// An address that all lanes have in common, kept in scalar registers: loads add
// the lane's offset themselves, where the compiler would add it before the loop
// and the address to that, lane by lane.
template <typename T>
using Global = const __attribute__((address_space(1))) T*;
__device__ __forceinline__ Global<uint8_t> common(const uint8_t* p) {
  uint64_t at = reinterpret_cast<uint64_t>(p);
  asm("" : "+s"(at));
  return reinterpret_cast<Global<uint8_t>>(at);
}
template <typename T>
__device__ __forceinline__ T load_at(Global<uint8_t> base, uint32_t lane_offset, int offset) {
  return *reinterpret_cast<Global<T>>(base + lane_offset + offset);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// The rows of one workgroup's tile, all of one sequence, and the keys that
// they see: row r (0 ..) of the sequence's is token r / group, head r % group.
struct TileRows {
  int seq, first_token, tokens, len;  // the call's array; the sequence's length
  int row0, rows;                     // the tile's first row; the sequence's (tokens x heads: 2^30 at most)
  __device__ __forceinline__ int pos(int64_t token) const { return (int)((int64_t)len - tokens + token); }
};
// Tiles of kRows rows: sequence b's begin at starts[b] group / kRows + b, which
// leaves it as many as it needs, whatever its neighbours have.
__device__ __forceinline__ bool tile_rows(const Attn4Args& a, int64_t tile, int tile_size, TileRows* t) {
  const auto first = [&](int b) { return (int64_t)a.plan.starts[b] * a.group / tile_size + b; };
  const int b = __builtin_amdgcn_readfirstlane(last_at_most(a.plan.sequences, tile, first));
  const int s0 = min(max(a.plan.starts[b], 0), a.tokens), s1 = min(max(a.plan.starts[b + 1], s0), a.tokens);
  t->seq = b;
  t->first_token = s0;
  t->tokens = s1 - s0;
  t->len = max(a.plan.lengths[b], 0);
  t->rows = t->tokens * a.group;
  const int64_t row0 = (tile - first(b)) * tile_size;
  if (row0 < 0 || row0 >= t->rows) return false;
  t->row0 = (int)row0;
  return true;
}
// The keys lo .. hi - 1 that the token at position pos sees.  Beyond what the
// table has room for (`cap` keys), one place stands for all the others: it has
// no page, and so is NaN.
struct Sees {
  int lo, hi;
};
__device__ __forceinline__ Sees sees(const Attn4Args& a, int len, int pos, int64_t cap) {
  if (pos < 0) return {0, 0};
  int64_t hi = a.causal ? (int64_t)pos + 1 : len, lo = a.window ? max(0, pos - a.window + 1) : 0;
  return {(int)min(lo, cap), (int)min(hi, cap + 1)};
}

// The keys that a workgroup's rows see, lo .. hi - 1, and its part of them, in
// steps of kStep keys from `base` on.
struct KeyRange {
  int lo, hi, base, step0, step1;
};
template <int kStep>
__device__ __forceinline__ KeyRange key_range(const Attn4Args& a, const TileRows& t, int tile_size, int64_t cap, int split,
                                              int splits, int unit) {
  const uint32_t group = a.group, last = min(t.row0 + tile_size, t.rows) - 1;
  const int tok0 = (int)((uint32_t)t.row0 / group), tok1 = (int)(last / group);
  const Sees s0 = sees(a, t.len, t.pos(tok0), cap), s1 = sees(a, t.len, t.pos(tok1), cap);
  KeyRange r;
  r.hi = max(s0.hi, s1.hi);
  r.lo = t.pos(tok0) < 0 ? 0 : s0.lo;
  r.base = r.lo & ~(kStep - 1);
  const int steps = r.hi > r.lo ? (int)(((int64_t)r.hi - r.base + kStep - 1) / kStep) : 0;
  const int per = ((steps + splits * unit - 1) / (splits * unit)) * unit;
  r.step0 = min(steps, split * per);
  r.step1 = min(steps, r.step0 + per);
  return r;
}

// The scale of four keys' blocks, of which `vs` holds all scales: the block of
// a lane is blk0 + blk (blk < kSpan).  As a word's highest byte.
template <int ND, int kSpan>
__device__ __forceinline__ uint32_t scale_of(const uint32_t (&vs)[ND], int key, int blk0, int blk) {
  const int at = ND * key + blk0, in = at / 4;
  const uint32_t lo = vs[in], hi = at % 4 + kSpan > 4 ? vs[in + 1 < ND ? in + 1 : in] : lo;
  return __builtin_amdgcn_perm(hi, lo, (uint32_t)(at % 4 + blk) << 24 | 0x0c0c0cu);
}
// The same, in an exponent's place, with other bits around it, which a conversion does not look at.
template <int ND, int kSpan>
__device__ __forceinline__ uint32_t exponent_of(const uint32_t (&vs)[ND], int key, int blk0, int blk) {
  const int at = ND * key + blk0, in = at / 4;
  if (at % 4 + kSpan > 4) return scale_of<ND, kSpan>(vs, key, blk0, blk) >> 1;
  return __builtin_amdgcn_alignbit(vs[in], vs[in], 8 * (at % 4 + blk) + 9);
}
constexpr uint32_t kNanScale = 0xff000000u;  // of such words, and above

// Weights go by a reference that a score may pass by this much (in powers of
// two) before the sums are brought to a new one, which is then rarely needed.
constexpr float kSlack = 8.0f;

// ------------------------------------------------------------- few rows
// The four waves of a workgroup take 32 keys at a time in turn.  A wave's loads go
// straight into a ring of its own in LDS, kDepth - 1 steps ahead: what keeps HBM
// busy is bytes in flight, and registers are too few for them.  No barrier is
// needed: a wave reads what it loaded itself.  (64 x 1 over 16384, 32/8 x 128:
// 218 us, 5.2 TB/s; a copy of this kernel without its arithmetic reads 5.2 to 5.5
// TB/s, so what is left there is the order of the reads.)
//
// A step in LDS, of two halves of 16 keys each (their pages may differ):
//   K   ND % 4 == 0: as the lanes take it, 16 bytes each, one after the other;
//       else the rows as they are
//   V   by parts of the columns.  Lane c of 16 has the columns 8 c .. of a part
//       of 128 (a word of a row), 4 c .. of one of 64 (a half), 2 c .. of one of
//       32 (a byte).  Of four keys 4 j + i, i outermost, so that a wave's words
//       are in different banks; the second half is kSkew further for the same.
//   scales of K, of V: rows as they are
template <int ND>
struct Step4 {
  static constexpr int kUnit = ND % 4 == 0 ? 4 : ND % 2 == 0 ? 2 : 1;  // words of K that a lane takes at once
  static constexpr int kWords = ND / 4, kHalf = (ND >> 1) & 1, kByte = ND & 1;
  static constexpr int kSide = 256 * ND;                     // 16 keys' codes
  static constexpr int kV = 2 * kSide, kSkew = 64;  // where V begins; what the second half is off, for the banks' sake
  static constexpr int kScales = 4 * kSide + kSkew;
  static constexpr int kBytes = kScales + 64 * ND;
  static constexpr int kLoads = 2 * ((ND + 3) / 4) + 2 * (kWords + kHalf + kByte) + 2;
  static constexpr int kDepth = ND <= 4 ? 3 : 2;
};

// How the keys are shared out.  An item is a tile of rows of one sequence with one
// key head; it takes steps of 32 keys, as many for every tile of a sequence.  All
// steps of all items, one after the other, are cut into equal parts, one for
// each workgroup that has room on the chip: whatever the lengths are, which only
// the device knows, the parts are done at about the same time.  A workgroup
// finishes items that are its own as a whole; of others it leaves parts: in its
// first slot that of the item that began before it, in its second slot that of
// the one that it begins and does not end.  (64 x 1 over 50 .. 8192 keys, 32/8 x
// 128, with one product for V: 70 us; cut as for sequences of the table's width, one
// workgroup for an item or a fixed fraction of one: 82.  64 x 4 over 4096: 76, not 100.)
//
// Where there are many items for each workgroup (see cut_of) each has one of its
// own instead, and the chip's scheduler evens them out: the way from one item to
// the next costs a workgroup about as much as 12 steps, mostly waiting, which
// another workgroup's start does not (1024 x 1 over 1024, with one product for V: 235
// us, not 257; with two 243).
constexpr int kLeastSteps = 8;  // of a part
constexpr int kItemSteps = 12;  // what an item weighs besides its steps, half of it on either side of them
struct Work {
  int first_token, tokens, len;
  int each, tiles;  // steps of an item (and kItemSteps), tiles of the sequence
};
__device__ __forceinline__ Work work_of(const Attn4Args& a, int b, int tile_size, int64_t cap) {
  Work w{};
  if (b >= a.plan.sequences) return w;
  const int s0 = min(max(a.plan.starts[b], 0), a.tokens), s1 = min(max(a.plan.starts[b + 1], s0), a.tokens);
  w.first_token = s0;
  w.tokens = s1 - s0;
  w.len = max(a.plan.lengths[b], 0);
  const int64_t hi = min((int64_t)w.len, cap + 1);
  // with a window, a tile's first token sees back from its place, and steps begin at multiples of 32
  const int64_t span = a.window && a.causal ? min(hi, (int64_t)a.window + tile_size + 32) : hi;
  w.each = (int)((span + 31) >> 5) + kItemSteps;
  w.tiles = (w.tokens * a.group + tile_size - 1) / tile_size;
  return w;
}
__device__ __forceinline__ Work uniform(Work w) {
  const auto u = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  return {u(w.first_token), u(w.tokens), u(w.len), u(w.each), u(w.tiles)};
}
// x / y of numbers from 0 on: exact below 2^52, where a fraction's distance from
// the next integer is more than the rounding of the quotient.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) { return (int64_t)((double)x / (double)y); }
__device__ __forceinline__ int64_t scan_of(int64_t v) {  // inclusive, over the wave
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int64_t below = __shfl_up((long long)v, o);
    if ((int)(threadIdx.x & 63) >= o) v += below;
  }
  return v;
}
__device__ __forceinline__ int64_t last_lane(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, 63) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), 63) << 32);
}

// Waits until at most kLeft of the wave's loads are under way.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kLeft) : "memory");
}
// Loads straight into LDS, `lds` and on, lane by lane: 16 bytes from an address
// that all lanes have in common and the lane's offset, or 4 from the lane's own
// address.  kAt is added on both sides.  (The waits: see load_lds16 in q8.h.)
template <int kAt>
__device__ __forceinline__ void load_lds16_at(Global<uint8_t> base, uint32_t lane_offset, uint32_t lds) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %2, %3 offset:%4"
               : "={m0}"(m0)
               : "s"(lds), "v"(lane_offset), "s"(base), "n"(kAt)
               : "memory");
}
__device__ __forceinline__ void load_lds4_at(Global<uint8_t> base, uint32_t lane_offset, uint32_t lds) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dword %2, %3"
               : "={m0}"(m0)
               : "s"(lds), "v"(lane_offset), "s"(base)
               : "memory");
}
__device__ __forceinline__ void load_lds4(uint64_t from, uint32_t lds) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dword %2, off" : "={m0}"(m0) : "s"(lds), "v"(from) : "memory");
}

// The workspace: two slots of a tile's rows for each workgroup (values, then each
// row's maximum and sum), then for each row of the call the first workgroup that
// has a part of it, and how many have (<< 8) with its place in the tile, or 0
// where there is nothing to add.
struct Slots {
  float* values;
  f32x2* stats;
  int2* of_row;
};
__device__ __forceinline__ Slots slots_of(float* workspace, int groups, int tile_size, int d) {
  Slots s;
  const int64_t rows = 2LL * groups * tile_size;
  s.values = workspace;
  s.stats = reinterpret_cast<f32x2*>(workspace + rows * d);
  s.of_row = reinterpret_cast<int2*>(s.stats + rows);
  return s;
}

// Workgroups a compute unit is to have room for, which bounds the registers: as
// many as these and LDS allow without spilling (one register of heads of 160 in tiles
// of 32 rows is) (64 x 1 over 4096, d = 192, 16 heads: 2 58 us, 3, of 168 registers, 63;
// d = 96: 3 and 4, of 128, 64).
constexpr int room_for(int nd, int nq) {
  return nq == 1 ? (nd <= 2 ? 4 : nd <= 4 ? 3 : 2) : nd == 1 ? 4 : nd == 2 ? 3 : nd <= 5 ? 2 : 1;
}

template <int ND, int NQ>
__global__ __launch_bounds__(256, room_for(ND, NQ)) void kv4_attention_kernel(Attn4Args a, int parts, int64_t item0) {
  using Step = Step4<ND>;
  constexpr int kRow = ND * 16, kTileRows = 16 * NQ, kAcc = 2 * ND, kD = ND * 32;
  constexpr bool kExact = NQ == 1;  // weights as two bf16 numbers
  const int own_lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ps_log2 = a.cache.page_log2;
  const int64_t cap = (int64_t)a.plan.width << ps_log2;

  // the rings of the four waves; at an item's end what they have to add
  constexpr int kPad = kD + 4, kRing = Step::kBytes * Step::kDepth, kShare = 16 * kPad * 4;
  __shared__ __attribute__((aligned(16))) uint8_t memory[4 * (kRing > kShare ? kRing : kShare)];
  __shared__ float stat[4][16][2];
  const uint8_t* ring = memory + wave * kRing;
  const uint32_t ring_at = lds_address(ring);

  // the part: steps `at` .. `end` - 1 of all
  const int sequences = a.plan.sequences, heads = a.cache.heads;
  const bool whole = parts == 0;  // one item, all of it
  Work of;
  int seq, tile, kvh, first = 0;  // the item, and its step where the part begins
  int64_t at = 0, end = 1, chunk = 1;
  if (whole) {
    const int64_t unit = item0 + blockIdx.x, of_tile = quotient(unit, heads);
    TileRows t;
    if (!tile_rows(a, of_tile, kTileRows, &t)) return;
    of = {t.first_token, t.tokens, t.len, 1, INT_MAX};
    seq = t.seq;
    tile = t.row0 / kTileRows;
    kvh = (int)(unit - of_tile * heads);
  } else {
    const auto weight = [&](const Work& w) { return (int64_t)w.tiles * heads * w.each; };
    const int per = (sequences + 63) / 64;  // sequences to a lane
    Work work = work_of(a, own_lane * per, kTileRows, cap);
    int64_t own = weight(work);
#pragma unroll 4
    for (int i = 1; i < per; ++i)  // (64 of these do not pass 63 bits)
      own = min(own + weight(work_of(a, own_lane * per + i, kTileRows, cap)), (int64_t)1 << 56);
    int64_t up_to = scan_of(own);
    // A plan whose rows overlap may ask for more than any other can: no more than that is done.
    const int64_t each = ((min(cap, (int64_t)INT_MAX) + 32) >> 5) + kItemSteps;
    const int64_t most = ((int64_t)a.tokens * a.group / kTileRows + sequences) * heads * each;
    const int64_t total = min(last_lane(up_to), most);
    chunk = max(quotient(total + parts - 1, parts), (int64_t)kLeastSteps);
    at = chunk * blockIdx.x;
    end = min(total, at + chunk);
    if (at >= end) return;
    int64_t before = 0;  // steps of the sequences before seq
    const auto of_who = [&](int who, int x) { return __builtin_amdgcn_readlane(x, who); };
    const auto find = [&]() {  // the lane whose steps `at` is one of
      const int who = __ffsll((unsigned long long)__ballot(before + up_to > at)) - 1;
      const int64_t less = up_to - own;
      before +=
          (int64_t)((uint64_t)(uint32_t)of_who(who, (int)less) | (uint64_t)(uint32_t)of_who(who, (int)(less >> 32)) << 32);
      return who;
    };
    int who = find();
    seq = who * per;
    if (per > 1) {
      for (int left = min(per, sequences - seq);; seq += 64, left -= 64) {
        work = work_of(a, own_lane < left ? seq + own_lane : sequences, kTileRows, cap);
        own = weight(work);
        up_to = scan_of(own);
        const int64_t all = last_lane(up_to);
        if (at < before + all || left <= 64) break;
        before += all;
      }
      who = find();
      seq += who;
    }
    of = {of_who(who, work.first_token), of_who(who, work.tokens), of_who(who, work.len), of_who(who, work.each),
          of_who(who, work.tiles)};
    const int item = (int)quotient(at - before, of.each);
    tile = item / heads;
    kvh = item - tile * heads;
    first = (int)min(max(at - before - (int64_t)item * of.each, (int64_t)0), (int64_t)of.each - 1);
  }
  const int64_t begin = at;
  while (at < end) {
  // (offsets made of it are not kept from one item to the next, which costs registers)
  int lane = own_lane;
  asm volatile("" : "+v"(lane));
  const int c16 = lane & 15, g = lane >> 4;
  const int count = (int)min((int64_t)(of.each - first), end - at);
  const int64_t item_at = at - first;
  const bool begins = item_at >= begin, shared = !begins || item_at + of.each > end;
  const int kvh_now = kvh;
  TileRows t;
  t.seq = seq;
  t.first_token = of.first_token;
  t.tokens = of.tokens;
  t.len = of.len;
  t.rows = of.tokens * a.group;
  t.row0 = tile * kTileRows;
  const int each = of.each;
  const KeyRange keys = key_range<32>(a, t, kTileRows, cap, 0, 1, 1);
  const int hi_all = keys.hi, lo_all = keys.lo, base = keys.base;
  const int step0 = min(keys.step1, max(first - kItemSteps / 2, 0));  // 0 of a whole item
  const int step1 = whole ? keys.step1 : min(keys.step1, max(first + count - kItemSteps / 2, 0));
  // on to the next item
  at += count;
  first = 0;
  if (++kvh == heads) {
    kvh = 0;
    if (++tile == of.tiles) {
      tile = 0;
      do {
        ++seq;
        of = uniform(work_of(a, seq, kTileRows, cap));
      } while (of.tiles == 0 && seq < sequences);
      if (seq >= sequences) end = at;
    }
  }

  // this lane's row of each tile of 16: its queries, its keys
  Sees row_sees[NQ];
  bf16x8_t q[NQ][ND];
  int hi_min = hi_all, lo_max = lo_all;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = t.row0 + n * 16 + c16;
    const bool has = r < t.rows;
    const int tok = has ? (int)((uint32_t)r / (uint32_t)a.group) : 0, gh = has ? r - tok * a.group : 0;
    row_sees[n] = has ? sees(a, t.len, t.pos(tok), cap) : Sees{0, 0};
    if (has) {
      hi_min = min(hi_min, row_sees[n].hi);
      lo_max = max(lo_max, row_sees[n].lo);
    }
    const uint16_t* p = a.q + (int64_t)(t.first_token + tok) * a.q_token + (int64_t)(kvh_now * a.group + gh) * a.q_head;
#pragma unroll
    for (int s = 0; s < ND; ++s) {
      const int u = s / Step::kUnit, in = s % Step::kUnit;
      const int col = (u * 4 + g) * Step::kUnit * 8 + in * 8;
      Raw8<uint16_t> w;
      w.fill(0);
      if (has) w.load(p + col, 8);
      q[n][s] = as_frag(w.w);
    }
  }
  // what the rows that see most and least leave to be masked
#pragma unroll
  for (int o = 1; o < 16; o *= 2) {
    hi_min = min(hi_min, __shfl_xor(hi_min, o));
    lo_max = max(lo_max, __shfl_xor(lo_max, o));
  }
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);

  f32x4 acc[NQ][kAcc];
  float m[NQ], l[NQ], rounded[NQ];  // sums of the weights, as they are and as a single bf16 number
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = rounded[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[n][i] = f32x4{0, 0, 0, 0};
  }
  const float to_log2 = a.scale * kLog2e;

  // Pages of the next 32 steps, two to a step, in the lanes.
  int pages = -1;
  auto look_up = [&](int step) {
    const int64_t key = (int64_t)base + ((int64_t)step + (lane >> 1) * 4) * 32 + (lane & 1) * 16;
    pages = key < hi_all ? page_of(a.cache, a.plan, t.seq, key >> ps_log2) : -1;
  };
  // the key head's places in a page
  const uint8_t* const k_at = a.cache.k.codes + ((int64_t)kvh_now << ps_log2) * kRow;
  const uint8_t* const v_at = a.cache.v.codes + ((int64_t)kvh_now << ps_log2) * kRow;
  const int64_t scales_at = ((int64_t)kvh_now << ps_log2) * ND;
  uint32_t lost = 0;  // slot by slot, two bits: keys without a page
  // 16 keys' codes, kHalves halves of them that follow one another
  auto load_codes = [&](auto halves_c, Global<uint8_t> k, Global<uint8_t> v, uint32_t to, uint32_t skew) {
    constexpr int kHalves = decltype(halves_c)::value;
    auto half = [&](auto s_c) {
      constexpr int kAt = decltype(s_c)::value * Step::kSide;  // 16 rows in memory, and their place in LDS
      const uint32_t v_to = to + Step::kV + skew + decltype(s_c)::value * Step::kSkew;
#pragma unroll
      for (int u = 0; u < (ND + 3) / 4; ++u) {
        const uint32_t off = ND % 4 == 0 ? c16 * kRow + g * 16 + u * 64 : lane * 16 + u * 1024;
        if (ND % 4 == 0 || lane < 16 * ND - 64 * u) load_lds16_at<kAt>(k, off, to + u * 1024);
      }
#pragma unroll
      for (int u = 0; u < Step::kWords; ++u)
        load_lds16_at<kAt>(v, (4 * ((lane >> 2) & 3) + (lane >> 4)) * kRow + (lane & 3) * 16 + u * 64,
                           v_to + u * 1024);
      if constexpr (Step::kHalf)
        if (lane < 32)
          load_lds16_at<kAt>(v, (4 * ((lane >> 1) & 3) + (lane >> 3)) * kRow + (lane & 1) * 16 + Step::kWords * 64,
                             v_to + Step::kWords * 1024);
      if constexpr (Step::kByte)
        if (lane < 16)
          load_lds16_at<kAt>(v, (4 * (lane & 3) + (lane >> 2)) * kRow + kRow - 16,
                             v_to + Step::kWords * 1024 + Step::kHalf * 512);
    };
    half(std::integral_constant<int, 0>{});
    if constexpr (kHalves == 2) half(std::integral_constant<int, 1>{});
  };
  auto load = [&](int step, int page_at, int slot) {
    const uint32_t to = ring_at + slot * Step::kBytes;
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // the slot's last step has been read
    const uint32_t key = (uint32_t)base + (uint32_t)step * 32, in_page = key & ((1u << ps_log2) - 1);
    const int page = __builtin_amdgcn_readlane(pages, 2 * page_at);
    const int64_t pg = max(page, 0), in_scales = scales_at + (int64_t)in_page * ND;
    const auto k = common(k_at + pg * a.cache.k.codes_page + (int64_t)in_page * kRow);
    const auto v = common(v_at + pg * a.cache.v.codes_page + (int64_t)in_page * kRow);
    const auto ks = common(a.cache.k.scales + pg * a.cache.k.scales_page + in_scales);
    const auto vs = common(a.cache.v.scales + pg * a.cache.v.scales_page + in_scales);
    const uint32_t scales_to = to + Step::kScales;
    uint32_t missing = page < 0 ? 3 : 0;
    if (ps_log2 > 4) {  // all 32 keys in one page (of which 16 may not be the sequence's)
      load_codes(std::integral_constant<int, 2>{}, k, v, to, 0);
      if (ND == 8 || lane < 8 * ND) {
        load_lds4_at(ks, lane * 4, scales_to);
        load_lds4_at(vs, lane * 4, scales_to + 32 * ND);
      }
    } else {
      const int page2 = __builtin_amdgcn_readlane(pages, 2 * page_at + 1);
      const int64_t pg2 = max(page2, 0);
      missing = (page < 0 ? 1 : 0) | (page2 < 0 ? 2 : 0);
      load_codes(std::integral_constant<int, 1>{}, k, v, to, 0);
      load_codes(std::integral_constant<int, 1>{}, common(k_at + pg2 * a.cache.k.codes_page),
                 common(v_at + pg2 * a.cache.v.codes_page), to + Step::kSide, Step::kSkew);
      if (ND == 8 || lane < 8 * ND) {
        const auto own = [&](Global<uint8_t> one, Global<uint8_t> two) {
          return reinterpret_cast<uint64_t>(lane < 4 * ND ? one : two - 16 * ND) + lane * 4;
        };
        load_lds4(own(ks, common(a.cache.k.scales + pg2 * a.cache.k.scales_page + scales_at)), scales_to);
        load_lds4(own(vs, common(a.cache.v.scales + pg2 * a.cache.v.scales_page + scales_at)), scales_to + 32 * ND);
      }
    }
    lost = (lost & ~(3u << (2 * slot))) | missing << (2 * slot);
  };

  uint32_t poison[NQ];  // blocks of the row's result that are NaN
#pragma unroll
  for (int n = 0; n < NQ; ++n) poison[n] = 0;

  auto compute = [&](int step, int slot) {
    const int k0 = (int)((uint32_t)base + (uint32_t)step * 32);
    const uint8_t* in = ring + slot * Step::kBytes;
    const uint32_t missing = lost >> (2 * slot) & 3;
    // scores: rows of keys, columns of queries
    f32x4 z[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) z[n][0] = z[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < ND / Step::kUnit; ++u) {
      uint32_t kw[2][Step::kUnit], e[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* k = in + s * Step::kSide;
        if constexpr (Step::kUnit == 4) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(k + u * 1024 + lane * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) kw[s][i] = x[i];
        } else if constexpr (Step::kUnit == 2) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(k + c16 * kRow + (u * 4 + g) * 8);
          kw[s][0] = x[0];
          kw[s][1] = x[1];
        } else {
          kw[s][0] = *reinterpret_cast<const uint32_t*>(k + c16 * kRow + (u * 4 + g) * 4);
        }
        e[s] = (uint32_t)in[Step::kScales + (16 * s + c16) * ND + (u * 4 + g) * Step::kUnit / 4] << 23;
      }
      if (missing) {
        asm volatile("");  // (a branch)
        if (missing & 1) e[0] = 255u << 23;  // no page: NaN
        if (missing & 2) e[1] = 255u << 23;
      }
#pragma unroll
      for (int i = 0; i < Step::kUnit; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t f[4] = {widen4<0>(kw[s][i], e[s]), widen4<1>(kw[s][i], e[s]), widen4<2>(kw[s][i], e[s]),
                                 widen4<3>(kw[s][i], e[s])};
#pragma unroll
          for (int n = 0; n < NQ; ++n) z[n][s] = mfma16(as_frag(f), q[n][u * Step::kUnit + i], z[n][s]);
        }
    }
    if (k0 < lo_max || (uint32_t)k0 + 32 > (uint32_t)hi_min) {  // some row does not see all of these keys
      asm volatile("");                     // a branch, no 16 comparisons at every step
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int lo = row_sees[n].lo - k0, hi = row_sees[n].hi - k0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * s + 4 * g + r;
            z[n][s][r] = j >= lo && j < hi ? z[n][s][r] : -INFINITY;
          }
      }
    }
    bf16x8_t p[NQ], rest[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = z[n][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, z[n][i >> 2][i & 3]);
      top *= to_log2;
      if (__any(top > m[n] + kSlack)) {
        const float now = fmaxf(m[n], max_of_groups(top));
        const float shrink = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[n] - now);
        m[n] = now;
        l[n] *= shrink;
        rounded[n] *= shrink;
        f32x4 of_row;  // the accumulators' rows are the queries
#pragma unroll
        for (int r = 0; r < 4; ++r) of_row[r] = __shfl(shrink, 4 * g + r);
#pragma unroll
        for (int i = 0; i < kAcc; ++i) acc[n][i] *= of_row;
      }
      const float less = m[n] == -INFINITY ? 0.0f : m[n];
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(fmaf(z[n][i >> 2][i & 3], to_log2, -less));
        l[n] += e[i];
      }
      uint32_t f[4], left[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = pack_bf16x2_hw(e[2 * i], e[2 * i + 1]);
        if constexpr (kExact) left[i] = left_off(f[i], e[2 * i], e[2 * i + 1]);
        else rounded[n] = dot_weights<0x3f803f80u>(f[i], rounded[n]);  // 1, 1
      }
      p[n] = as_frag(f);
      if constexpr (kExact) rest[n] = as_frag(left);
    }
    // V's columns by parts: 8 columns to a lane (words), 4 (halves), 2 (bytes).  A product's lane of P has keys 4 g ..
    // of both halves; to them belong, in the lanes of V, of half g % 2 the keys 4 (g / 2) .. and 8 + 4 (g / 2) ..
    const int side = g & 1, key0 = 4 * (g >> 1);  // key i of the lane's 8: half `side`, key0 + 8 (i / 4) + i % 4
    const bool edge = k0 < lo_all || (uint32_t)k0 + 32 > (uint32_t)hi_all;
    const uint32_t* scales = reinterpret_cast<const uint32_t*>(in + Step::kScales + 32 * ND);
    bool some_nan = false;  // a byte of the step's scales is 255
    if (ND == 8 || lane < 8 * ND) {
      const uint32_t w = scales[lane];
      some_nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u;
    }
    some_nan = __any(some_nan);
    uint32_t vs[2][ND];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < ND; ++i) vs[h][i] = scales[(16 * side + key0 + 8 * h) / 4 * ND + i];
    if (missing) {  // another page's: nothing that is not finite
      asm volatile("");
      const bool mine = missing >> side & 1;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < ND; ++i) vs[h][i] = mine ? 0 : vs[h][i];
    }
    const uint8_t* v_in = in + Step::kV + side * (Step::kSide + Step::kSkew);
#pragma unroll
    for (int part = 0; part < Step::kWords + Step::kHalf + Step::kByte; ++part) {
      const bool word = part < Step::kWords, half = !word && part == Step::kWords && Step::kHalf;
      const int bytes = word ? 4 : half ? 2 : 1;
      const int tile0 = word ? part * 8 : Step::kWords * 8 + (half ? 0 : Step::kHalf * 4);
      const int blk0 = word ? part * 4 : half ? Step::kWords * 4 : ND - 1;
      const int blk = word ? c16 >> 2 : half ? c16 >> 3 : 0;
      uint32_t e[8];  // of the lane's block
#pragma unroll
      for (int i = 0; i < 8; ++i)
        e[i] = word   ? exponent_of<ND, 4>(vs[i >> 2], i & 3, blk0, blk)
               : half ? exponent_of<ND, 2>(vs[i >> 2], i & 3, blk0, blk)
                      : exponent_of<ND, 1>(vs[i >> 2], i & 3, blk0, blk);
      if (edge) {  // what lies outside may hold anything
        asm volatile("");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = k0 + 16 * side + key0 + 8 * (i >> 2) + (i & 3);
          e[i] = j >= lo_all && j < hi_all ? e[i] : 0;
        }
      }
      if (some_nan) {
        // NaN times a weight of 0 would reach rows that do not see the key: such a block counts as 0, and is noted for
        // the rows that do see it
        uint32_t nan_keys = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((e[i] >> 23 & 255) == 255) {
            nan_keys |= 1u << i;
            e[i] = 0;
          }
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
          const uint32_t who = (uint32_t)(__ballot(nan_keys >> (i & 7) & 1) >> (16 * (i >> 3))) & 0xffff;
          if (who == 0) continue;
          const int j = k0 + 16 * (i >> 3 & 1) + 8 * ((i & 7) >> 2) + 4 * (i >> 4) + (i & 3);
          uint32_t blocks = who ? 1 : 0;
          if (word)
            blocks = (who & 0xf ? 1 : 0) | (who & 0xf0 ? 2 : 0) | (who & 0xf00 ? 4 : 0) | (who & 0xf000 ? 8 : 0);
          else if (half) blocks = (who & 0xff ? 1 : 0) | (who & 0xff00 ? 2 : 0);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            if (j >= row_sees[n].lo && j < row_sees[n].hi) poison[n] |= blocks << blk0;
        }
      }
      uint32_t vw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // four keys' pieces of a part follow one another, key % 4 outermost
        const uint8_t* v = v_in + Step::kWords * 1024 * !word + Step::kHalf * 512 * (!word && !half);
        const int at = (i & 3) * 64 + (key0 / 4 + 2 * (i >> 2)) * 16 + c16;
        if (word) vw[i] = reinterpret_cast<const uint32_t*>(v + part * 1024)[at];
        else if (half) vw[i] = reinterpret_cast<const uint16_t*>(v)[at];
        else vw[i] = v[at];
      }
      auto columns = [&](auto byte_c) {
        constexpr int byte = decltype(byte_c)::value;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = widen4<byte>(vw[i], e[i]);
        bf16x16_t pairs;
        __builtin_memcpy(&pairs, w, 32);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          f32x4 &even = acc[n][tile0 + 2 * byte], &odd = acc[n][tile0 + 2 * byte + 1];
          even = mfma_pairs<0>(p[n], pairs, even);
          odd = mfma_pairs<1>(p[n], pairs, odd);
          if constexpr (kExact) {
            even = mfma_pairs<0>(rest[n], pairs, even);
            odd = mfma_pairs<1>(rest[n], pairs, odd);
          }
        }
      };
      columns(std::integral_constant<int, 0>{});
      if (bytes > 1) columns(std::integral_constant<int, 1>{});
      if (bytes > 2) {
        columns(std::integral_constant<int, 2>{});
        columns(std::integral_constant<int, 3>{});
      }
    }
  };

  const int turns = step1 > step0 + wave ? (step1 - step0 - wave + 3) / 4 : 0;  // steps of this wave
  if (turns > 0) {
    int at = -1, ahead = 0;  // steps whose loads have been issued
    auto fetch = [&]() {
      if (ahead >= turns) return;
      const int step = step0 + wave + 4 * ahead;
      if ((at = (at + 1) & 31) == 0) look_up(step);
      load(step, at, ahead % Step::kDepth);
      ++ahead;
    };
#pragma unroll
    for (int i = 0; i < Step::kDepth - 1; ++i) fetch();
    for (int i = 0; i < turns; ++i) {
      fetch();
      const int left = ahead - i - 1;
      if (Step::kDepth > 2 && left >= 2) wait_loads<2 * Step::kLoads>();
      else if (left >= 1) wait_loads<Step::kLoads>();
      else wait_loads<0>();
      compute(step0 + wave + 4 * i, i % Step::kDepth);
    }
  }

  // The waves' parts, one tile of 16 rows after the other, in order.
  int thread = threadIdx.x;
  asm volatile("" : "+v"(thread));
  float(*share)[16][kPad] = reinterpret_cast<float(*)[16][kPad]>(memory);
  const Slots slots = slots_of(a.partial, parts, kTileRows, kD);
  const int64_t slot = 2 * (int64_t)blockIdx.x + begins;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] = sum_of_groups(l[n]);
    if constexpr (!kExact) {  // the results by the rounded weights; with others' by the weights as they are
      rounded[n] = sum_of_groups(rounded[n]);
      const float ratio = l[n] == 0.0f ? 1.0f : l[n] / rounded[n];
      f32x4 of_row;
#pragma unroll
      for (int r = 0; r < 4; ++r) of_row[r] = __shfl(ratio, 4 * g + r);
#pragma unroll
      for (int i = 0; i < kAcc; ++i) acc[n][i] *= of_row;
    }
    __syncthreads();
    if (g == 0) {
      stat[wave][c16][0] = m[n];
      stat[wave][c16][1] = l[n];
    }
    uint32_t nan_blocks[4];  // of the accumulators' rows
#pragma unroll
    for (int r = 0; r < 4; ++r) nan_blocks[r] = __shfl(poison[n], 4 * g + r);
#pragma unroll
    for (int i = 0; i < kAcc; ++i) {
      const bool word = i < Step::kWords * 8, half = !word && i < Step::kWords * 8 + Step::kHalf * 4;
      const int wide = word ? 8 : half ? 4 : 2;
      const int first = word ? i / 8 * 128 : Step::kWords * 128 + (half ? 0 : Step::kHalf * 64);
      const int in = word ? i % 8 : half ? i - Step::kWords * 8 : i - Step::kWords * 8 - Step::kHalf * 4;
      const int blk = first / 32 + (word ? c16 >> 2 : half ? c16 >> 3 : 0);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        share[wave][4 * g + r][first + c16 * wide + in] = nan_blocks[r] >> blk & 1 ? __uint_as_float(0x7fc00000u) : acc[n][i][r];
    }
    __syncthreads();
    // a row's 8 columns per thread
    for (int u = thread; u < 16 * kD / 8; u += 256) {
      const int rr = u / (kD / 8), col = (u - rr * (kD / 8)) * 8;
      const int r = t.row0 + n * 16 + rr;
      if (r >= t.rows) continue;
      float top = stat[0][rr][0];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, stat[w][rr][0]);
      const float less = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(stat[w][rr][0] - less);
        const float lw = stat[w][rr][1];
        if (lw == 0.0f) continue;  // nothing seen, or weights of 0 only
        sum += f * lw;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += f * share[w][rr][col + i];
      }
      const int tok = (int)((uint32_t)r / (uint32_t)a.group), gh = r - tok * a.group;
      const int64_t token = t.first_token + tok, head = (int64_t)kvh_now * a.group + gh;
      const int64_t row = token * a.q_heads + head;
      const Sees s = sees(a, t.len, t.pos(tok), cap);
      const bool sees_some = s.hi > s.lo;
      if (begins && !whole && col == 0) {  // the first workgroup, and how many share the item
        const int owners = shared ? (int)quotient(item_at - begin + each - 1, chunk) + 1 : 0;
        slots.of_row[row] = {(int)blockIdx.x, owners << 8 | (n * 16 + rr)};
      }
      if (shared) {
        const int64_t place = slot * kTileRows + n * 16 + rr;
        float* p = slots.values + place * kD + col;
#pragma unroll
        for (int i = 0; i < 8; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
        if (col == 0) slots.stats[place] = {top, sees_some ? sum : -1.0f};  // below 0: the row sees no key at all
      } else {
        // no key: 0; keys of weight 0 only (all scores -infinity): 0 / 0
        const float inv = sees_some ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = sees_some ? o[i] * inv : 0.0f;
        store8(a.out + token * a.out_token + head * a.out_head + col, o);
        if (a.lse && col == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
      }
    }
  }
  __syncthreads();  // the parts have been read: their place is the rings' again
  }
}

// ------------------------------------------------------------ many rows
// A workgroup takes 128 rows, 32 to a wave, and 64 keys at a time.  K's and V's
// codes are widened once for its four waves: each wave widens a quarter of the
// next 64 keys, straight from memory into the fragments of the 32 x 32 x 16
// instruction, and writes them to LDS as they are read, 16 bytes a lane one
// after the other, while the products of the present 64 keys run.
// 4 x 2048 over 8192, 32/8 x 128: 656 to 680 us, 900 to 930 TFLOP/s.  The matrix
// units are busy 38% of the time, the vector units 52 to 61% (a third of it the
// exponentials), LDS half; two waves a SIMD, one with products and one with
// vector work, take 1.5 times as long as the longer of them alone.
// 256 rows a workgroup, four of its eight waves widening K and four V, halve the
// widening and are no faster (717 us next to 690 in one session), nor is a higher
// priority while products run (714).
// Of kAll products and the reads of LDS that they need, in this order: kAhead reads,
// then one after every product.  (Left alone, the reads come one or two ahead, and
// each product waits: 4 x 2048 over 8192, 32/8 x 128: 1% more; 2 x 1024 over 4096
// with d = 256: 7%, and 6 ahead 4%.)
template <int kAll, int kAhead>
__device__ __forceinline__ void read_ahead() {
  constexpr int ahead = kAhead < kAll ? kAhead : kAll;
  __builtin_amdgcn_sched_group_barrier(0x100, ahead, 0);
#pragma unroll
  for (int i = 0; i < kAll - ahead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, ahead, 0);
}

template <int ND>
struct Quarter4 {
  static constexpr int kScales = ND % 4 == 0 ? ND / 4 : ND <= 2 ? 1 : ND;  // of a lane's ND words of K
  static constexpr int kFours = ND / 4, kTwo = (ND >> 1) & 1, kOne = ND & 1;  // how V's columns go to 32 lanes
  uint32_t k[ND], ks[kScales];
  uint32_t v[8][kFours + kTwo + kOne];
  uint32_t vs[2][ND];
  bool k_lost, v_lost;  // the page is missing (looked at when the loads are there: not to wait for them before)
};

template <int ND>
__global__ __launch_bounds__(256, ND <= 4 ? 2 : 1) void kv4_prompt_kernel(Attn4Args a, int splits, int64_t unit0,
                                                                          int64_t tiles) {
  using Q4 = Quarter4<ND>;
  constexpr int kRow = ND * 16, kRows = 128, kFrag = 1024, kSide = 4 * ND * kFrag;
  __shared__ __attribute__((aligned(16))) uint8_t frags[2][2 * kSide];  // K, V
  __shared__ uint32_t nan_any[2][4], nan_blocks[2][64];
  const int lane = threadIdx.x & 63, c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the last rows of a sequence, which see most keys, first
  const int64_t unit = unit0 + blockIdx.x, rest = unit / splits, tile = tiles - 1 - rest / a.cache.heads;
  const int split = (int)(unit - rest * splits), kvh = (int)(rest % a.cache.heads);
  TileRows t;
  if (!tile_rows(a, tile, kRows, &t)) return;
  const int ps_log2 = a.cache.page_log2;
  const int64_t cap = (int64_t)a.plan.width << ps_log2;
  const KeyRange keys = key_range<64>(a, t, kRows, cap, split, splits, 1);

  // this lane's row: its queries, its keys
  const int r = t.row0 + wave * 32 + c32;
  const bool has = r < t.rows;
  const int tok = has ? (int)((uint32_t)r / (uint32_t)a.group) : 0, gh = has ? r - tok * a.group : 0;
  const Sees my = has ? sees(a, t.len, t.pos(tok), cap) : Sees{0, 0};
  int hi_min = has ? my.hi : keys.hi, lo_max = has ? my.lo : keys.lo, hi_max = my.hi;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    hi_min = min(hi_min, __shfl_xor(hi_min, o));
    lo_max = max(lo_max, __shfl_xor(lo_max, o));
    hi_max = max(hi_max, __shfl_xor(hi_max, o));
  }
  hi_min = __builtin_amdgcn_readfirstlane(hi_min);
  lo_max = __builtin_amdgcn_readfirstlane(lo_max);
  hi_max = __builtin_amdgcn_readfirstlane(hi_max);
  bf16x8_t q[2 * ND];
  {
    const uint16_t* p = a.q + (int64_t)(t.first_token + tok) * a.q_token + (int64_t)(kvh * a.group + gh) * a.q_head;
#pragma unroll
    for (int s = 0; s < 2 * ND; ++s) {
      Raw8<uint16_t> w;
      w.fill(0);
      if (has) w.load(p + (s / ND * 2 + h) * 8 * ND + s % ND * 8, 8);
      q[s] = as_frag(w.w);
    }
  }

  f32x16 acc[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int x = 0; x < 16; ++x) acc[i][x] = 0.0f;
  float m = -INFINITY, l = 0.0f, rounded = 0.0f;  // sums of the weights, as they are and as V's product takes them
  uint32_t poison = 0;
  const float to_log2 = a.scale * kLog2e;

  // Pages of 16 steps, four to a step, in the lanes.
  int pages = -1;
  auto look_up = [&](int step) {
    const int64_t key = (int64_t)keys.base + (int64_t)step * 64 + lane * 16;
    pages = key < keys.hi ? page_of(a.cache, a.plan, t.seq, key >> ps_log2) : -1;
  };
  auto load = [&](Q4& w, int step, int at) {
    const uint32_t key0 = (uint32_t)keys.base + (uint32_t)step * 64, in_mask = (1u << ps_log2) - 1;
    {  // K: keys 32 (wave / 2) .., a quarter of each row's ND words by lane half and wave
      const int sub = (wave & 2) + (c32 >> 4);
      const int page = __shfl(pages, 4 * at + sub);
      const int64_t pg = page < 0 ? 0 : page;
      const int64_t row = ((int64_t)kvh << ps_log2) + ((key0 + sub * 16) & in_mask) + (c32 & 15);
      const uint8_t* p = a.cache.k.codes + pg * a.cache.k.codes_page + row * kRow + ((wave & 1) * 2 + h) * 4 * ND;
      if constexpr (ND % 4 == 0) {
#pragma unroll
        for (int i = 0; i < ND; i += 4) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(p + 4 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) w.k[i + j] = x[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < ND; ++i) w.k[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
      w.k_lost = page < 0;
      const uint8_t* e = a.cache.k.scales + pg * a.cache.k.scales_page + row * ND;
#pragma unroll
      for (int i = 0; i < Q4::kScales; ++i) {
        const int word = ((wave & 1) * 2 + h) * ND + i * (ND / Q4::kScales);
        w.ks[i] = e[word / 4];
      }
    }
    {  // V: 16 keys, all columns
      const int page = __builtin_amdgcn_readlane(pages, 4 * at + wave);
      const int64_t pg = page < 0 ? 0 : page;
      const int64_t row = ((int64_t)kvh << ps_log2) + ((key0 + wave * 16) & in_mask);
      w.v_lost = page < 0;
      const auto vc = common(a.cache.v.codes + pg * a.cache.v.codes_page + row * kRow);
      const auto vs = common(a.cache.v.scales + pg * a.cache.v.scales_page + row * ND);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int in = (i >> 2) * 8 + (i & 3);
        const uint32_t at_row = 4 * h * kRow;
#pragma unroll
        for (int j = 0; j < Q4::kFours; ++j) w.v[i][j] = load_at<uint16_t>(vc, at_row + 2 * c32, in * kRow + 64 * j);
        if constexpr (Q4::kTwo) w.v[i][Q4::kFours] = load_at<uint8_t>(vc, at_row + c32, in * kRow + 64 * Q4::kFours);
        if constexpr (Q4::kOne)
          w.v[i][Q4::kFours + Q4::kTwo] = load_at<uint8_t>(vc, at_row + (c32 >> 1), in * kRow + kRow - 16);
      }
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        w.vs[0][i] = load_at<uint32_t>(vs, 4 * h * ND, 4 * i);
        w.vs[1][i] = load_at<uint32_t>(vs, 4 * h * ND, 8 * ND + 4 * i);
      }
    }
  };
  auto put = [&](int buf, int frag, const uint32_t (&w)[4]) {
    *reinterpret_cast<u32x4*>(&frags[buf][frag * kFrag + lane * 16]) = u32x4{w[0], w[1], w[2], w[3]};
  };
  auto widen = [&](Q4& w, int step, int buf) {
    if (__any(w.k_lost)) {
      asm volatile("");  // (a branch)
#pragma unroll
      for (int i = 0; i < Q4::kScales; ++i) w.ks[i] = w.k_lost ? 255u : w.ks[i];  // no page: NaN
    }
    if (w.v_lost) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < ND; ++i) w.vs[0][i] = w.vs[1][i] = 0;  // another page's: nothing that is not finite
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const uint32_t e = w.ks[i / (ND / Q4::kScales)] << 23;
      const uint32_t f[4] = {widen4<0>(w.k[i], e), widen4<1>(w.k[i], e), widen4<2>(w.k[i], e), widen4<3>(w.k[i], e)};
      put(buf, wave * ND + i, f);  // key tile wave / 2, step (wave % 2) ND + i of its columns
    }
    const int k0 = (int)((uint32_t)keys.base + (uint32_t)step * 64) + wave * 16;
    const bool edge = k0 < keys.lo || (uint32_t)k0 + 16 > (uint32_t)keys.hi;
    uint32_t some_nan = 0;
#pragma unroll
    for (int part = 0; part < Q4::kFours + Q4::kTwo + Q4::kOne; ++part) {
      const bool four = part < Q4::kFours, two = !four && part == Q4::kFours && Q4::kTwo;
      const int tile0 = four ? part * 4 : Q4::kFours * 4 + (two ? 0 : Q4::kTwo * 2);
      const int blk = four ? c32 >> 3 : two ? c32 >> 4 : 0;
      uint32_t e[8], most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = four  ? scale_of<ND, 4>(w.vs[i >> 2], i & 3, tile0, blk)
               : two ? scale_of<ND, 2>(w.vs[i >> 2], i & 3, tile0, blk)
                     : scale_of<ND, 1>(w.vs[i >> 2], i & 3, tile0, blk);
        most = max(most, e[i]);
      }
      if (edge) {  // what lies outside may hold anything
        asm volatile("");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = k0 + (i >> 2) * 8 + 4 * h + (i & 3);
          e[i] = j >= keys.lo && j < keys.hi ? e[i] : 0;
        }
      }
      if (__any(most >= kNanScale)) {  // such a block counts as 0, and is noted for the rows that see it
        uint32_t nan_keys = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e[i] >= kNanScale) {
            nan_keys |= 1u << i;
            e[i] = 0;
          }
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const uint32_t who = (uint32_t)(__ballot(nan_keys >> (i & 7) & 1) >> (32 * (i >> 3)));
          uint32_t blocks = who ? 1 : 0;
          if (four)
            blocks = (who & 0xff ? 1 : 0) | (who & 0xff00 ? 2 : 0) | (who & 0xff0000 ? 4 : 0) | (who & 0xff000000u ? 8 : 0);
          else if (two) blocks = (who & 0xffff ? 1 : 0) | (who & 0xffff0000u ? 2 : 0);
          uint32_t* to = &nan_blocks[buf][wave * 16 + ((i & 7) >> 2) * 8 + 4 * (i >> 3) + (i & 3)];
          if (lane == 0) *to = (some_nan ? *to : 0) | blocks << tile0;
        }
        some_nan = 1;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] >>= 1;  // into the exponent's place
      auto column = [&](auto byte_c) {
        constexpr int byte = decltype(byte_c)::value;
        uint32_t even[4], odd[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = widen4<byte>(w.v[2 * j][part], e[2 * j]);
          const uint32_t y = widen4<byte>(w.v[2 * j + 1][part], e[2 * j + 1]);
          if (four || two) {
            even[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            odd[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
          } else {  // a lane's column is one of the byte's two
            even[j] = __builtin_amdgcn_perm(y, x, c32 & 1 ? 0x07060302u : 0x05040100u);
          }
        }
        const int frag = 4 * ND + wave * ND + tile0 + 2 * byte;
        put(buf, frag, even);
        if (four || two) put(buf, frag + 1, odd);
      };
      column(std::integral_constant<int, 0>{});
      if (four) column(std::integral_constant<int, 1>{});
    }
    if (lane == 0) nan_any[buf][wave] = some_nan;
  };
  auto frag = [&](int buf, int i) {
    uint32_t w[4];
    const u32x4 x = *reinterpret_cast<const u32x4*>(&frags[buf][i * kFrag + lane * 16]);
    w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
    return as_frag(w);
  };
  auto compute = [&](int step, int buf) {
    const int k0 = (int)((uint32_t)keys.base + (uint32_t)step * 64);
    if (k0 >= hi_max) return;  // no row of this wave sees any of them
    f32x16 z[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int x = 0; x < 16; ++x) z[s][x] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 2 * ND; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        z[s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(buf, s * 2 * ND + i), q[i], z[s], 0, 0, 0);
    read_ahead<4 * ND, 4>();
    if (k0 < lo_max || (uint32_t)k0 + 64 > (uint32_t)hi_min) {
      asm volatile("");
      const int lo = my.lo - k0 - 4 * h, hi = my.hi - k0 - 4 * h;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int j = 32 * s + 8 * (x >> 2) + (x & 3);
          z[s][x] = j >= lo && j < hi ? z[s][x] : -INFINITY;
        }
    }
    float top = z[0][0];
#pragma unroll
    for (int x = 1; x < 32; ++x) top = fmaxf(top, z[x >> 4][x & 15]);
    top *= to_log2;
    if (__any(top > m + kSlack)) {
      const float now = fmaxf(m, max_of_halves(top));
      const float shrink = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= shrink;
      rounded *= shrink;
#pragma unroll
      for (int i = 0; i < ND; ++i) acc[i] *= shrink;
    }
    const float less = m == -INFINITY ? 0.0f : m;
    bf16x8_t p[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = 8 * (s & 1) + 2 * j;
        const float e0 = __builtin_amdgcn_exp2f(fmaf(z[s >> 1][x], to_log2, -less));
        const float e1 = __builtin_amdgcn_exp2f(fmaf(z[s >> 1][x + 1], to_log2, -less));
        l += e0 + e1;
        f[j] = pack_bf16x2_hw(e0, e1);
        rounded = dot_weights<0x3f803f80u>(f[j], rounded);  // 1, 1
      }
      p[s] = as_frag(f);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < ND; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(buf, 4 * ND + s * ND + i), p[s], acc[i], 0, 0, 0);
    read_ahead<4 * ND, 4>();
    const u32x4 any = *reinterpret_cast<const u32x4*>(&nan_any[buf][0]);
    if (__builtin_amdgcn_readfirstlane(any[0] | any[1] | any[2] | any[3])) {
#pragma unroll 1
      for (int j = 0; j < 64; ++j)
        if (nan_any[buf][j >> 4] && k0 + j >= my.lo && k0 + j < my.hi) poison |= nan_blocks[buf][j];
    }
  };

  if (keys.step0 < keys.step1) {
    Q4 w;
    int at = 0;
    look_up(keys.step0);
    load(w, keys.step0, 0);
    widen(w, keys.step0, 0);
    auto fetch = [&](int step) {
      if (step >= keys.step1) return;
      if (++at == 16) {
        at = 0;
        look_up(step);
      }
      load(w, step, at);
    };
    fetch(keys.step0 + 1);
    __syncthreads();
    int buf = 0;
    for (int step = keys.step0; step < keys.step1; ++step, buf ^= 1) {
      if (step + 1 < keys.step1) widen(w, step + 1, buf ^ 1);
      fetch(step + 2);
      compute(step, buf);
      __syncthreads();
    }
  }

  l = sum_of_halves(l);
  rounded = sum_of_halves(rounded);
  if (!has) return;
  const int64_t token = t.first_token + tok, head = (int64_t)kvh * a.group + gh, row = token * a.q_heads + head;
  const bool sees_some = my.hi > my.lo;
  const int64_t all_rows = (int64_t)a.tokens * a.q_heads;
  // a part's result goes by its own rounded weights, and with others by the weights as they are
  const float inv = splits > 1 ? l == 0.0f ? 1.0f : l / rounded : sees_some ? 1.0f / rounded : 0.0f;
  float* part_out = a.partial + ((int64_t)split * all_rows + row) * (ND * 32);
  uint16_t* out = a.out + token * a.out_token + head * a.out_head;
#pragma unroll
  for (int part = 0; part < Q4::kFours + Q4::kTwo + Q4::kOne; ++part) {
    const bool four = part < Q4::kFours, two = !four && part == Q4::kFours && Q4::kTwo;
    const int tile0 = four ? part * 4 : Q4::kFours * 4 + (two ? 0 : Q4::kTwo * 2), wide = four ? 4 : two ? 2 : 1;
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      // 4 wide columns, from tile0 32 + (8 rb + 4 h) wide on: all of one block
      const int col = tile0 * 32 + (8 * rb + 4 * h) * wide;
      const bool nan = poison >> (col >> 5) & 1;
      float o[16];
#pragma unroll
      for (int x = 0; x < 4 * wide; ++x) {
        const float y = acc[tile0 + x % wide][4 * rb + x / wide] * inv;
        o[x] = nan ? __uint_as_float(0x7fc00000u) : sees_some ? y : 0.0f;
      }
      if (splits > 1) {
#pragma unroll
        for (int x = 0; x < 4 * wide; x += 4)
          *reinterpret_cast<f32x4*>(part_out + col + x) = f32x4{o[x], o[x + 1], o[x + 2], o[x + 3]};
      } else if (wide == 1) {
#pragma unroll
        for (int x = 0; x < 4; ++x) store1(out + col + x, o[x]);
      } else {
#pragma unroll
        for (int x = 0; x < 4 * wide; x += 8) {
          const float v8[8] = {o[x], o[x + 1], o[x + 2], o[x + 3], o[x + 4], o[x + 5], o[x + 6], o[x + 7]};
          store8(out + col + x, v8);
        }
      }
    }
  }
  if (h == 0) {
    if (splits > 1) {
      float* st = a.partial + (int64_t)splits * all_rows * (ND * 32) + ((int64_t)split * all_rows + row) * 2;
      st[0] = m;
      st[1] = sees_some ? l : -1.0f;  // a row that sees no key in any part
    } else if (a.lse) {
      a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    }
  }
}

// The parts of a row, added in a fixed order.  A thread takes 4 columns of a
// row and every `slices`th part, its loads independent of one another; the
// slices are added through LDS.  stats: each part's maximum and sum.
struct Part {
  float top, sum;
  f32x4 o;
  __device__ __forceinline__ void add(float t, float l, f32x4 x) {
    if (l == 0.0f) return;  // nothing seen, or weights of 0 only
    const float now = fmaxf(top, t), less = now == -INFINITY ? 0.0f : now;
    const float f = __builtin_amdgcn_exp2f(top - less), h = __builtin_amdgcn_exp2f(t - less);
    sum = sum * f + l * h;
    o = o * f + x * h;
    top = now;
  }
};
// groups > 0: the slots of so many workgroups, tiles of tile_size rows; else
// `splits` parts of every row, [part][row].
__global__ __launch_bounds__(256) void kv4_join_kernel(Attn4Args a, int groups, int tile_size, int splits, int slices) {
  __shared__ Part share[256];
  const int64_t all_rows = (int64_t)a.tokens * a.q_heads;
  const int d = a.cache.d, lanes = d / 4, items = 256 / slices;
  const int slice = threadIdx.x / items, mine = threadIdx.x - slice * items;
  const Slots slots = slots_of(a.partial, groups, tile_size, d);
  const f32x2* stats = groups ? slots.stats : reinterpret_cast<const f32x2*>(a.partial + (int64_t)splits * all_rows * d);
  // rows behind the last sequence have no parts
  const int64_t rows = (int64_t)min(max(a.plan.starts[a.plan.sequences], 0), a.tokens) * a.q_heads;
  for (int64_t first = (int64_t)blockIdx.x * items; first < all_rows * lanes; first += (int64_t)gridDim.x * items) {
    const int64_t item = first + mine, row = item / lanes;
    const int col = 4 * (int)(item - row * lanes);
    Part p = {-INFINITY, 0.0f, {0, 0, 0, 0}};
    bool none = false;
    int parts = row < rows ? splits : 0;
    int64_t at = row, step = all_rows, second = 0;  // of part i: at + i step, less `second` from the second on
    const int2 of = groups ? slots.of_row[min(row, all_rows - 1)] : int2{0, 0};
    if (groups && row < rows) {
      // (rows of a plan that makes no sense may have no record)
      const int owner = min(max(of.x, 0), groups - 1), local = min(of.y & 255, tile_size - 1);
      parts = min(of.y >> 8, groups - owner);
      at = (2LL * owner + 1) * tile_size + local;
      step = 2LL * tile_size;
      second = tile_size;
    }
    for (int i0 = slice; i0 < parts; i0 += 8 * slices) {
      f32x2 st[8];
      f32x4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = min(i0 + i * slices, parts - 1);
        const int64_t from = at + n * step - (n > 0 ? second : 0);
        st[i] = stats[from];
        x[i] = *reinterpret_cast<const f32x4*>(a.partial + from * d + col);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i * slices < parts) {
          none |= st[i][1] < 0.0f;
          p.add(st[i][0], st[i][1], x[i]);
        }
    }
    if (slices > 1) {
      __syncthreads();  // the last items' are done with
      share[threadIdx.x] = p;
      __syncthreads();
      if (slice == 0)
        for (int i = 1; i < slices; ++i) p.add(share[i * items + mine].top, share[i * items + mine].sum, share[i * items + mine].o);
    }
    if (slice == 0 && parts > 0) {
      const int token = (int)(row / a.q_heads), head = (int)(row - (int64_t)token * a.q_heads);
      const float inv = none ? 0.0f : 1.0f / p.sum;
      if (none) p.o = f32x4{0, 0, 0, 0};
      uint16_t* out = a.out + (int64_t)token * a.out_token + (int64_t)head * a.out_head + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) store1(out + i, p.o[i] * inv);
      if (a.lse && col == 0) a.lse[row] = none || p.sum == 0.0f ? -INFINITY : (p.top + __builtin_amdgcn_logf(p.sum)) * kLn2;
    }
  }
}

constexpr int kMostSplits = 256, kUnits = 256;  // parts, compute units

// How a call is cut: tiles of 16, 32 or 128 rows, by the rows that a sequence
// has on average.  Over 4096 keys, 32/8 heads, in tiles of 16, 32 and 128:
//   rows to a key head       16             20             64             80            128       256 (4 sequences)
//   64 sequences, d = 128    76  74 112    106  76 201    194 139 209    261 208 223    309 243 289    65 46 45
//   d = 64                   45  58  97     67  60  97    128 103 114    162 131 144    220 185 201
//   d = 256                 114 167 419    180 169 619    303 380 634    428 505 642    574 600 876
// (From 65 rows to about 128, and for d = 256 from 33, another choice would gain 5 to
// 25%; beyond, the tiles of 128 win by the more the more rows there are.)
// Tiles of 16 and 32: equal parts (`groups`) for as many workgroups as have room,
// or an item to each workgroup (0) from 4 items for each such place on (256 x 1 over
// 1024 has 2.7, with one product for V: 77 us in parts, 71 in items; over 20 .. 2048: 83
// and 83, and the worse the longer one sequence is next to the others).  Tiles of 128:
// the keys in `splits` parts until the chip has work enough.
struct Cut {
  int rows, groups, splits;
  int64_t tiles;
};
Cut cut_of(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size, int64_t sequences,
           int64_t width) {
  const int64_t group = q_heads / kv_heads, rows = tokens * group, keys = width * page_size;
  Cut c{};
  c.rows = rows > 64 * sequences ? 128 : rows > 16 * sequences ? 32 : 16;
  c.tiles = rows / c.rows + sequences;
  c.splits = 1;
  // items that there are, whatever the sequences' shares of the tokens
  const int64_t items = std::max<int64_t>(1, std::max(rows / c.rows, std::min(sequences, tokens)) * kv_heads);
  if (c.rows < 128) {
    const int64_t room = kUnits * room_for((int)d / 32, c.rows / 16);
    // steps, if every sequence fills the table; a million of one item are more than enough parts (and the product of all
    // sizes at their ends is more than 63 bits)
    const int64_t most = c.tiles * kv_heads * (std::min<int64_t>((keys + 31) / 32, 1 << 20) + 2 + kItemSteps);
    if (items < 4 * room) c.groups = (int)std::min(room, (most + kLeastSteps - 1) / kLeastSteps);
  } else {
    const int64_t most = std::max<int64_t>(1, (keys + 127) / 128);
    c.splits = (int)std::min({most, (512 + items - 1) / items, (int64_t)kMostSplits});
  }
  return c;
}
int64_t workspace_of(const Cut& c, int64_t rows, int64_t d) {
  if (c.groups) return (2LL * c.groups * c.rows * (d + 2) + 2 * rows) * 4;
  return c.splits == 1 ? 0 : rows * c.splits * (d + 2) * 4;
}

template <int ND>
hipError_t go(const Attn4Args& a, const Cut& c, hipStream_t stream) {
  constexpr int64_t kMost = 1 << 23;  // workgroups of a launch: 2^32 threads are refused
  const int64_t rows = (int64_t)a.tokens * a.q_heads;
  const int64_t units = c.groups ? c.groups : c.tiles * a.cache.heads * c.splits;
  for (int64_t u = 0; u < units; u += kMost) {
    const dim3 grid((unsigned)std::min(kMost, units - u));
    if (c.rows == 16) hipLaunchKernelGGL((kv4_attention_kernel<ND, 1>), grid, dim3(256), 0, stream, a, c.groups, u);
    else if (c.rows == 32) hipLaunchKernelGGL((kv4_attention_kernel<ND, 2>), grid, dim3(256), 0, stream, a, c.groups, u);
    else hipLaunchKernelGGL((kv4_prompt_kernel<ND>), grid, dim3(256), 0, stream, a, c.splits, u, c.tiles);
  }
  if (!c.groups && c.splits == 1) return hipGetLastError();
  // parts that a row has, if all are alike
  const int64_t parts =
      c.groups ? c.groups / std::max<int64_t>(1, (int64_t)std::min(a.tokens, a.plan.sequences) * a.cache.heads) : c.splits;
  int slices = 1;
  while (slices < 32 && slices * 8 < parts) slices *= 2;
  const int64_t items = rows * (ND * 8), per = 256 / slices;
  hipLaunchKernelGGL(kv4_join_kernel, dim3((unsigned)std::min((items + per - 1) / per, kMost)), dim3(256), 0, stream, a,
                     c.groups, c.rows, c.splits, slices);
  return hipGetLastError();
}

}  // namespace

int64_t kv4_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size,
                                int64_t sequences, int64_t width) {
  if (tokens == 0 || sequences == 0) return 0;
  return workspace_of(cut_of(tokens, q_heads, kv_heads, d, page_size, sequences, width), tokens * q_heads, d);
}

hipError_t launch_kv4_attention(const Attn4Args& a, hipStream_t stream) {
  const Cut c = cut_of(a.tokens, a.q_heads, a.cache.heads, a.cache.d, 1LL << a.cache.page_log2, a.plan.sequences,
                       a.plan.width);
  switch (a.cache.d / 32) {
    case 1: return go<1>(a, c, stream);
    case 2: return go<2>(a, c, stream);
    case 3: return go<3>(a, c, stream);
    case 4: return go<4>(a, c, stream);
    case 5: return go<5>(a, c, stream);
    case 6: return go<6>(a, c, stream);
    case 7: return go<7>(a, c, stream);
    default: return go<8>(a, c, stream);
  }
}

}  // namespace harp
