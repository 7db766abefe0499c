// Attention over a cache in 4 bits.
//
// For one key head, the rows of a sequence are its call's tokens times the
// query heads that share the key head.  With S = K Q^T (keys by rows) and
// O^T = V^T P^T, the matrix instructions' layouts fit one another: what a lane
// holds of S, for one row of Q and its keys, is what it has to give of P, and
// both products have a lane's row of Q in common, so the softmax needs no
// exchange but the maximum.  The order of keys within a step is free; it is
// the one in which S comes out.
//
// K's and V's codes become bf16 exactly (E2M1 times a power of two) by one
// conversion instruction for two values, scale included.  A lane's piece of K
// is as it is in memory; V has to be transposed: a lane takes the same columns
// of 8 keys and pairs them by byte permutations.
//
// Scores, maxima, sums and accumulators are fp32.  The weights are rounded to
// bf16 for the product with V: each is off by at most 2^-9 of itself, the result
// by about as much as its own rounding to bf16 adds.
#include <algorithm>
#include <cmath>

#include "kv4.h"
#include "q8.h"

namespace harp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ bf16x8_t as_frag(const uint32_t (&w)[4]) {
  bf16x8_t r;
  __builtin_memcpy(&r, w, 16);
  return r;
}
__device__ __forceinline__ f32x4 mfma16(const bf16x8_t& a, const bf16x8_t& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// Byte kByte's two codes, times 2^(e - 127), e in the exponent's place.
template <int kByte>
__device__ __forceinline__ uint32_t widen4(uint32_t codes, uint32_t e) {
  const bf16x2_t v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __uint_as_float(e), kByte);
  uint32_t w;
  __builtin_memcpy(&w, &v, 4);
  return w;
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
  int64_t row0, rows;                 // the tile's first row; the sequence's
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
  t->rows = (int64_t)t->tokens * a.group;
  t->row0 = (tile - first(b)) * tile_size;
  return t->row0 >= 0 && t->row0 < t->rows;
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
  const int64_t row1 = min(t.row0 + tile_size, t.rows);
  const int tok0 = (int)(t.row0 / a.group), tok1 = (int)((row1 - 1) / a.group);
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
constexpr uint32_t kNanScale = 0xff000000u;  // of such words, and above

// Weights go by a reference that a score may pass by this much (in powers of
// two) before the sums are brought to a new one, which is then rarely needed.
constexpr float kSlack = 8.0f;

// ------------------------------------------------------------- few rows
// A wave takes 32 keys at a time, every fourth 32 of its workgroup's part.  Its
// loads go straight into a ring of its own in LDS, kDepth - 1 steps ahead: what
// keeps HBM busy is bytes in flight, and registers are too few for them (one
// step ahead in registers, three waves a SIMD: 5.2 TB/s at 64 x 16384 tokens of
// 8 x 128).  No barrier is needed: a wave reads what it loaded itself.
//
// A step in LDS, of two halves of 16 keys each (their pages may differ):
//   K   ND % 4 == 0: as the lanes take it, 16 bytes each, one after the other;
//       else the rows as they are
//   V   by parts of the columns.  Lane c of 16 has the columns 8 c .. of a part
//       of 128 (a word of a row), 4 c .. of one of 64 (a half), 2 c .. of one of
//       32 (a byte).  Of four keys 4 g + i, i outermost, so that a wave's words
//       are consecutive.
//   scales of K, of V: rows as they are
template <int ND>
struct Step4 {
  static constexpr int kUnit = ND % 4 == 0 ? 4 : ND % 2 == 0 ? 2 : 1;  // words of K that a lane takes at once
  static constexpr int kWords = ND / 4, kHalf = (ND >> 1) & 1, kByte = ND & 1;
  static constexpr int kSide = 256 * ND;                     // 16 keys' codes
  static constexpr int kV = 2 * kSide, kScales = 4 * kSide;  // where they begin
  static constexpr int kBytes = 4 * kSide + 64 * ND;
  static constexpr int kScaleLoads = (ND + 3) / 4;
  static constexpr int kLoads = 2 * ((ND + 3) / 4) + 2 * (kWords + kHalf + kByte) + kScaleLoads;
  static constexpr int kDepth = ND <= 4 ? 3 : 2;
};

// Waits until at most kLeft of the wave's loads are under way.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kLeft) : "memory");
}
__device__ __forceinline__ void load_lds4(uint64_t from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(from)
               : "memory");
}

// Workgroups a compute unit is to have room for, which bounds the registers.
constexpr int room_for(int nd, int nq) { return nd <= 4 && (nq == 1 || nd <= 2) ? 3 : nd * nq <= 10 ? 2 : 1; }

template <int ND, int NQ>
__global__ __launch_bounds__(256, room_for(ND, NQ)) void kv4_attention_kernel(Attn4Args a, int splits, int64_t unit0) {
  using Step = Step4<ND>;
  constexpr int kRow = ND * 16, kTileRows = 16 * NQ, kAcc = 2 * ND, kD = ND * 32;
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // one workgroup: a part of the keys of a key head of a tile of rows
  const int64_t unit = unit0 + blockIdx.x, rest = unit / splits, tile = rest / a.cache.heads;
  const int split = (int)(unit - rest * splits), kvh = (int)(rest - tile * a.cache.heads);
  TileRows t;
  if (!tile_rows(a, tile, kTileRows, &t)) return;
  const int ps_log2 = a.cache.page_log2;
  const int64_t cap = (int64_t)a.plan.width << ps_log2;
  const KeyRange keys = key_range<32>(a, t, kTileRows, cap, split, splits, 4);
  const int hi_all = keys.hi, lo_all = keys.lo, base = keys.base, step0 = keys.step0, step1 = keys.step1;

  // this lane's row of each tile of 16: its queries, its keys
  Sees row_sees[NQ];
  bf16x8_t q[NQ][ND];
  int hi_min = hi_all, lo_max = lo_all;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = t.row0 + n * 16 + c16;
    const bool has = r < t.rows;
    const int tok = has ? (int)(r / a.group) : 0, gh = has ? (int)(r - (int64_t)tok * a.group) : 0;
    row_sees[n] = has ? sees(a, t.len, t.pos(tok), cap) : Sees{0, 0};
    if (has) {
      hi_min = min(hi_min, row_sees[n].hi);
      lo_max = max(lo_max, row_sees[n].lo);
    }
    const uint16_t* p = a.q + (int64_t)(t.first_token + tok) * a.q_token + (int64_t)(kvh * a.group + gh) * a.q_head;
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
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[n][i] = f32x4{0, 0, 0, 0};
  }
  const float to_log2 = a.scale * kLog2e;

  // the rings of the four waves; at the end what they have to add
  constexpr int kPad = kD + 4, kRing = Step::kBytes * Step::kDepth, kShare = 16 * kPad * 4;
  __shared__ __attribute__((aligned(16))) uint8_t memory[4 * (kRing > kShare ? kRing : kShare)];
  __shared__ float stat[4][16][2];
  const uint8_t* ring = memory + wave * kRing;
  const uint32_t ring_at = lds_address(ring);

  // Pages of this wave's next 32 steps, two to a step, in the lanes.
  int pages = -1;
  auto look_up = [&](int step) {
    const int64_t key = (int64_t)base + ((int64_t)step + (lane >> 1) * 4) * 32 + (lane & 1) * 16;
    pages = key < hi_all ? page_of(a.cache, a.plan, t.seq, key >> ps_log2) : -1;
  };
  // the lane's scales: of K or V, of which half, which word of the 4 ND
  uint64_t scales_at[Step::kScaleLoads];
#pragma unroll
  for (int n = 0; n < Step::kScaleLoads; ++n) {
    const int w = 64 * n + lane;
    scales_at[n] = reinterpret_cast<uint64_t>(w < 8 * ND ? a.cache.k.scales : a.cache.v.scales) +
                   (uint64_t)((((int64_t)kvh << ps_log2) * ND) + w % (4 * ND) * 4);
  }
  uint32_t lost = 0;  // slot by slot, two bits: keys without a page
  auto load = [&](int step, int at, int slot) {
    const uint32_t to = ring_at + slot * Step::kBytes;
    int64_t k_scales[2], v_scales[2];
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // the slot's last step has been read
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int page = __builtin_amdgcn_readlane(pages, 2 * at + s);
      const uint32_t key = (uint32_t)base + (uint32_t)step * 32 + s * 16;
      const uint32_t in_page = key & ((1u << ps_log2) - 1);
      const int64_t row = ((int64_t)kvh << ps_log2) + in_page, pg = page < 0 ? 0 : page;
      const uint32_t bit = 1u << (2 * slot + s);
      lost = page < 0 ? lost | bit : lost & ~bit;
      const TileSrc k = tile_src(a.cache.k.codes + pg * a.cache.k.codes_page + row * kRow, 16 * kRow);
      const TileSrc v = tile_src(a.cache.v.codes + pg * a.cache.v.codes_page + row * kRow, 16 * kRow);
      k_scales[s] = pg * a.cache.k.scales_page + (int64_t)in_page * ND;
      v_scales[s] = pg * a.cache.v.scales_page + (int64_t)in_page * ND;
#pragma unroll
      for (int u = 0; u < (ND + 3) / 4; ++u) {
        const uint32_t off = ND % 4 == 0 ? c16 * kRow + g * 16 + u * 64 : lane * 16 + u * 1024;
        if (ND % 4 == 0 || lane < 16 * ND - 64 * u) load_lds16(k, to + s * Step::kSide + u * 1024, off, 0);
      }
      const uint32_t v_to = to + Step::kV + s * Step::kSide;
#pragma unroll
      for (int u = 0; u < Step::kWords; ++u)
        load_lds16(v, v_to + u * 1024, (4 * ((lane >> 2) & 3) + (lane >> 4)) * kRow + (lane & 3) * 16 + u * 64, 0);
      if constexpr (Step::kHalf)
        if (lane < 32)
          load_lds16(v, v_to + Step::kWords * 1024, (4 * ((lane >> 1) & 3) + (lane >> 3)) * kRow + (lane & 1) * 16 + Step::kWords * 64, 0);
      if constexpr (Step::kByte)
        if (lane < 16)
          load_lds16(v, v_to + Step::kWords * 1024 + Step::kHalf * 512, (4 * (lane & 3) + (lane >> 2)) * kRow + kRow - 16, 0);
    }
#pragma unroll
    for (int n = 0; n < Step::kScaleLoads; ++n) {
      const int w = 64 * n + lane;
      const bool second = w / (4 * ND) & 1;
      const int64_t off = w < 8 * ND ? second ? k_scales[1] : k_scales[0] : second ? v_scales[1] : v_scales[0];
      if (w < 16 * ND) load_lds4(scales_at[n] + (uint64_t)off, to + Step::kScales + 256 * n);
    }
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
        if (missing >> s & 1) e[s] = 255u << 23;  // no page: NaN
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
    if (k0 < lo_max || k0 + 32 > hi_min) {  // some row does not see all of these keys
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
    bf16x8_t p[NQ];
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
#pragma unroll
        for (int i = 0; i < kAcc; ++i) acc[n][i] *= shrink;
      }
      const float less = m[n] == -INFINITY ? 0.0f : m[n];
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(fmaf(z[n][i >> 2][i & 3], to_log2, -less));
        l[n] += e[i];
      }
      const uint32_t f[4] = {pack_bf16x2_hw(e[0], e[1]), pack_bf16x2_hw(e[2], e[3]), pack_bf16x2_hw(e[4], e[5]),
                             pack_bf16x2_hw(e[6], e[7])};
      p[n] = as_frag(f);
    }
    // V's columns by parts: 8 columns to a lane (words), 4 (halves), 2 (bytes)
    const bool edge = k0 < lo_all || k0 + 32 > hi_all;
    uint32_t vs[2][ND];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        vs[s][i] = reinterpret_cast<const uint32_t*>(in + Step::kScales + (32 + 16 * s + 4 * g) * ND)[i];
        if (missing >> s & 1) vs[s][i] = 0;  // another page's: nothing that is not finite
      }
#pragma unroll
    for (int part = 0; part < Step::kWords + Step::kHalf + Step::kByte; ++part) {
      const bool word = part < Step::kWords, half = !word && part == Step::kWords && Step::kHalf;
      const int bytes = word ? 4 : half ? 2 : 1;
      const int tile0 = word ? part * 8 : Step::kWords * 8 + (half ? 0 : Step::kHalf * 4);
      const int blk0 = word ? part * 4 : half ? Step::kWords * 4 : ND - 1;
      const int blk = word ? c16 >> 2 : half ? c16 >> 3 : 0;
      // the scale of the lane's block, one byte of the four keys' scales, as a number's highest byte
      uint32_t e[8], most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = word   ? scale_of<ND, 4>(vs[i >> 2], i & 3, blk0, blk)
               : half ? scale_of<ND, 2>(vs[i >> 2], i & 3, blk0, blk)
                      : scale_of<ND, 1>(vs[i >> 2], i & 3, blk0, blk);
        most = max(most, e[i]);
      }
      if (edge) {  // what lies outside may hold anything
        asm volatile("");
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = k0 + 16 * (i >> 2) + 4 * g + (i & 3);
          e[i] = j >= lo_all && j < hi_all ? e[i] : 0;
        }
      }
      if (__any(most >= kNanScale)) {
        // NaN times a weight of 0 would reach rows that do not see the key: such a block counts as 0, and is noted for
        // the rows that do see it
        uint32_t nan_keys = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e[i] >= kNanScale) {
            nan_keys |= 1u << i;
            e[i] = 0;
          }
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
          const uint32_t who = (uint32_t)(__ballot(nan_keys >> (i & 7) & 1) >> (16 * (i >> 3))) & 0xffff;
          if (who == 0) continue;
          const int j = k0 + 16 * ((i & 7) >> 2) + 4 * (i >> 3) + (i & 3);
          uint32_t blocks = who ? 1 : 0;
          if (word)
            blocks = (who & 0xf ? 1 : 0) | (who & 0xf0 ? 2 : 0) | (who & 0xf00 ? 4 : 0) | (who & 0xf000 ? 8 : 0);
          else if (half) blocks = (who & 0xff ? 1 : 0) | (who & 0xff00 ? 2 : 0);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            if (j >= row_sees[n].lo && j < row_sees[n].hi) poison[n] |= blocks << blk0;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] >>= 1;  // into the exponent's place
      uint32_t vw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint8_t* v = in + Step::kV + (i >> 2) * Step::kSide;
        if (word) vw[i] = *reinterpret_cast<const uint32_t*>(v + part * 1024 + (i & 3) * 256 + lane * 4);
        else if (half) vw[i] = *reinterpret_cast<const uint16_t*>(v + Step::kWords * 1024 + (i & 3) * 128 + lane * 2);
        else vw[i] = v[Step::kWords * 1024 + Step::kHalf * 512 + (i & 3) * 64 + lane];
      }
      auto column = [&](auto byte_c) {
        constexpr int byte = decltype(byte_c)::value;
        uint32_t even[4], odd[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = widen4<byte>(vw[2 * j], e[2 * j]);
          const uint32_t y = widen4<byte>(vw[2 * j + 1], e[2 * j + 1]);
          even[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          odd[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          acc[n][tile0 + 2 * byte] = mfma16(as_frag(even), p[n], acc[n][tile0 + 2 * byte]);
          acc[n][tile0 + 2 * byte + 1] = mfma16(as_frag(odd), p[n], acc[n][tile0 + 2 * byte + 1]);
        }
      };
      column(std::integral_constant<int, 0>{});
      if (bytes > 1) column(std::integral_constant<int, 1>{});
      if (bytes > 2) {
        column(std::integral_constant<int, 2>{});
        column(std::integral_constant<int, 3>{});
      }
    }
  };

  const int mine = step1 > step0 + wave ? (step1 - step0 - wave + 3) / 4 : 0;  // steps of this wave
  if (mine > 0) {
    int at = -1, ahead = 0;  // steps whose loads have been issued
    auto fetch = [&]() {
      if (ahead >= mine) return;
      const int step = step0 + wave + 4 * ahead;
      if ((at = (at + 1) & 31) == 0) look_up(step);
      load(step, at, ahead % Step::kDepth);
      ++ahead;
    };
#pragma unroll
    for (int i = 0; i < Step::kDepth - 1; ++i) fetch();
    for (int i = 0; i < mine; ++i) {
      fetch();
      const int left = ahead - i - 1;
      if (Step::kDepth > 2 && left >= 2) wait_loads<2 * Step::kLoads>();
      else if (left >= 1) wait_loads<Step::kLoads>();
      else wait_loads<0>();
      compute(step0 + wave + 4 * i, i % Step::kDepth);
    }
  }

  // The waves' parts, one tile of 16 rows after the other, in order.
  float(*share)[16][kPad] = reinterpret_cast<float(*)[16][kPad]>(memory);
  const int64_t all_rows = (int64_t)a.tokens * a.q_heads;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] = sum_of_groups(l[n]);
    __syncthreads();
    if (g == 0) {
      stat[wave][c16][0] = m[n];
      stat[wave][c16][1] = l[n];
    }
#pragma unroll
    for (int i = 0; i < kAcc; ++i) {
      const bool word = i < Step::kWords * 8, half = !word && i < Step::kWords * 8 + Step::kHalf * 4;
      const int wide = word ? 8 : half ? 4 : 2;
      const int first = word ? i / 8 * 128 : Step::kWords * 128 + (half ? 0 : Step::kHalf * 64);
      const int in = word ? i % 8 : half ? i - Step::kWords * 8 : i - Step::kWords * 8 - Step::kHalf * 4;
      const int blk = first / 32 + (word ? g : half ? g >> 1 : 0);  // of the lane's four values
      const bool nan = poison[n] >> blk & 1;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        share[wave][c16][first + (4 * g + r) * wide + in] = nan ? __uint_as_float(0x7fc00000u) : acc[n][i][r];
    }
    __syncthreads();
    // a row's 8 columns per thread
    for (int u = threadIdx.x; u < 16 * kD / 8; u += 256) {
      const int rr = u / (kD / 8), col = (u - rr * (kD / 8)) * 8;
      const int64_t r = t.row0 + n * 16 + rr;
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
      const int tok = (int)(r / a.group), gh = (int)(r - (int64_t)tok * a.group);
      const int64_t token = t.first_token + tok, head = (int64_t)kvh * a.group + gh;
      const int64_t row = token * a.q_heads + head;
      if (splits > 1) {
        float* p = a.partial + ((int64_t)split * all_rows + row) * kD + col;
#pragma unroll
        for (int i = 0; i < 8; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
        if (col == 0) {
          const Sees s = sees(a, t.len, t.pos(tok), cap);
          float* st = a.partial + (int64_t)splits * all_rows * kD + ((int64_t)split * all_rows + row) * 2;
          st[0] = top;
          st[1] = s.hi > s.lo ? sum : -1.0f;  // a row that sees no key in any part
        }
      } else {
        const Sees s = sees(a, t.len, t.pos(tok), cap);
        // no key: 0; keys of weight 0 only (all scores -infinity): 0 / 0
        const float inv = s.hi > s.lo ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = s.hi > s.lo ? o[i] * inv : 0.0f;
        store8(a.out + token * a.out_token + head * a.out_head + col, o);
        if (a.lse && col == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------ many rows
// A workgroup takes 128 rows, 32 to a wave, and 64 keys at a time.  K's and V's
// codes are widened once for its four waves: each wave widens a quarter of the
// next 64 keys, straight from memory into the fragments of the 32 x 32 x 16
// instruction, and writes them to LDS as they are read, 16 bytes a lane one
// after the other, while the products of the present 64 keys run.
template <int ND>
struct Quarter4 {
  static constexpr int kScales = ND % 4 == 0 ? ND / 4 : ND <= 2 ? 1 : ND;  // of a lane's ND words of K
  static constexpr int kFours = ND / 4, kTwo = (ND >> 1) & 1, kOne = ND & 1;  // how V's columns go to 32 lanes
  uint32_t k[ND], ks[kScales];
  uint32_t v[8][kFours + kTwo + kOne];
  uint32_t vs[2][ND];
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
  const int64_t r = t.row0 + wave * 32 + c32;
  const bool has = r < t.rows;
  const int tok = has ? (int)(r / a.group) : 0, gh = has ? (int)(r - (int64_t)tok * a.group) : 0;
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
  float m = -INFINITY, l = 0.0f;
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
      const uint8_t* e = a.cache.k.scales + pg * a.cache.k.scales_page + row * ND;
#pragma unroll
      for (int i = 0; i < Q4::kScales; ++i) {
        const int word = ((wave & 1) * 2 + h) * ND + i * (ND / Q4::kScales);
        w.ks[i] = page < 0 ? 255u : e[word / 4];  // no page: NaN
      }
    }
    {  // V: 16 keys, all columns
      const int page = __builtin_amdgcn_readlane(pages, 4 * at + wave);
      const int64_t pg = page < 0 ? 0 : page;
      const int64_t row = ((int64_t)kvh << ps_log2) + ((key0 + wave * 16) & in_mask);
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
        const uint32_t e0 = load_at<uint32_t>(vs, 4 * h * ND, 4 * i), e1 = load_at<uint32_t>(vs, 4 * h * ND, 8 * ND + 4 * i);
        w.vs[0][i] = page < 0 ? 0u : e0;  // another page's: nothing that is not finite
        w.vs[1][i] = page < 0 ? 0u : e1;
      }
    }
  };
  auto put = [&](int buf, int frag, const uint32_t (&w)[4]) {
    *reinterpret_cast<u32x4*>(&frags[buf][frag * kFrag + lane * 16]) = u32x4{w[0], w[1], w[2], w[3]};
  };
  auto widen = [&](const Q4& w, int step, int buf) {
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const uint32_t e = w.ks[i / (ND / Q4::kScales)] << 23;
      const uint32_t f[4] = {widen4<0>(w.k[i], e), widen4<1>(w.k[i], e), widen4<2>(w.k[i], e), widen4<3>(w.k[i], e)};
      put(buf, wave * ND + i, f);  // key tile wave / 2, step (wave % 2) ND + i of its columns
    }
    const int k0 = (int)((uint32_t)keys.base + (uint32_t)step * 64) + wave * 16;
    const bool edge = k0 < keys.lo || k0 + 16 > keys.hi;
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
#pragma unroll
      for (int i = 0; i < 2 * ND; ++i)
        z[s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(buf, s * 2 * ND + i), q[i], z[s], 0, 0, 0);
    }
    if (k0 < lo_max || k0 + 64 > hi_min) {
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
      }
      p[s] = as_frag(f);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < ND; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(buf, 4 * ND + s * ND + i), p[s], acc[i], 0, 0, 0);
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
  if (!has) return;
  const int64_t token = t.first_token + tok, head = (int64_t)kvh * a.group + gh, row = token * a.q_heads + head;
  const bool sees_some = my.hi > my.lo;
  const int64_t all_rows = (int64_t)a.tokens * a.q_heads;
  const float inv = splits > 1 ? 1.0f : sees_some ? 1.0f / l : 0.0f;
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
__global__ __launch_bounds__(256) void kv4_join_kernel(Attn4Args a, int splits, int slices) {
  __shared__ Part share[256];
  const int64_t all_rows = (int64_t)a.tokens * a.q_heads;
  const int d = a.cache.d, lanes = d / 4, items = 256 / slices;
  const int slice = threadIdx.x / items, mine = threadIdx.x - slice * items;
  const float* stats = a.partial + (int64_t)splits * all_rows * d;
  // rows behind the last sequence have no parts
  const int64_t rows = (int64_t)min(max(a.plan.starts[a.plan.sequences], 0), a.tokens) * a.q_heads;
  for (int64_t first = (int64_t)blockIdx.x * items; first < rows * lanes; first += (int64_t)gridDim.x * items) {
    const int64_t item = first + mine, row = item / lanes;
    const int col = 4 * (int)(item - row * lanes);
    Part p = {-INFINITY, 0.0f, {0, 0, 0, 0}};
    bool none = false;
    if (row < rows) {
      const float* from = a.partial + row * d + col;
      for (int i0 = slice; i0 < splits; i0 += 8 * slices) {
        f32x2 st[8];
        f32x4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t at = (int64_t)min(i0 + i * slices, splits - 1) * all_rows;
          st[i] = *reinterpret_cast<const f32x2*>(stats + (at + row) * 2);
          x[i] = *reinterpret_cast<const f32x4*>(from + at * d);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i * slices < splits) {
            none |= st[i][1] < 0.0f;
            p.add(st[i][0], st[i][1], x[i]);
          }
      }
    }
    if (slices > 1) {
      __syncthreads();  // the last items' are done with
      share[threadIdx.x] = p;
      __syncthreads();
      if (slice == 0)
        for (int i = 1; i < slices; ++i) p.add(share[i * items + mine].top, share[i * items + mine].sum, share[i * items + mine].o);
    }
    if (slice == 0 && row < rows) {
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

constexpr int kMostSplits = 256;

// How a call is cut: tiles of 16, 32 or 128 rows, by the rows that a sequence
// has on average, and the keys in parts until the chip has work enough.
struct Cut {
  int rows, splits;
  int64_t tiles;
};
Cut cut_of(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t page_size, int64_t sequences, int64_t width) {
  const int64_t group = q_heads / kv_heads, rows = tokens * group;
  Cut c;
  c.rows = rows > 64 * sequences ? 128 : rows > 16 * sequences ? 32 : 16;
  c.tiles = rows / c.rows + sequences;
  const int64_t busy = std::max<int64_t>(1, std::max(rows / c.rows, std::min(sequences, tokens)) * kv_heads);
  const int64_t keys = width * page_size, most = std::max<int64_t>(1, (keys + 127) / 128);
  const int64_t fill = ((c.rows == 128 ? 512 : 768) + busy - 1) / busy;
  const int64_t even = busy >= 256 && c.rows < 128 ? (keys + 2047) / 2048 : 1;
  c.splits = (int)std::min({most, std::max(fill, even), (int64_t)kMostSplits});
  return c;
}

template <int ND>
hipError_t go(const Attn4Args& a, const Cut& c, hipStream_t stream) {
  const int64_t units = c.tiles * a.cache.heads * c.splits;
  constexpr int64_t kMost = 1 << 23;  // workgroups of a launch: 2^32 threads are refused
  for (int64_t u = 0; u < units; u += kMost) {
    const dim3 grid((unsigned)std::min(kMost, units - u));
    if (c.rows == 16) hipLaunchKernelGGL((kv4_attention_kernel<ND, 1>), grid, dim3(256), 0, stream, a, c.splits, u);
    else if (c.rows == 32) hipLaunchKernelGGL((kv4_attention_kernel<ND, 2>), grid, dim3(256), 0, stream, a, c.splits, u);
    else hipLaunchKernelGGL((kv4_prompt_kernel<ND>), grid, dim3(256), 0, stream, a, c.splits, u, c.tiles);
  }
  if (c.splits > 1) {
    const int64_t rows = (int64_t)a.tokens * a.q_heads;
    int slices = 1;
    while (slices < 32 && slices * 8 < c.splits) slices *= 2;
    const int64_t items = rows * (ND * 8), per = 256 / slices;
    hipLaunchKernelGGL(kv4_join_kernel, dim3((unsigned)std::min((items + per - 1) / per, kMost)), dim3(256), 0, stream,
                       a, c.splits, slices);
  }
  return hipGetLastError();
}

}  // namespace

int64_t kv4_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size,
                                int64_t sequences, int64_t width) {
  if (tokens == 0 || sequences == 0) return 0;
  const Cut c = cut_of(tokens, q_heads, kv_heads, page_size, sequences, width);
  return c.splits == 1 ? 0 : tokens * q_heads * c.splits * (d + 2) * 4;
}

hipError_t launch_kv4_attention(const Attn4Args& a, hipStream_t stream) {
  const Cut c = cut_of(a.tokens, a.q_heads, a.cache.heads, 1LL << a.cache.page_log2, a.plan.sequences, a.plan.width);
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
