// y = A W^T of E4M3-coded matrices with one scale per block of 128 along the
// reduction, on the 8-bit matrix instructions of gfx950
// (v_mfma_f32_16x16x128_f8f6f4: one instruction reduces exactly one block).
//
//   y[m][n] = sum_b sa[m][b] sw[n/128][b] sum_{k in b} a[m][k] w[n][k]
//
// Inside one 8-bit matrix instruction the products are added at a limited
// width: its sums are off by 1.3e-5 (relative, measured on normal operands;
// the 16x16x32 form is no better).  That is far below a bf16 result's rounding
// (2^-9), which is what it is used for.  fp32 results take the bf16 matrix
// instructions on the same codes (4 significant bits, exact in bf16), whose
// sums are off by 1e-8.
//
// The weight is the instruction's first operand, so a lane's four results are
// four neighbouring n of one row m: the row's scale is one value per lane and
// the store one vector.
#include <algorithm>

#include "q8.h"

namespace harp {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ void store4(T* p, int n, const f32x4& v);
template <>
__device__ __forceinline__ void store4<float>(float* p, int n, const f32x4& v) {
  struct __attribute__((packed, aligned(4))) R { float f[4]; };
  if (n >= 4) *reinterpret_cast<R*>(p) = R{{v[0], v[1], v[2], v[3]}};
  else
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t* p, int n, const f32x4& v) {
  struct __attribute__((packed, aligned(2))) R { uint32_t w[2]; };
  const uint32_t lo = pack_bf16x2_hw(v[0], v[1]), hi = pack_bf16x2_hw(v[2], v[3]);
  if (n >= 4) *reinterpret_cast<R*>(p) = R{{lo, hi}};
  else
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
}

// Tiles in LDS: 128-byte rows (one block of 128) of eight 16-byte pieces,
// exchanged by spread(row) so that the fragment reads below cover all banks.
// A wave reads its weight rows in the order n = 16 (r / 4) + 4 i + r % 4 for
// instruction i of four and row r of it: a lane's results of four
// instructions are then 16 neighbouring n.  Eight neighbouring r are rows
// 0..3 and 16..19 (weight) or 0..7 (activations, read in order), hence the
// two forms.
__device__ __forceinline__ int spread_w(int row) { return (row & 3) | ((row >> 2) & 4); }
__device__ __forceinline__ int spread_a(int row) { return row & 7; }

// A fragment: the pieces q and q + 4 of a row.
__device__ __forceinline__ i32x8 frag(const uint8_t* lds, int row, int x, int q) {
  const uint8_t* p = lds + row * kQBlk;
  const i32x4 a = *reinterpret_cast<const i32x4*>(p + ((q ^ x) << 4));
  const i32x4 b = *reinterpret_cast<const i32x4*>(p + (((q ^ x) ^ 4) << 4));
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Eight of a fragment's 32 codes as bf16 (exact).
__device__ __forceinline__ bf16x8_t widen(const i32x8& f, int t) {
  bf16x2_t v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * t + i], 1.0f, false);
    v[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * t + i], 1.0f, true);
  }
  bf16x8_t r;
  __builtin_memcpy(&r, v, 16);
  return r;
}

constexpr int kChunk = 8;  // steps whose row scales are brought in together

// One 16 MT MW x 16 NT NW tile of y per workgroup of MW x NW waves, each with
// 16 MT rows (m) by 16 NT columns (n) of it.  LDS holds two steps of one
// block of 128: while a step is computed the next one is on its way.
// 64 x 64 per wave; 32 x 64 (MT = 2) below 384 tiles of 128 x 128, where twice
// the workgroups even the load out: 777 x 5120 x 4112, fp32 results, 59 us
// against 70, while at 432 tiles (bf16) 68 against 53.  fp32 results multiply
// on the bf16 instructions: 96 conversions go with every 32 of them.
template <int MT, int MW, int NW, int NT, bool E8, typename TO, Rows kRows>
__global__ __launch_bounds__(64 * MW * NW) void matmul_tile_kernel(MatmulArgs g, int kb_per_split, int tiles_m,
                                                                   int tiles_n) {
  constexpr int BM = 16 * MT * MW, BN = 16 * NT * NW, WAVES = MW * NW;
  constexpr int PA = BM / 8 / WAVES, PW = BN / 8 / WAVES;  // 8-row pieces of each operand a wave brings in
  static_assert(PA * 8 * WAVES == BM && PW * 8 * WAVES == BN, "");
  __shared__ __align__(16) uint8_t la[2][BM * kQBlk];
  __shared__ __align__(16) uint8_t lw[2][BN * kQBlk];
  __shared__ uint32_t ls[2][BM * kChunk];
  const uint32_t lds_a = lds_address(la), lds_w = lds_address(lw), lds_s = lds_address(ls);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tm, tn;
  tile_of((int)blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int wm = (wave / NW) * (16 * MT), wn = (wave % NW) * (16 * NT);
  const int q = lane >> 4, i16 = lane & 15;
  const int kb0 = (int)blockIdx.y * kb_per_split, kb1 = min(g.nkb, kb0 + kb_per_split);
  // bf16 results with E8M0 scales: the instruction applies the scales
  constexpr bool kHwScale = E8 && sizeof(TO) == 2, kWide = sizeof(TO) == 4;

  // what this lane brings in: piece pc of rows 8 (wave + WAVES i) + lane / 8,
  // to be found at lane * 16 of its 1024 bytes of LDS
  const uint8_t* abase = g.a + (int64_t)m0 * g.lda;
  const uint8_t* wbase = g.w + (int64_t)n0 * g.ldw;
  const int rows_a = min(BM, g.rows - m0), rows_w = min(BN, g.n - n0);
  const int lrow = lane >> 3;
  const int pca = ((lane & 7) ^ lrow) * 16;
  // spread_w of row 8 (wave + WAVES i) + lrow: WAVES is even, so bit 4 of the
  // row is bit 1 of the wave
  static_assert(WAVES % 4 == 0 || PW == 1, "");
  const int pcw = ((lane & 7) ^ (lrow & 3) ^ ((wave & 2) << 1)) * 16;
  TileSrc ra, rw;
  unsigned va[PA], vw[PW];
  if constexpr (kRows != kNarrow) {
    ra = tile_src(abase, (rows_a - 1) * (int)g.lda + g.k);
    rw = tile_src(wbase, (rows_w - 1) * (int)g.ldw + g.k);
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = (wave + WAVES * i) * 8 + lrow;
      va[i] = r < rows_a ? (unsigned)(r * (int)g.lda + pca) : kNoLoad;
    }
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      const int r = (wave + WAVES * i) * 8 + lrow;
      vw[i] = r < rows_w ? (unsigned)(r * (int)g.ldw + pcw) : kNoLoad;
    }
  }
  // asks for a step; what comes through registers is kept after the products
  u32x4 xa[PA], xw[PW];
  auto bring = [&](int kb, int buf) {
    const int kk = kb * kQBlk, na = g.k - kk - pca, nw = g.k - kk - pcw;
    // kCut: a piece with n bytes left is loaded from 16 - n bytes before
    const unsigned ca = kRows == kCut && na > 0 && na < 16 ? 16 - na : 0, cw = kRows == kCut && nw > 0 && nw < 16 ? 16 - nw : 0;
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = (wave + WAVES * i) * 8 + lrow;
      if constexpr (kRows == kWhole)
        load_lds16(ra, lds_a + (uint32_t)(buf * BM * kQBlk + (wave + WAVES * i) * 1024), na > 0 ? va[i] : kNoLoad, kk);
      else if constexpr (kRows == kCut) xa[i] = load_16(ra, na > 0 ? va[i] + kk - ca : kNoLoad);
      else xa[i] = load16_bytes(abase + (int64_t)r * g.lda + kk + pca, r < rows_a ? na : 0);
    }
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      const int r = (wave + WAVES * i) * 8 + lrow;
      if constexpr (kRows == kWhole)
        load_lds16(rw, lds_w + (uint32_t)(buf * BN * kQBlk + (wave + WAVES * i) * 1024), nw > 0 ? vw[i] : kNoLoad, kk);
      else if constexpr (kRows == kCut) xw[i] = load_16(rw, nw > 0 ? vw[i] + kk - cw : kNoLoad);
      else xw[i] = load16_bytes(wbase + (int64_t)r * g.ldw + kk + pcw, r < rows_w ? nw : 0);
    }
  };
  auto keep = [&](int kb, int buf) {
    if constexpr (kRows == kWhole) return;
    const int na = g.k - kb * kQBlk - pca, nw = g.k - kb * kQBlk - pcw;
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      if (kRows == kCut && na > 0 && na < 16) xa[i] = shift_down(xa[i], 16 - na);
      *reinterpret_cast<u32x4*>(la[buf] + (wave + WAVES * i) * 1024 + lane * 16) = xa[i];
    }
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      if (kRows == kCut && nw > 0 && nw < 16) xw[i] = shift_down(xw[i], 16 - nw);
      *reinterpret_cast<u32x4*>(lw[buf] + (wave + WAVES * i) * 1024 + lane * 16) = xw[i];
    }
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  // Scales of the rows: a load of one step's 64 would touch 64 cache lines, so
  // they come kChunk steps at a time, 8 rows by 8 steps per wave's load, and
  // wait in LDS as [row][step] (E8M0: the byte, one per word).
  constexpr int kSB = E8 ? 1 : 4;
  const uint8_t* sbase = static_cast<const uint8_t*>(g.a_scales) + (int64_t)m0 * g.nkb * kSB;
  TileSrc rs;
  if constexpr (kRows != kNarrow) rs = tile_src(sbase, rows_a * g.nkb * kSB);
  auto bring_scales = [&](int kb, int buf) {
    const int k1 = lane & (kChunk - 1);
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = (wave + WAVES * i) * 8 + lrow;
      const bool in = r < rows_a && kb + k1 < kb1;
      if constexpr (kRows != kNarrow) {
        load_lds_word<kSB>(rs, lds_s + (uint32_t)((buf * BM * kChunk + (wave + WAVES * i) * 64) * 4), in ? (unsigned)((r * g.nkb + k1) * kSB) : kNoLoad,
                           kb * kSB);
      } else {
        const int64_t at = (int64_t)r * g.nkb + kb + k1;
        uint32_t v = 0;
        if (in) v = E8 ? sbase[at] : reinterpret_cast<const uint32_t*>(sbase)[at];
        ls[buf][(wave + WAVES * i) * 64 + lane] = v;
      }
    }
  };
  const int64_t sw_row = (int64_t)min((n0 + wn) / kQBlk, (g.n - 1) / kQBlk) * g.nkb;
  uint32_t sw;
  auto load_sw = [&](int kb) {
    if constexpr (E8) sw = static_cast<const uint8_t*>(g.w_scales)[sw_row + kb];
    else sw = static_cast<const uint32_t*>(g.w_scales)[sw_row + kb];
  };

  bring(kb0, 0);
  keep(kb0, 0);
  bring_scales(kb0, 0);
  load_sw(kb0);
  // every wave's own loads have landed before the barrier lets others read
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  for (int kb = kb0; kb < kb1; ++kb) {
    const int step = kb - kb0, buf = step & 1, in = step % kChunk;
    float s[MT];
    int sb[MT];
    // the weight's scale becomes a number here and not, with a wait for every
    // load, in the step that asks for it
    if constexpr (!kHwScale) asm volatile("" : "+v"(sw));
    const int swb = (int)sw;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const uint32_t sa = ls[step / kChunk & 1][(wm + j * 16 + i16) * kChunk + in];
      sb[j] = (int)sa;
      if constexpr (!kHwScale)
        s[j] = E8 ? e8m0_value(sa) * e8m0_value(sw) : __uint_as_float(sa) * __uint_as_float(sw);
    }
    if (kb + 1 < kb1) {
      bring(kb + 1, buf ^ 1);
      load_sw(kb + 1);
      if (in == kChunk - 1) bring_scales(kb + 1, (step / kChunk & 1) ^ 1);
    }
    i32x8 fa[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) fa[j] = frag(la[buf], wm + j * 16 + i16, i16 & 7, q);
    auto weight = [&](int i) {
      const int row = (i >> 2) * 64 + (i16 >> 2) * 16 + (i & 3) * 4 + (i16 & 3);
      return frag(lw[buf], wn + row, (i16 & 3) | (i16 & 4), q);
    };
    i32x8 fw = weight(0);
    f32x4 p[2][MT];
#pragma unroll
    for (int i = 0; i <= NT; ++i) {
      i32x8 next;
      if (i + 1 < NT) next = weight(i + 1);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (i < NT) {
          if constexpr (kHwScale) {
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], acc[i][j], 0, 0, 0, swb, 0, sb[j]);
          } else if constexpr (kWide) {
            p[i & 1][j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < 4; ++t)
              p[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fw, t), widen(fa[j], t), p[i & 1][j], 0, 0, 0);
          } else {
            p[i & 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
          }
        }
        if constexpr (!kHwScale) {
          if (i > 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i - 1][j][e] = fmaf(p[(i - 1) & 1][j][e], s[j], acc[i - 1][j][e]);
          // keep the order: a matrix instruction, then the scaling of a result of the row before
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      fw = next;
    }
    if (kb + 1 < kb1) keep(kb + 1, buf ^ 1);
    // this step's reads are done and the next step's loads have landed
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm + j * 16 + i16;
    if (m >= g.rows) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = n0 + wn + (i >> 2) * 64 + q * 16 + (i & 3) * 4;
      if (n >= g.n) continue;
      if (gridDim.y > 1)
        store4<float>(g.partial + ((int64_t)blockIdx.y * g.rows + m) * g.n + n, g.n - n, acc[i][j]);
      else store4<TO>(static_cast<TO*>(g.y) + (int64_t)m * g.ldy + n, g.n - n, acc[i][j]);
    }
  }
}

// The large form, bf16 results: 256 x 256 tiles, 8 waves, each 64 rows (m) by
// 128 columns (n).  Nothing in the loop waits for a load that was issued less
// than a whole step before, and the loads are never drained: LDS holds two
// steps in three parts (A, and the two halves W0, W1 of each wave's weight
// rows), and a part is filled again for two steps on as soon as every wave has
// read it.  Per step k, in parts of 8 result rows:
//   row 0      multiply; A of step k is in registers
//   barrier 1  W1(k) has landed
//   rows 1..3  multiply; fill W1(k + 1), A(k + 2)
//   barrier 2  A(k + 1), W0(k + 1) and the scales of k + 1 have landed
//   rows 4..7  multiply; fill the scales of k + 2, W0(k + 2); read A(k + 1) and
//              row 0 of W0(k + 1)
// The scaling of a product runs under the matrix instructions after it.
//
// One workgroup per compute unit walks over tiles, and the steps run on from
// one tile into the next: its first loads are on their way during the last
// steps, and the stores of a tile drain during the first step of the next
// (kStores is added to what that step's waits count on).  Bound by the matrix
// instructions: at 16384 x 13824 x 5120 they alone, on the same operands, take
// 674 us; the whole 1003 to 1039 us with fp32 scales (2.3 PFLOP/s; every
// block's product is scaled on the vector unit, a multiply-add per result and
// block) and 895 to 924 us with E8M0, which the instruction applies itself
// (2.6 PFLOP/s, a per-tensor library product's rate).
constexpr int kBigA = 4, kBigW = 4;  // loads per wave and step: A, W (half of them W0)
constexpr int kStores = 16;          // stores per wave and tile

// Waits until at most kLoads loads (kMore more operations in a tile's first
// step) are outstanding, then for the other waves.  The choice is made inside
// the statement: a branch that the compiler sees lets it move the scaling of
// products past it.
template <int kLoads, int kMore>
__device__ __forceinline__ void wait_barrier(int step) {
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\t"
      "s_cbranch_scc1 .Lfirst%=\n\t"
      "s_waitcnt vmcnt(%1)\n"
      ".Lfirst%=:\n\t"
      "s_waitcnt vmcnt(%2)\n\t"
      "s_barrier" ::"s"(step), "i"(kLoads), "i"(kLoads + kMore)
      : "memory", "scc");
}

template <bool E8>
__global__ __launch_bounds__(512) void matmul_big_kernel(MatmulArgs g, int tiles_m, int tiles_n, bool whole_y) {
  constexpr int B = 256, NT = 8, kHalf = B * kQBlk;  // bytes of one operand of a step
  constexpr uint32_t kW = 2 * kHalf, kS = 4 * kHalf, kSBuf = 2048;
  __shared__ __align__(16) uint8_t smem[kS + 2 * kSBuf];
  const uint32_t lds = lds_address(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 128;
  const int q = lane >> 4, i16 = lane & 15, lrow = lane >> 3;
  const int nkb = g.nkb;
  constexpr int kSB = E8 ? 1 : 4;

  // What this lane brings in: pieces of rows 8 wave + lrow (+ 64 i), as in
  // matmul_tile_kernel; scales of row 64 wave + lane (waves 0..3) or of weight
  // block `lane` (wave 4).  Rows past the matrix's end are past the
  // descriptor's, too; in the last block, pieces past the row's end are not
  // loaded.
  const int last = (nkb - 1) * kQBlk;
  const int pca = ((lane & 7) ^ lrow) * 16, pcw = ((lane & 7) ^ (lrow & 3) ^ ((wave & 2) << 1)) * 16;
  const unsigned va = (unsigned)((wave * 8 + lrow) * (int)g.lda + pca), vw = (unsigned)((wave * 8 + lrow) * (int)g.ldw + pcw);
  const unsigned va_last = last + pca < g.k ? va : kNoLoad, vw_last = last + pcw < g.k ? vw : kNoLoad;
  const unsigned vs = wave < 4 ? (unsigned)((wave * 64 + lane) * nkb * kSB)
                               : wave == 4 && lane < 2 ? (unsigned)(lane * nkb * kSB) : kNoLoad;
  auto a_of = [&](int m0) { return tile_src(g.a + (int64_t)m0 * g.lda, (min(B, g.rows - m0) - 1) * (int)g.lda + g.k); };
  auto w_of = [&](int n0) { return tile_src(g.w + (int64_t)n0 * g.ldw, (min(B, g.n - n0) - 1) * (int)g.ldw + g.k); };
  auto s_of = [&](int m0, int n0) {
    const int blocks = (g.n - 1) / kQBlk - n0 / kQBlk + 1;
    const void* scales = wave == 4 ? g.w_scales : g.a_scales;
    return tile_src(static_cast<const uint8_t*>(scales) + (int64_t)(wave == 4 ? n0 / kQBlk : m0) * nkb * kSB,
                    (wave == 4 ? min(2, blocks) : min(B, g.rows - m0)) * nkb * kSB);
  };
  // `to`: the LDS offset of the step's buffers, 0 or kHalf
  auto fill_a = [&](TileSrc src, int kb, uint32_t to, int i) {
    load_lds16(src, lds + to + (uint32_t)(wave + 8 * i) * 1024, (kb == nkb - 1 ? va_last : va) + 64 * i * (unsigned)g.lda, kb * kQBlk);
  };
  auto fill_w = [&](TileSrc src, int kb, uint32_t to, int i) {  // i even: W0, odd: W1
    load_lds16(src, lds + kW + to + (uint32_t)(wave + 8 * i) * 1024, (kb == nkb - 1 ? vw_last : vw) + 64 * i * (unsigned)g.ldw,
               kb * kQBlk);
  };
  auto fill_s = [&](TileSrc src, int kb, uint32_t to) {
    load_lds_word<kSB>(src, lds + kS + to / (kHalf / kSBuf) + (uint32_t)wave * 256, vs, kb * kSB);
  };

  f32x4 acc[NT][4], p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = f32x4{0, 0, 0, 0};
  i32x8 fa[4], fw;
  float s[4] = {0, 0, 0, 0};
  uint32_t sa[4], sw;
  // offsets of this lane's fragments in the buffers of the step at hand; the
  // other step's are at ^ kHalf, a fragment's second piece is at ^ 64
  uint32_t oa = (uint32_t)((wm + i16) * kQBlk + ((q ^ (i16 & 7)) << 4)), to = 0;
  uint32_t ow = kW + (uint32_t)((wn + (i16 >> 2) * 16 + (i16 & 3)) * kQBlk + ((q ^ (i16 & 7)) << 4));
  auto read = [&](uint32_t at, int off) {
    const i32x4 x = *reinterpret_cast<const i32x4*>(smem + at + off), y = *reinterpret_cast<const i32x4*>(smem + (at ^ 64) + off);
    return i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  auto weight = [&](uint32_t at, int i) { return read(at, ((i >> 2) * 64 + (i & 3) * 4) * kQBlk); };
  auto read_scales = [&](uint32_t buf) {
    const uint32_t* ls = reinterpret_cast<const uint32_t*>(smem + kS + buf / (kHalf / kSBuf));
    sw = ls[256 + (wave & 1)];
#pragma unroll
    for (int j = 0; j < 4; ++j) sa[j] = ls[wm + j * 16 + i16];
  };

  const int tiles = tiles_m * tiles_n;
  int tm, tn;
  tile_of((int)blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  int m0 = tm * B, n0 = tn * B;
  TileSrc a0 = a_of(m0), w0 = w_of(n0), s0 = s_of(m0, n0);
  for (int t = 0; t < 2; ++t) {
    for (int i = 0; i < kBigA; ++i) fill_a(a0, t, t * kHalf, i);
    for (int i = 0; i < kBigW; ++i)
      if (t == 0 || (i & 1) == 0) fill_w(w0, t, t * kHalf, i);
    fill_s(s0, t, t * kHalf);
  }
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int j = 0; j < 4; ++j) fa[j] = read(oa, j * 16 * kQBlk);
  fw = weight(ow, 0);
  read_scales(0);

  for (int tile = (int)blockIdx.x; tile < tiles; tile += (int)gridDim.x) {
    // the next tile (the last one's: itself again, and nobody reads it)
    tile_of(tile + (int)gridDim.x < tiles ? tile + (int)gridDim.x : tile, tiles_m, tiles_n, &tm, &tn);
    const int m1 = tm * B, n1 = tn * B;
    const TileSrc a1 = a_of(m1), w1 = w_of(n1), s1 = s_of(m1, n1);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    // what the last tile left in p has been added; the first step adds it again
    // times s, and a NaN in it would come through a zero s
    p[2] = p[3] = f32x4{0, 0, 0, 0};
    s[2] = s[3] = 0.0f;
    auto step = [&](int kb) {
      const int k1 = kb + 1 < nkb ? kb + 1 : 0, k2 = kb + 2 < nkb ? kb + 2 : kb + 2 - nkb;
      const TileSrc wn1 = kb + 1 < nkb ? w0 : w1, an2 = kb + 2 < nkb ? a0 : a1, wn2 = kb + 2 < nkb ? w0 : w1,
                    sn2 = kb + 2 < nkb ? s0 : s1;
      const uint32_t oan = oa ^ kHalf, own = ow ^ kHalf;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const i32x8 next = i + 1 < NT ? weight(ow, i + 1) : weight(own, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (E8) {
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], acc[i][j], 0, 0, 0, (int)sw, 0, (int)sa[j]);
          } else {
            p[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            // the products of two instructions ago
            const int pj = (j + 2) & 3, pi = j >= 2 ? i : i > 0 ? i - 1 : NT - 1;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[pi][pj][e] = fmaf(p[pj][e], s[pj], acc[pi][pj][e]);
            if (i == 0 && j == 1) {
#pragma unroll
              for (int t = 0; t < 4; ++t) s[t] = __uint_as_float(sa[t]) * __uint_as_float(sw);
            }
          }
          if (i == NT - 1) fa[j] = read(oan, j * 16 * kQBlk);
          // one load per two instructions at most: more at a time fill the
          // memory pipe's queue, and the wave stands still until they fit
          if (i == 1 && (j & 1) == 0) fill_w(wn1, k1, to ^ kHalf, 1 + j);
          if ((i == 2 || i == 3) && (j & 1) == 0) fill_a(an2, k2, to, (i - 2) * 2 + j / 2);
          if (i == 4 && j == 1) fill_s(sn2, k2, to);
          if ((i == 5 || i == 6) && j == 1) fill_w(wn2, k2, to, (i - 5) * 2);
          __builtin_amdgcn_sched_barrier(0);
        }
        fw = next;
        // newer than W1(k): A(k + 1), the scales, W0(k + 1) (and the stores)
        if (i == 0) wait_barrier<kBigA + kBigW / 2 + 1, kStores>(kb);
        // newer than W0(k + 1): (the stores,) W1(k + 1), A(k + 2)
        if (i == 3) wait_barrier<kBigA + kBigW / 2, kStores>(kb);
      }
      oa = oan;
      ow = own;
      to ^= kHalf;
      read_scales(to);
    };
    for (int kb = 0; kb < nkb; ++kb) step(kb);
    if constexpr (!E8) {
#pragma unroll
      for (int j = 2; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[NT - 1][j][e] = fmaf(p[j][e], s[j], acc[NT - 1][j][e]);
    }
    if (whole_y) {
      // rows of whole 16-byte pieces: always the same number of stores
      const TileSrc ry = tile_src(static_cast<const uint16_t*>(g.y) + (int64_t)m0 * g.ldy + n0,
                                  ((min(B, g.rows - m0) - 1) * (int)g.ldy + g.n - n0) * 2);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          const int col = wn + (i >> 2) * 64 + q * 16 + (i & 3) * 4;
          u32x4 v;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[2 * h] = pack_bf16x2_hw(acc[i + h][j][0], acc[i + h][j][1]);
            v[2 * h + 1] = pack_bf16x2_hw(acc[i + h][j][2], acc[i + h][j][3]);
          }
          store_16(ry, n0 + col < g.n ? (unsigned)((wm + j * 16 + i16) * (int)g.ldy + col) * 2u : kNoLoad, v);
        }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + wm + j * 16 + i16;
        if (m >= g.rows) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int n = n0 + wn + (i >> 2) * 64 + q * 16 + (i & 3) * 4;
          if (n < g.n) store4<uint16_t>(static_cast<uint16_t*>(g.y) + (int64_t)m * g.ldy + n, g.n - n, acc[i][j]);
        }
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the next step counts on kStores at most
    }
    m0 = m1;
    n0 = n1;
    a0 = a1;
    w0 = w1;
    s0 = s1;
  }
  // no load may be in flight into LDS when the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Few rows (a decoding step): the weight is read once and bounds the time, so
// it goes straight from global memory into the fragments.  A workgroup
// computes 16 NT columns (n) of 16 rows; its 8 waves share the blocks of
// the reduction out, each a contiguous run, and add their sums through LDS: one
// launch, no workspace.  Each wave keeps kRing blocks of both operands on
// their way.  1 x 4096 x 4096: 6 to 7 us of the call's 8 (the ring form 13);
// 13824 x 5120 takes 18 to 22 us here and 14 to 15 in the ring form, where the
// weight streams better: hence up to 2^25 codes.  Row scales: a lane's load of one block's would touch 16 lines, so lane
// (q, i16) loads block q of four for row i16 and the others ask it.
template <int NT, bool E8, typename TO>
__global__ __launch_bounds__(512) void matmul_few_kernel(MatmulArgs g, int per) {
  __shared__ __align__(16) f32x4 part[8][NT][64];
  constexpr bool kHwScale = E8 && sizeof(TO) == 2, kWide = sizeof(TO) == 4;
  constexpr int kRing = 4;  // blocks on their way, and whose scales come together
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, i16 = lane & 15;
  const int n0 = (int)blockIdx.x * 16 * NT, m0 = (int)blockIdx.y * 16;
  const int kb0 = wave * per, kb1 = min(g.nkb, kb0 + per);
  const TileSrc rw = tile_src(g.w + (int64_t)n0 * g.ldw, (min(16 * NT, g.n - n0) - 1) * (int)g.ldw + g.k);
  const TileSrc ra = tile_src(g.a + (int64_t)m0 * g.lda, (min(16, g.rows - m0) - 1) * (int)g.lda + g.k);
  const int end = min(g.k, kb1 * kQBlk);

  i32x8 fw[kRing][NT], fa[kRing];
  auto load = [&](int slot, int kb) {
    // pieces past the end are not loaded; one that the end cuts is loaded from
    // 16 bytes before it and shifted when it is used
    unsigned v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = kb * kQBlk + q * 16 + h * 64;
      v[h] = at < end ? (unsigned)min(at, g.k - 16) : kNoLoad;
    }
    auto piece = [&](TileSrc src, int row, int64_t ld, i32x8& f) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 w = load_16(src, v[h] + (unsigned)(row * (int)ld));
#pragma unroll
        for (int c = 0; c < 4; ++c) f[4 * h + c] = (int)w[c];
      }
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) piece(rw, 16 * t + i16, g.ldw, fw[slot][t]);
    piece(ra, i16, g.lda, fa[slot]);
  };
  auto cut = [&](int kb, i32x8& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int over = kb * kQBlk + q * 16 + h * 64 + 16 - g.k;
      if (over > 0 && over < 16) {
        const u32x4 w = shift_down(u32x4{(uint32_t)f[4 * h], (uint32_t)f[4 * h + 1], (uint32_t)f[4 * h + 2],
                                         (uint32_t)f[4 * h + 3]}, over);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[4 * h + c] = (int)w[c];
      }
    }
  };

  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0, 0, 0, 0};
  const int64_t sw_row = (int64_t)(n0 / kQBlk) * g.nkb;
  const int64_t sa_row = (int64_t)min(m0 + i16, g.rows - 1) * g.nkb;
  uint32_t sa, sw;
  auto load_scales = [&](int kb) {
    const int at = min(kb + q, g.nkb - 1);
    sw = scale_bits<E8>(g.w_scales, sw_row + at);
    sa = scale_bits<E8>(g.a_scales, sa_row + at);
  };

  if (kb0 < kb1) {
    load_scales(kb0);
#pragma unroll
    for (int t = 0; t < kRing; ++t) load(t, kb0 + t);
    const bool cuts = (g.k & 15) != 0 && kb1 == g.nkb;
    for (int kb = kb0; kb < kb1; kb += kRing) {
      const uint32_t w4 = sw;
      const uint32_t s4 = kHwScale ? sa : __float_as_uint(scale_value<E8>(sa) * scale_value<E8>(sw));
      load_scales(kb + kRing);
#pragma unroll
      for (int t = 0; t < kRing; ++t) {
        if (cuts && kb + t == g.nkb - 1) {
#pragma unroll
          for (int i = 0; i < NT; ++i) cut(kb + t, fw[t][i]);
          cut(kb + t, fa[t]);
        }
        // blocks past the run: codes zero, and a scale that may be anything
        const bool in = kb + t < kb1;
        const int swb = __builtin_amdgcn_readlane((int)w4, 16 * t);
        const uint32_t sj = (uint32_t)__shfl((int)s4, 16 * t + i16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (kHwScale) {
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[t][i], fa[t], acc[i], 0, 0, 0, in ? swb : 127, 0,
                                                                      in ? (int)sj : 127);
          } else {
            f32x4 p = {0, 0, 0, 0};
            if constexpr (kWide) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fw[t][i], u), widen(fa[t], u), p, 0, 0, 0);
            } else {
              p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[t][i], fa[t], p, 0, 0, 0, 0, 0, 0);
            }
            const float f = in ? __uint_as_float(sj) : 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], f, acc[i][e]);
          }
        }
        load(t, kb + kRing + t);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int u = threadIdx.x; u < NT * 64; u += 512) {
    const int l = u & 63, t = u >> 6, m = m0 + (l & 15), n = n0 + 16 * t + 4 * (l >> 4);
    f32x4 s = part[0][t][l];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += part[w][t][l][e];
    }
    if (m < g.rows && n < g.n) store4<TO>(static_cast<TO*>(g.y) + (int64_t)m * g.ldy + n, g.n - n, s);
  }
}

// Tiles that wait for memory rather than multiply: a batch of rows that is
// small for its weight, or too few tiles for 256 x 256.  LDS holds a ring of
// kRing steps, all but one of them on their way, and nothing is ever drained.
// One 16 MT WM x 16 NT WN tile per workgroup of WM x WN waves.  A step's
// scales come with it: by lane for the rows, a load that touches 64 lines but
// is one of a step's five.  64 x 13824 x 5120: 17 us (4.3 TB/s of codes).
template <int MT, int NT, int WM, int WN, bool E8, typename TO>
__global__ __launch_bounds__(64 * WM * WN) void matmul_ring_kernel(MatmulArgs g, int kb_per_split, int tiles_m,
                                                                   int tiles_n, int first_tile) {
  constexpr bool kHwScale = E8 && sizeof(TO) == 2, kWide = sizeof(TO) == 4;
  constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN, WAVES = WM * WN;
  static_assert(BM <= 128 && BN <= kQBlk && NT <= 2 && WAVES >= 4, "");
  constexpr int kScales = (BM + BN) * kQBlk, kBytes = kScales + 1024;
  constexpr int kRing = std::min(144 * 1024 / kBytes, 12);
  constexpr int LA = (BM / 8 + WAVES - 1) / WAVES, LW = BN / 8 / WAVES, kLoads = LA + LW + 1;  // per wave and step
  // a step: W, A, and 64 words each from four waves: the row scales (waves 0
  // and 1), the weight's (2), words that nobody reads (the others)
  __shared__ __align__(16) uint8_t ring[kRing][kBytes];
  __shared__ __align__(16) uint8_t spare[1024];
  const uint32_t lds_ring = lds_address(ring), lds_spare = lds_address(spare);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, i16 = lane & 15, lrow = lane >> 3;
  int tm, tn;
  tile_of(first_tile + (int)blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int wm = wave / WN * (16 * MT), wn = wave % WN * (16 * NT);
  const int kb0 = (int)blockIdx.y * kb_per_split, kb1 = min(g.nkb, kb0 + kb_per_split);
  const int rows_a = min(BM, g.rows - m0), rows_w = min(BN, g.n - n0);
  const TileSrc ra = tile_src(g.a + (int64_t)m0 * g.lda, (rows_a - 1) * (int)g.lda + g.k);
  const TileSrc rw = tile_src(g.w + (int64_t)n0 * g.ldw, (rows_w - 1) * (int)g.ldw + g.k);
  // NT = 2: a wave reads its weight rows in the order 8 (r / 4) + 4 i + r % 4,
  // so that a lane's results are 8 neighbouring n; the exchange of pieces
  // goes by bits 0, 1 and 3 of the row then, by bits 0..2 otherwise
  const int pca = ((lane & 7) ^ lrow) * 16;
  const int pcw = NT == 2 ? ((lane & 7) ^ (lrow & 3) ^ ((wave & 1) << 2)) * 16 : pca;
  const unsigned va = (unsigned)((wave * 8 + lrow) * (int)g.lda + pca), vw = (unsigned)((wave * 8 + lrow) * (int)g.ldw + pcw);
  const int last = (kb1 - 1) * kQBlk;
  constexpr int kSB = E8 ? 1 : 4;
  const TileSrc rs =
      wave == 2 ? tile_src(static_cast<const uint8_t*>(g.w_scales) + (int64_t)(n0 / kQBlk) * g.nkb * kSB, g.nkb * kSB)
                : tile_src(static_cast<const uint8_t*>(g.a_scales) + (int64_t)m0 * g.nkb * kSB, rows_a * g.nkb * kSB);
  const unsigned vs = wave < 2 ? (unsigned)((wave * 64 + lane) * g.nkb * kSB) : wave == 2 && lane == 0 ? 0u : kNoLoad;
  // Past the last step, and rows past the tile, the loads give zeros: their
  // number per step is constant.
  auto fill = [&](int kb, int slot) {
    const int kk = min(kb * kQBlk, last);
    const uint32_t at = lds_ring + (uint32_t)(slot * kBytes);
    const bool ia = kb < kb1 && kb * kQBlk + pca < g.k, iw = kb < kb1 && kb * kQBlk + pcw < g.k;
#pragma unroll
    for (int i = 0; i < LW; ++i)
      load_lds16(rw, at + (uint32_t)(wave + WAVES * i) * 1024, iw ? vw + 8 * WAVES * i * (unsigned)g.ldw : kNoLoad, kk);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      // 16 rows: two waves' worth; the others' zeros go where nobody reads
      const bool mine = BM >= 8 * WAVES || wave < BM / 8;
      load_lds16(ra, mine ? at + (uint32_t)(BN * kQBlk + (wave + WAVES * i) * 1024) : lds_spare,
                 ia && mine ? va + 8 * WAVES * i * (unsigned)g.lda : kNoLoad, kk);
    }
    load_lds_word<kSB>(rs, at + (uint32_t)(kScales + min(wave, 3) * 256), vs, min(kb, kb1 - 1) * kSB);
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < kRing - 1; ++t) fill(kb0 + t, t);
  int slot = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    // newer than this step's loads: those of kRing - 2 steps.  After the
    // barrier everyone's have landed and the last step's slot has been read.
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"(kLoads * (kRing - 2)) : "memory");
    const uint8_t* lw = ring[slot];
    const uint32_t* ls = reinterpret_cast<const uint32_t*>(lw + kScales);
    i32x8 fw[NT], fa[MT];
    uint32_t sa[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
      fw[i] = NT == 2 ? frag(lw, wn + (i16 >> 2) * 8 + i * 4 + (i16 & 3), (i16 & 3) | (i16 & 4), q)
                      : frag(lw, wn + i16, i16 & 7, q);
    const uint32_t sw = ls[128];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      fa[j] = frag(lw + BN * kQBlk, wm + j * 16 + i16, i16 & 7, q);
      sa[j] = ls[wm + j * 16 + i16];
    }
    fill(kb + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const float f = kHwScale ? 0.0f : scale_value<E8>(sa[j]) * scale_value<E8>(sw);
      f32x4 p[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (kHwScale) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[i], fa[j], acc[i][j], 0, 0, 0, (int)sw, 0, (int)sa[j]);
        } else {
          p[i] = f32x4{0, 0, 0, 0};
          if constexpr (kWide) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              p[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fw[i], u), widen(fa[j], u), p[i], 0, 0, 0);
          } else {
            p[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[i], fa[j], p[i], 0, 0, 0, 0, 0, 0);
          }
        }
      }
      if constexpr (!kHwScale) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[i][e], f, acc[i][j][e]);
      }
    }
    slot = slot + 1 == kRing ? 0 : slot + 1;
    // the barrier above must find this step's reads done
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  // no load may be in flight into LDS when the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm + j * 16 + i16;
    if (m >= g.rows) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = n0 + wn + q * 4 * NT + i * 4;
      if (n >= g.n) continue;
      if (gridDim.y > 1) store4<float>(g.partial + ((int64_t)blockIdx.y * g.rows + m) * g.n + n, g.n - n, acc[i][j]);
      else store4<TO>(static_cast<TO*>(g.y) + (int64_t)m * g.ldy + n, g.n - n, acc[i][j]);
    }
  }
}

// y = the splits' partial results added in order.
template <typename TO>
__global__ __launch_bounds__(256) void matmul_join_kernel(MatmulArgs g, int splits) {
  const int64_t total = (int64_t)g.rows * g.n;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    float s = 0.0f;
    for (int p = 0; p < splits; ++p) s += g.partial[p * total + e];
    const int64_t m = e / g.n;
    store1(static_cast<TO*>(g.y) + m * g.ldy + (e - m * g.n), s);
  }
}

// Which kernel, from sizes alone (the workspace depends on it).  Both sides at
// the borders:
//   few    weights of up to 2^25 codes, see matmul_few_kernel
//   big    from 160 tiles: 1024 x 13824 x 5120 (216) 77 us, kMany 106
//   batch  64 x 64 tiles that all fit at once: 256 x 4096 x 4096 15 us, kMid 30
//   mid    128 x 128 tiles that all fit: 1024 x 4096 x 4096 25 us, kMany 44;
//          at 432 tiles, two rounds, 71 against kMany's 53
enum class Way { kFew, kBatch, kMid, kMany, kBig };
Way way_of(int64_t rows, int64_t n, int64_t k, bool wide) {
  if (rows <= 16 && k >= 16 && n * k <= (1 << 25)) return Way::kFew;
  const int64_t big = ((rows + 255) / 256) * ((n + 255) / 256);
  if (!wide && rows > 128 && k > kQBlk && big >= 160) return Way::kBig;
  if (rows <= 128 || ((rows + 63) / 64) * ((n + 63) / 64) <= 256) return Way::kBatch;
  return ((rows + 127) / 128) * ((n + 127) / 128) <= 256 ? Way::kMid : Way::kMany;
}
// Rows of a tile of matmul_ring_kernel in the batch way.
int batch_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || rows > 128 ? 64 : 128; }

// The reduction is split into as many parts as the compute units can take at
// once, of 4 blocks at least: another round costs more than the idle units
// (64 x 13824 x 5120: whole 19 us, in two 24 us and 4 to join).
int split(int64_t tiles, int64_t nkb) {
  const int64_t s = std::max<int64_t>(1, std::min(std::min<int64_t>(256 / tiles, nkb / 4), (int64_t)16));
  const int64_t per = (nkb + s - 1) / s;
  return (int)((nkb + per - 1) / per);
}
int splits_of(int64_t rows, int64_t n, int64_t k, bool wide) {
  switch (way_of(rows, n, k, wide)) {
    case Way::kBatch: return split(((rows + batch_rows(rows) - 1) / batch_rows(rows)) * ((n + 63) / 64), q_nblk(k));
    case Way::kMid: return split(((rows + 127) / 128) * ((n + 127) / 128), q_nblk(k));
    default: return 1;
  }
}

// Rows of whole, aligned 16-byte pieces whose tiles stay within a descriptor's
// 2 GiB.
bool direct_ok(const MatmulArgs& g) {
  return ((reinterpret_cast<uintptr_t>(g.a) | reinterpret_cast<uintptr_t>(g.w) | (uintptr_t)g.lda | (uintptr_t)g.ldw |
           (uintptr_t)g.k) & 15) == 0 && g.lda <= (1 << 22) && g.ldw <= (1 << 22);
}

template <int MT, int MW, int NW, int NT, bool E8, typename TO, Rows kRows>
void tile_go(const MatmulArgs& g, int splits, hipStream_t stream) {
  constexpr int BM = 16 * MT * MW, BN = 16 * NT * NW;
  const int tm = (g.rows + BM - 1) / BM, tn = (g.n + BN - 1) / BN, per = (g.nkb + splits - 1) / splits;
  hipLaunchKernelGGL((matmul_tile_kernel<MT, MW, NW, NT, E8, TO, kRows>), dim3(tm * tn, splits), dim3(64 * MW * NW), 0,
                     stream, g, per, tm, tn);
}

template <int NT, bool E8, typename TO>
void few_go(const MatmulArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((matmul_few_kernel<NT, E8, TO>), dim3((g.n + 16 * NT - 1) / (16 * NT), (g.rows + 15) / 16), dim3(512), 0,
                     stream, g, (g.nkb + 7) / 8);
}

template <int MT, int NT, int WM, int WN, bool E8, typename TO>
void ring_go(const MatmulArgs& g, int splits, hipStream_t stream) {
  constexpr int BM = 16 * MT * WM, BN = 16 * NT * WN;
  const int tm = (g.rows + BM - 1) / BM, tn = (g.n + BN - 1) / BN, per = (g.nkb + splits - 1) / splits;
  for (int first = 0; first < tm * tn; first += kTilesPerLaunch)
    hipLaunchKernelGGL((matmul_ring_kernel<MT, NT, WM, WN, E8, TO>), dim3(std::min(tm * tn - first, kTilesPerLaunch), splits),
                       dim3(64 * WM * WN), 0, stream, g, per, tm, tn, first);
}

template <bool E8, typename TO>
hipError_t matmul_go(const MatmulArgs& g, hipStream_t stream) {
  constexpr bool kWide = sizeof(TO) == 4;
  const int s = splits_of(g.rows, g.n, g.k, kWide);
  const Way way = way_of(g.rows, g.n, g.k, kWide);
  const bool near = g.lda <= (1 << 22) && g.ldw <= (1 << 22);
  if (way == Way::kFew && near) {
    few_go<1, E8, TO>(g, stream);
  } else if (!direct_ok(g)) {
    // rows that are no whole pieces: the few-rows form reads its weight faster
    // (its 512 threads per 32 columns make one launch up to 2^27)
    if (s == 1 && near && g.k >= 16 && g.rows <= 16 && g.n <= (1 << 27)) few_go<2, E8, TO>(g, stream);
    else if (near && g.k >= 16) tile_go<4, 2, 2, 4, E8, TO, kCut>(g, s, stream);
    else tile_go<4, 2, 2, 4, E8, TO, kNarrow>(g, s, stream);
  } else if (way == Way::kBig) {
    const int tm = (g.rows + 255) / 256, tn = (g.n + 255) / 256;
    const bool whole_y = ((reinterpret_cast<uintptr_t>(g.y) | (uintptr_t)(g.ldy * 2) | (uintptr_t)(g.n * 2)) & 15) == 0 &&
                         g.ldy <= (1 << 21);  // 256 rows of 2-byte results end before kNoLoad
    hipLaunchKernelGGL((matmul_big_kernel<E8>), dim3(std::min(tm * tn, 256)), dim3(512), 0, stream, g, tm, tn, whole_y);
  } else if (way == Way::kMid) {
    ring_go<4, 2, 2, 4, E8, TO>(g, s, stream);
  } else if (way == Way::kMany) {
    if ((int64_t)((g.rows + 127) / 128) * ((g.n + 127) / 128) < 384) tile_go<2, 2, 2, 4, E8, TO, kWhole>(g, s, stream);
    else tile_go<4, 2, 2, 4, E8, TO, kWhole>(g, s, stream);
  } else {
    switch (batch_rows(g.rows)) {
      case 16: ring_go<1, 1, 1, 4, E8, TO>(g, s, stream); break;
      case 32: ring_go<2, 1, 1, 4, E8, TO>(g, s, stream); break;
      case 64: ring_go<4, 1, 1, 4, E8, TO>(g, s, stream); break;
      default: ring_go<8, 1, 1, 4, E8, TO>(g, s, stream);
    }
  }
  if (s > 1) {
    const int64_t wg = ((int64_t)g.rows * g.n + 255) / 256;
    hipLaunchKernelGGL((matmul_join_kernel<TO>), dim3((unsigned)(wg < 4096 ? wg : 4096)), dim3(256), 0, stream, g, s);
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_q8_workspace(int64_t rows, int64_t n, int64_t k) {
  if (rows == 0) return 0;
  const int s = std::max(splits_of(rows, n, k, false), splits_of(rows, n, k, true));
  return s > 1 ? (int64_t)s * rows * n * 4 : 0;
}

hipError_t launch_matmul_q8(const MatmulArgs& g, bool e8, DT out, hipStream_t stream) {
  if (out == DT::F32) return e8 ? matmul_go<true, float>(g, stream) : matmul_go<false, float>(g, stream);
  return e8 ? matmul_go<true, uint16_t>(g, stream) : matmul_go<false, uint16_t>(g, stream);
}

}  // namespace harp
