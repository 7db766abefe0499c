// dW = dY^T X with X from an 8-bit checkpoint, on the bf16 matrix
// instructions.
//
//   dw[n][k] = sum_m dy[m][n] s[m][k/128] c[m][k]
//
// The scale changes along the reduction, so x is decoded before the product.
// A code has 4 significant bits: times a power of two (E8M0) it is exact in
// bf16 and so is every product.  Times an fp32 scale it has up to 28 bits, and
// x is a sum of bf16 parts, one product each: three parts (24 bits) for fp32
// results, one for bf16 results, which adds an error as large as the result's
// own rounding (in all 2.35e-3 of the result where that alone is 1.66e-3; x's
// codes are off by 2^-5 of it).  Two parts take 69 us instead of 40 at
// 1500 x 4099 x 1037 and 1158 instead of 465 at 16384 x 4096 x 4096; who wants
// them asks for an fp32 result.  Up to one step of rows, where writing dw bounds
// the time, bf16 results take two parts.
//
// Both operands are stored along the other axis than the one summed over:
// they stay that way in LDS ([m][n], [m][k]) and the transposing LDS read
// (ds_read_b64_tr_b16) gives a lane its neighbouring m.
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace harp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;  // rows (m) per step, two instructions' worth

// LDS tile of kStep rows of W bf16 values: 32-byte segments exchanged by the
// row's number, so that the 16 rows of a fragment read cover all banks.
template <int W>
__device__ __forceinline__ int seg_off(int row, int seg) {
  return row * W * 2 + ((seg ^ (((row & 3) | (row >> 1 & 12)) & (W / 16 - 1))) << 5);
}

// Offset of lane (q, i16)'s part of the first column segment of a wave
// (`first`, a multiple of the segments it reads) in a fragment read; segment
// first + f is at this ^ 32 f.
template <int W>
__device__ __forceinline__ uint32_t frag_base(int first, int lane) {
  return (uint32_t)(seg_off<W>(8 * (lane >> 4) + ((lane & 15) >> 2), first) + (lane & 3) * 8);
}
// Half of the 8 values m = 32 sub + 8q .. + 7 of column i16 of segment f: 4h .. + 3.
template <int W>
__device__ __forceinline__ s16x4 frag_half(const uint8_t* lds, uint32_t base, int sub, int f, int h) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(lds + (base ^ (uint32_t)(f << 5)) + (32 * sub + 4 * h) * W * 2));
}
__device__ __forceinline__ bf16x8_t frag_of(const s16x4 (&v)[2]) {
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

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

// acc += a b.  kAcc: the accumulators are named as accumulation registers (a
// wave that has 256 of them leaves the compiler no other place, and left to
// itself it moves them about in the loop).  Nothing reads or writes one again
// before 32 more instructions or settle().  The factors come from LDS reads, for
// which the compiler waits; a vector instruction that wrote one would have to be
// two wait states earlier, and the built code has none.
template <bool kAcc>
__device__ __forceinline__ void mfma(f32x4& acc, bf16x8_t a, bf16x8_t b) {
  if constexpr (kAcc) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  else acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
// Lets the accumulators' last writes arrive: the zeros' and the matrix
// instructions'.  They are operands on both sides of the wait: nothing else
// keeps the compiler, which sees no matrix instruction here, from moving an
// access to one across it.
template <bool kAcc, int NI, int NJ>
__device__ __forceinline__ void settle(f32x4 (&acc)[NI][NJ]) {
  if constexpr (!kAcc) return;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    if (t == 0) asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  }
}

// Two values as PARTS bf16 parts each, handed to put(part, pair).  Parts are
// cut off towards zero and the last one is rounded, so all have the value's
// sign and none overflows; what a cut leaves is exact, and three parts hold all
// 24 bits.  Every part is multiplied by dy on its own, and dy may be infinite or
// its first product overflow: a later part of the other sign, or 0, would make a
// NaN of that.  So what is left of a value v is brought between +-2^-126 (v
// itself if that is nearer to 0) and v, which adds at most 2^-126 times dy to an
// exact value; also after an infinity, whose rest is NaN, which the median
// leaves out.
template <int PARTS, typename F>
__device__ __forceinline__ void split_parts(float va, float vb, F put) {
  if constexpr (PARTS == 1) return put(0, pack_bf16x2_hw(va, vb));
  const float least_a = __builtin_amdgcn_fmed3f(va, 0x1p-126f, -0x1p-126f);
  const float least_b = __builtin_amdgcn_fmed3f(vb, 0x1p-126f, -0x1p-126f);
  float a = va, b = vb;
#pragma unroll
  for (int t = 0; t < PARTS - 1; ++t) {
    const uint32_t w = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
    put(t, w);
    a = __builtin_amdgcn_fmed3f(a - bf16_lo(w), least_a, va);
    b = __builtin_amdgcn_fmed3f(b - bf16_hi(w), least_b, vb);
  }
  put(PARTS - 1, pack_bf16x2_hw(a, b));
}

// One tile of dw per workgroup of 4 waves, each 16 NI (k) by 16 NJ (n) of it;
// PARTS: bf16 parts of x.  Per step of 64 rows a wave multiplies from
// registers (the fragments of half a step), while it
//   first half    reads the second half's fragments, then decodes the next
//                 step's rows, which are in registers, into the other buffer
//   second half   (after a barrier) reads the next step's first fragments and
//                 asks for the rows of the step after that.
// Global loads have a whole step to arrive.  Bound by the matrix instructions:
// 16384 x 4096 x 4096, E8M0, 414 to 426 us, 1.3 PFLOP/s, 0.84 of a plain bf16
// product's (4 by 4 fragments per wave, with twice the LDS reads per
// instruction: 608 us).
template <int NI, int NJ, bool E8, int PARTS, typename TO, Rows kRows>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 2))) void wgrad_tile_kernel(
    WgradArgs g, int m_per_split, int tiles_n, int tiles_k, int first_tile) {
  constexpr int BK = 32 * NI, BN = 32 * NJ, R = NI * PARTS;
  constexpr int UD = kStep * BN / 8 / 256, UX = kStep * BK / 16 / 256;  // pieces per thread: 8 of dy, 16 of x
  __shared__ __align__(16) uint8_t ld[2][kStep * BN * 2];
  const uint32_t lds_d = lds_address(ld);
  __shared__ __align__(16) uint8_t lx[PARTS][2][kStep * BK * 2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tn, tk;
  tile_of(first_tile + (int)blockIdx.x, tiles_n, tiles_k, &tn, &tk);
  const int k0 = tk * BK, n0 = tn * BN;
  const int wk = (wave & 1) * NI, wn = (wave >> 1) * NJ;  // in segments of 16
  const int mlo = (int)blockIdx.y * m_per_split, mhi = min(g.rows, mlo + m_per_split);

  // Columns past the end give results that are not stored.  Rows past the end
  // are past the descriptors' ends, too, and give zeros.
  // dy, kWhole: load u of wave w brings rows (w << 3) + the bits of u in bits
  // (1,) 2 and 5 + the lane's, so that the exchange of segments depends on u
  // in bit 1 only.
  constexpr int kRowsD = 512 / BN;  // rows of dy per load of a wave
  unsigned vdd[2];
  if constexpr (kRows == kWhole) {
    const int lr = lane / (BN / 8), pp = lane % (BN / 8);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int row = wave * 8 + lr + (kRowsD == 2 ? 2 * t : 0);
      const int x = ((row & 3) | (row >> 1 & 12)) & (BN / 16 - 1);
      const int col = ((pp >> 1) ^ x) * 16 + (pp & 1) * 8;
      vdd[t] = n0 + col < g.n ? (unsigned)(row * (int)g.lddy + col) * 2u : kNoLoad;
    }
  }
  auto row_of_load = [](int u) { return kRowsD == 2 ? (u >> 1 & 1) * 4 + (u >> 2) * 32 : (u & 1) * 4 + (u >> 1) * 32; };
  // the others: piece of 8 columns (dy) or 16 (x) of a thread's rows
  const int dcol = tid % (BN / 8) * 8, xcol = tid % (BK / 16) * 16;
  const int drow = tid / (BN / 8), xrow = tid / (BK / 16);
  const int dn = g.n - n0 - dcol, xn = g.k - k0 - xcol;
  const int cut_d = kRows == kCut && dn > 0 && dn < 8 ? 16 - 2 * dn : 0, cut_x = kRows == kCut && xn > 0 && xn < 16 ? 16 - xn : 0;
  constexpr int kSB = E8 ? 1 : 4;
  unsigned vd, vx, vs;
  if constexpr (kRows != kNarrow) {
    vd = dn > 0 ? (unsigned)((drow * (int)g.lddy + dcol) * 2 - cut_d) : kNoLoad;
    vx = xn > 0 ? (unsigned)(xrow * (int)g.ldx + xcol - cut_x) : kNoLoad;
    vs = xn > 0 ? (unsigned)(xrow * g.nkb + (k0 + xcol) / kQBlk) * kSB : kNoLoad;
  }

  // rows of the next steps, as they come: of one step for the large tile, whose
  // steps are long, of two for the small one
  constexpr int kSets = kRows == kCut && NI * NJ * 4 <= 64 ? 2 : 1;
  u32x4 rd[kSets][UD], rx[kSets][UX];
  uint32_t rs[kSets][UX];
  // descriptors of a step's rows; they begin with the row, not the tile, so
  // that a shifted piece of the first columns is inside
  auto rows_left = [&](int m0) { return max(0, min(mhi - m0, kStep)); };
  auto src_dy = [&](int m0) {
    const int left = kRows == kNarrow ? 0 : rows_left(m0);
    return tile_src(g.dy + (int64_t)(left ? m0 : mlo) * g.lddy, left ? ((left - 1) * (int)g.lddy + g.n) * 2 : 0);
  };
  auto src_x = [&](int m0) {
    const int left = kRows == kNarrow ? 0 : rows_left(m0);
    return tile_src(g.x + (int64_t)(left ? m0 : mlo) * g.ldx, left ? (left - 1) * (int)g.ldx + g.k : 0);
  };
  auto src_s = [&](int m0) {
    const int left = kRows == kNarrow ? 0 : rows_left(m0);
    return tile_src(static_cast<const uint8_t*>(g.x_scales) + (int64_t)(left ? m0 : mlo) * g.nkb * kSB, left * g.nkb * kSB);
  };
  auto bring_dy = [&](TileSrc src, int buf, int u) {
    const unsigned v = vdd[kRowsD == 2 ? u & 1 : 0];
    const int row = row_of_load(u) + (kRowsD == 2 ? (u & 1) * 2 : 0);
    load_lds16(src, lds_d + (uint32_t)((buf * kStep + row + wave * 8) * BN * 2), v + (unsigned)(n0 * 2 + row_of_load(u) * (int)g.lddy * 2), 0);
  };
  auto load_dy = [&](int set, TileSrc src, int m0, int u) {
    const int r = u * (2048 / BN);
    if constexpr (kRows == kCut) rd[set][u] = load_16(src, vd + (unsigned)(n0 * 2 + r * (int)g.lddy * 2));
    else if constexpr (kRows == kNarrow)
      rd[set][u] = load16_bytes(reinterpret_cast<const uint8_t*>(g.dy + (int64_t)(m0 + drow + r) * g.lddy + n0 + dcol),
                                m0 + drow + r < mhi ? min(dn, 8) * 2 : 0);  // dn is up to 2^30
  };
  auto load_x = [&](int set, TileSrc src, TileSrc scales, int m0, int u) {
    const int r = u * (4096 / BK);
    if constexpr (kRows == kNarrow) {
      rx[set][u] = load16_bytes(g.x + (int64_t)(m0 + xrow + r) * g.ldx + k0 + xcol, m0 + xrow + r < mhi ? xn : 0);
      const bool in = m0 + xrow + r < mhi && xn > 0;
      rs[set][u] = 0;
      if (in) rs[set][u] = scale_bits<E8>(g.x_scales, (int64_t)(m0 + xrow + r) * g.nkb + (k0 + xcol) / kQBlk);
    } else {
      rx[set][u] = load_16(src, vx + (unsigned)(k0 + r * (int)g.ldx));
      rs[set][u] = load_word<kSB>(scales, vs + (unsigned)(r * g.nkb * kSB));
    }
  };
  auto keep_dy = [&](int set, int buf, int u) {
    if constexpr (kRows != kWhole) {
      if (cut_d) rd[set][u] = shift_down(rd[set][u], cut_d);
      *reinterpret_cast<u32x4*>(ld[buf] + seg_off<BN>(drow + u * (2048 / BN), dcol >> 4) + (dcol & 8) * 2) = rd[set][u];
    }
  };
  static_assert(4096 / BK >= 16 || UX == 1 || (4096 / BK) % 8 == 0, "");
  uint32_t xat = (uint32_t)seg_off<BK>(xrow, xcol >> 4);
  // decodes piece u in five units: 4 codes each, then the writes
  u32x4 xw[PARTS][2];
  auto keep_x = [&](int set, int u, int c) {
    if (c < 4) {
      if (kRows == kCut && c == 0 && cut_x) rx[set][u] = shift_down(rx[set][u], cut_x);
      if constexpr (E8 && PARTS == 1) {
        xw[0][c >> 1][2 * (c & 1)] = widen2(rx[set][u][c], rs[set][u] << 23, false);
        xw[0][c >> 1][2 * (c & 1) + 1] = widen2(rx[set][u][c], rs[set][u] << 23, true);
      } else {
        const float s = scale_value<E8>(rs[set][u]);
        float v[4];
        dec4(rx[set][u][c], v);
#pragma unroll
        for (int e = 0; e < 2; ++e) split_parts<PARTS>(v[2 * e] * s, v[2 * e + 1] * s, [&](int t, uint32_t w) {
          xw[t][c >> 1][2 * (c & 1) + e] = w;
        });
      }
      return;
    }
    // bits 3 and 4 of the row, which u changes, exchange segments 4 and 8 apart
    constexpr int kUp = 4096 / BK;
    const uint32_t at = (xat ^ (uint32_t)(((u * kUp >> 1 & 12) & (BK / 16 - 1)) << 5)) + u * kUp * BK * 2;
    // odd pieces write their halves in the other order: eight lanes then fill
    // 128 different bytes
#pragma unroll
    for (int t = 0; t < PARTS; ++t) {
      const bool odd = tid & 1;
      const u32x4 lo = xw[t][0], hi = xw[t][1];
      u32x4 first, second;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        first[e] = odd ? hi[e] : lo[e];
        second[e] = odd ? lo[e] : hi[e];
      }
      *reinterpret_cast<u32x4*>(lx[t][0] + at + (odd ? 16 : 0)) = first;
      *reinterpret_cast<u32x4*>(lx[t][0] + at + (odd ? 0 : 16)) = second;
    }
  };

  constexpr bool kAcc = NI * NJ * 4 > 128;
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  s16x4 fr[2][NJ + R][2];  // fragments of two half steps: dy's, then x's
  // offsets of the buffer that is read; the other one is at ^ kFlip
  constexpr uint32_t kFlipD = kStep * BN * 2, kFlipX = kStep * BK * 2;
  uint32_t fbd = frag_base<BN>(wn, lane), fbx = frag_base<BK>(wk, lane);
  auto read_half = [&](int set, int sub, int u) {  // half u & 1 of fragment u / 2
    const int f = u >> 1, h = u & 1;
    if (f < NJ) fr[set][f][h] = frag_half<BN>(ld[0], fbd, sub, f, h);
    else fr[set][f][h] = frag_half<BK>(lx[(f - NJ) / NI][0], fbx, sub, (f - NJ) % NI, h);
  };
  // A half step is S instructions; the rest of the work goes between them, in
  // small units, since one wave per SIMD has nothing else to fill the gaps.
  constexpr int S = R * NJ, kReads = 2 * (R + NJ), kKeeps = (kRows == kWhole ? 0 : UD) + 5 * UX;
  constexpr int kAsks = UX + UD, kLate = S * 3 / 4;
  // the rows of step k are in set k % kSets until they are decoded
  auto step = [&](auto parity, int m0, int buf) {
    constexpr int set = kSets == 2 ? 1 - decltype(parity)::value : 0;
    // keeps the compiler from holding every segment's address in a register
    asm volatile("" : "+v"(fbd), "+v"(fbx), "+v"(xat));
#pragma unroll
    for (int t = 0; t < S; ++t) {
      if (t < S / 2) {
#pragma unroll
        for (int u = t * kReads / (S / 2); u < (t + 1) * kReads / (S / 2); ++u) read_half(1, 1, u);
      } else {
#pragma unroll
        for (int u = (t - S / 2) * kKeeps / (S / 2); u < (t + 1 - S / 2) * kKeeps / (S / 2); ++u) {
          if (u < 5 * UX) keep_x(set, u / 5, u % 5);
          else keep_dy(set, buf ^ 1, u - 5 * UX);
        }
      }
      mfma<kAcc>(acc[t / NJ % NI][t % NJ], frag_of(fr[0][NJ + t / NJ]), frag_of(fr[0][t % NJ]));
      __builtin_amdgcn_sched_barrier(0);
    }
    // this buffer has been read by every wave, the other one is complete
    if constexpr (kRows == kWhole) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fbd ^= kFlipD;
    fbx ^= kFlipX;
    xat ^= kFlipX;
    const int m2 = m0 + (kSets + 1) * kStep;
    const TileSrc sd = src_dy(m2), sx = src_x(m2), ss = src_s(m2);
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
      for (int u = t * kAsks / S; u < (t + 1) * kAsks / S; ++u) {
        if (u < UX) load_x(set, sx, ss, m2, u);
        else if (kRows == kWhole) bring_dy(sd, buf, u - UX);
        else load_dy(set, sd, m2, u - UX);
      }
      if (t < kLate) {
#pragma unroll
        for (int u = t * kReads / kLate; u < (t + 1) * kReads / kLate; ++u) read_half(0, 0, u);
      }
      mfma<kAcc>(acc[t / NJ % NI][t % NJ], frag_of(fr[1][NJ + t / NJ]), frag_of(fr[1][t % NJ]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (mlo < mhi) {
    const int m1 = mlo + kStep;
    [[maybe_unused]] const TileSrc sd0 = src_dy(mlo), sd1 = src_dy(m1);
#pragma unroll
    for (int u = 0; u < UD; ++u) {
      if constexpr (kRows == kWhole) {
        bring_dy(sd0, 0, u);
        bring_dy(sd1, 1, u);
      } else {
        load_dy(0, sd0, mlo, u);
      }
    }
#pragma unroll
    for (int u = 0; u < UX; ++u) load_x(0, src_x(mlo), src_s(mlo), mlo, u);
#pragma unroll
    for (int u = 0; u < UD; ++u) keep_dy(0, 0, u);
#pragma unroll
    for (int u = 0; u < 5 * UX; ++u) keep_x(0, u / 5, u % 5);
    xat ^= kFlipX;
#pragma unroll
    for (int k = 1; k <= kSets; ++k) {
      const int mk = mlo + k * kStep;
#pragma unroll
      for (int u = 0; u < UX; ++u) load_x(k % kSets, src_x(mk), src_s(mk), mk, u);
#pragma unroll
      for (int u = 0; u < UD; ++u) load_dy(k % kSets, src_dy(mk), mk, u);
    }
    if constexpr (kRows == kWhole) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int u = 0; u < kReads; ++u) read_half(0, 0, u);
    int buf = 0;
    settle<kAcc>(acc);
    for (int m0 = mlo; m0 < mhi; m0 += kSets * kStep) {
      step(std::integral_constant<int, 0>{}, m0, buf);
      buf ^= 1;
      if constexpr (kSets == 2) {  // past the last row: a step of zeros
        step(std::integral_constant<int, 1>{}, m0 + kStep, buf);
        buf ^= 1;
      }
    }
    settle<kAcc>(acc);
    // no load may be in flight into LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = n0 + (wn + j) * 16 + (lane & 15);
    if (n >= g.n) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = k0 + (wk + i) * 16 + (lane >> 4) * 4;
      if (k >= g.k) continue;
      if (gridDim.y > 1) store4<float>(g.partial + ((int64_t)blockIdx.y * g.n + n) * g.k + k, g.k - k, acc[i][j]);
      else store4<TO>(static_cast<TO*>(g.dw) + (int64_t)n * g.lddw + k, g.k - k, acc[i][j]);
    }
  }
}

template <typename TO>
__global__ __launch_bounds__(256) void wgrad_join_kernel(WgradArgs g, int splits) {
  const int64_t total = (int64_t)g.n * g.k;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    float s = 0.0f;
    for (int p = 0; p < splits; ++p) s += g.partial[p * total + e];
    const int64_t n = e / g.k;
    store1(static_cast<TO*>(g.dw) + n * g.lddw + (e - n * g.k), s);
  }
}

// Tiles along k of the two kinds, in segments of 32: (more parts of x: narrower).
constexpr int kBigK(int parts) { return parts == 1 ? 8 : parts == 2 ? 4 : 2; }
constexpr int kSmallK(int parts) { return parts == 1 ? 4 : 2; }

// The rows are split while 128 x 128 tiles leave compute units idle and every
// split keeps 4 steps (the workspace depends on sizes alone).  Without a split
// the tile is the large one (8 fragments of dy by kBigK of x per wave) if its
// rounds over the 256 compute units take less time than the small one's (4 by
// kSmallK): per round 2.7 times the small one's with one part, 1.8 with three.
// 4096 rows, n = 4096, one part: k = 2048 small 78 us, large 103 (one round of
// the large against two); k = 2304 118 and 104 (against three), 3328 147 and
// 107; 16384 x 4096 x 4096 608 and 421.  Three parts: k = 2048 222 and 204,
// 2560 278 and 304.  For few rows, which the stores of dw bound, the rule is not
// as good: 64 x 8192 x 4096, fp32 results, E8M0 40 and 46 (large taken), three
// parts 57 and 66; bf16 results 31 and 28.
struct WgradShape {
  bool big;
  int splits, m_per_split;
};
WgradShape wgrad_shape(int64_t rows, int64_t n, int64_t k, int parts) {
  auto tiles = [&](int64_t bn, int64_t bk) { return ((n + bn - 1) / bn) * ((k + bk - 1) / bk); };
  auto rounds = [&](int64_t bn, int64_t bk) { return (tiles(bn, bk) + 255) / 256; };
  const int64_t t = tiles(128, 128), steps = (rows + kStep - 1) / kStep;
  int64_t p = 1;
  while (t * p < 256 && p * 2 * 4 <= steps && p < 64) p *= 2;
  const int64_t per = (steps + p - 1) / p;
  WgradShape s;
  s.big = t >= 256 && (parts == 1 ? 8 : 6) * rounds(256, 32 * kBigK(parts)) <= 3 * rounds(128, 32 * kSmallK(parts));
  s.m_per_split = (int)(per * kStep);
  s.splits = per > 0 ? (int)((steps + per - 1) / per) : 1;
  return s;
}

template <int NI, int NJ, bool E8, int PARTS, typename TO, Rows kRows>
void wgrad_tile_go(const WgradArgs& g, const WgradShape& s, hipStream_t stream) {
  constexpr int BK = 32 * NI, BN = 32 * NJ;
  const int tn = (g.n + BN - 1) / BN, tk = (g.k + BK - 1) / BK;
  for (int first = 0; first < tn * tk; first += kTilesPerLaunch)
    hipLaunchKernelGGL((wgrad_tile_kernel<NI, NJ, E8, PARTS, TO, kRows>),
                       dim3(std::min(tn * tk - first, kTilesPerLaunch), s.splits), dim3(256), 0, stream, g,
                       s.m_per_split, tn, tk, first);
}

template <bool E8, int PARTS, typename TO>
hipError_t wgrad_go(const WgradArgs& g, hipStream_t stream) {
  const WgradShape s = wgrad_shape(g.rows, g.n, g.k, PARTS);
  const bool whole = ((reinterpret_cast<uintptr_t>(g.dy) | reinterpret_cast<uintptr_t>(g.x) | (uintptr_t)(g.lddy * 2) |
                       (uintptr_t)g.ldx | (uintptr_t)(g.n * 2) | (uintptr_t)g.k) & 15) == 0;
  // a descriptor holds 64 rows in 2 GiB
  const bool narrow = g.n < 8 || g.k < 16 || g.lddy > (1 << 22) || g.ldx > (1 << 22);
  if (narrow) wgrad_tile_go<kSmallK(PARTS), 4, E8, PARTS, TO, kNarrow>(g, s, stream);
  else if (s.big && whole) wgrad_tile_go<kBigK(PARTS), 8, E8, PARTS, TO, kWhole>(g, s, stream);
  else if (s.big) wgrad_tile_go<kBigK(PARTS), 8, E8, PARTS, TO, kCut>(g, s, stream);
  else wgrad_tile_go<kSmallK(PARTS), 4, E8, PARTS, TO, kCut>(g, s, stream);
  if (s.splits > 1) {
    const int64_t wg = ((int64_t)g.n * g.k + 255) / 256;
    hipLaunchKernelGGL((wgrad_join_kernel<TO>), dim3((unsigned)(wg < 4096 ? wg : 4096)), dim3(256), 0, stream, g,
                       s.splits);
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_q8_wgrad_workspace(int64_t rows, int64_t n, int64_t k) {
  const int s = wgrad_shape(rows, n, k, 1).splits;
  return s > 1 ? (int64_t)s * n * k * 4 : 0;
}

hipError_t launch_matmul_q8_wgrad(const WgradArgs& g, bool e8, DT out, hipStream_t stream) {
  if (out == DT::F32) return e8 ? wgrad_go<true, 1, float>(g, stream) : wgrad_go<false, 3, float>(g, stream);
  if (e8) return wgrad_go<true, 1, uint16_t>(g, stream);
  return g.rows <= kStep ? wgrad_go<false, 2, uint16_t>(g, stream) : wgrad_go<false, 1, uint16_t>(g, stream);
}

}  // namespace harp
