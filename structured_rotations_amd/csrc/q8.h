// The 8-bit operators: E4M3 codes with one fp32 or E8M0 scale per block of
// 128 columns.  Device helpers of the format, and the host launchers that the
// C entry points call after every argument has been checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "kernels.h"

namespace harp {

constexpr int kQBlk = 128;            // columns (and rows of a weight) per scale
constexpr float kQTop = 448.0f;       // largest E4M3 value
constexpr float kQFloor = 0x1p-120f;  // smallest scale: 1 / scale stays finite

inline int64_t q_nblk(int64_t n) { return (n + kQBlk - 1) / kQBlk; }

// ------------------------------------------------------------ device side
// Eight consecutive values of a row at their own alignment: gfx950 takes
// dword-wide global accesses at any address, so one path serves every row
// stride and base.
struct __attribute__((packed, aligned(2))) Raw8H { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Raw8F { uint32_t w[8]; };
struct __attribute__((packed, aligned(1))) Raw8C { uint32_t w[2]; };

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  Raw8H r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16x2_hw(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<Raw8H*>(p) = r;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  Raw8F r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
  *reinterpret_cast<Raw8F*>(p) = r;
}
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2_hw(v, v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// The first n values of a chunk.
template <typename T>
__device__ __forceinline__ void store8_tail(T* p, int n, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1(p + i, v[i]);
}
template <typename T>
__device__ __forceinline__ void store8_of(T* p, int n, const float (&v)[8]) {
  if (n >= 8) store8(p, v);
  else store8_tail<T>(p, n, v);
}

// Two of four codes as bf16, times the power of two whose E8M0 byte is the
// exponent field of `scale`.
__device__ __forceinline__ uint32_t widen2(uint32_t codes, uint32_t scale, bool hi) {
  const bf16x2_t v = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, __uint_as_float(scale), true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, __uint_as_float(scale), false);
  uint32_t w;
  __builtin_memcpy(&w, &v, 4);
  return w;
}
struct __attribute__((packed, aligned(1))) Raw16 { uint32_t w[4]; };

// 16 bytes of a row, the ones past its end (n) zero.
__device__ __forceinline__ u32x4 load16_bytes(const uint8_t* p, int n) {
  u32x4 v = {0, 0, 0, 0};
  if (n >= 16) {
    const Raw16 r = *reinterpret_cast<const Raw16*>(p);
    v = u32x4{r.w[0], r.w[1], r.w[2], r.w[3]};
  } else {
    for (int i = 0; i < n; ++i) {
      const uint32_t b = (uint32_t)p[i] << (8 * (i & 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] |= (i >> 2) == j ? b : 0u;
    }
  }
  return v;
}

// v's bytes from number `by` on (0..15), zeros behind them.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int by) {
  if (by & 8) v = u32x4{v[2], v[3], 0, 0};
  if (by & 4) v = u32x4{v[1], v[2], v[3], 0};
  const int b = 8 * (by & 3);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (uint32_t)((((uint64_t)(i < 3 ? v[i + 1] : 0) << 32) | v[i]) >> b);
  return v;
}

// Four E4M3 codes of four values (round to nearest, ties to even; the inputs
// are within 448 up to an fp32 rounding, which rounds to 448).
__device__ __forceinline__ uint32_t enc4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// Four values of four E4M3 codes (exact).
__device__ __forceinline__ void dec4(uint32_t w, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}
// Eight values as they are in memory, and what they are.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 8) {
      const Raw8H r = *reinterpret_cast<const Raw8H*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void fill(uint32_t bits) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bits >> 16 | (bits & 0xffff0000u);
  }
  __device__ __forceinline__ float operator[](int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};
template <>
struct Raw8<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 8) {
      const Raw8F r = *reinterpret_cast<const Raw8F*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = r.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
    }
  }
  __device__ __forceinline__ void fill(uint32_t bits) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bits;
  }
  __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(w[i]); }
};
struct RawCodes {
  uint32_t w[2];
  __device__ __forceinline__ void load(const uint8_t* p, int n) {
    if (n >= 8) {
      const Raw8C r = *reinterpret_cast<const Raw8C*>(p);
      w[0] = r.w[0];
      w[1] = r.w[1];
    } else {
      w[0] = w[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    dec4(w[0], v);
    dec4(w[1], v + 4);
  }
};
__device__ __forceinline__ void store8_codes(uint8_t* p, int n, const float (&v)[8]) {
  Raw8C r;
  r.w[0] = enc4(v[0], v[1], v[2], v[3]);
  r.w[1] = enc4(v[4], v[5], v[6], v[7]);
  if (n >= 8) {
    *reinterpret_cast<Raw8C*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint8_t)(r.w[i >> 2] >> (8 * (i & 3)));
  }
}

// Coding of values v = w * mult (mult: the row's 1/rms, or 1) that share a
// block whose largest |w| has the bits amax (as bits, NaN and infinity are the
// largest): `scale` is the block's scale, code8 turns eight w into values to
// be rounded to codes.
//
// fp32 scales: code = 448 w / max|w|.  mult cancels, and the quotient is
// corrected by its remainder, so that values that lie half way between two
// codes (common: w is a sum of bf16 values, with few bits) are exactly there
// and go to the even code.  448 is kept as 0.4375 * 2^10, so that nothing
// overflows for any fp32 w.
// E8M0 scales: code = (w * mult) / scale, one rounding.
template <bool E8>
struct Coder {
  float scale, num, den, rcp, cor;

  __device__ __forceinline__ Coder(uint32_t amax, float mult) {
    const float top = __uint_as_float(amax);
    float s = fmaxf(top * mult / kQTop, kQFloor);
    if constexpr (E8) s = __uint_as_float((__float_as_uint(s) + 0x007fffffu) & 0x7f800000u);  // up to a power of two
    const bool bad = amax >= 0x7f800000u || !(top * mult < __uint_as_float(0x7f800000u));
    scale = bad ? __uint_as_float(0x7fc00000u) : s;
    num = 0.4375f;
    den = fmaxf(top, kQTop * kQFloor / mult) * 0x1p-10f;
    rcp = cor = 1.0f / den;
    // far from every normal row's range: no correction
    if (E8 || bad || !(mult >= 0x1p-60f && mult <= 0x1p60f && den >= 0x1p-100f)) {
      num = bad ? scale : mult;
      den = cor = 0.0f;
      rcp = 1.0f / s;
    }
  }
  __device__ __forceinline__ void code8(const float (&w)[8], float (&c)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = w[i] * num;
      const float y = t * rcp;
      if constexpr (E8) c[i] = y;
      else c[i] = fmaf(fmaf(-y, den, t), cor, y);
    }
  }
};
template <bool E8>
__device__ __forceinline__ void store_scale(void* scales, int64_t i, float s) {
  if constexpr (E8) static_cast<uint8_t*>(scales)[i] = s != s ? 255 : (uint8_t)(__float_as_uint(s) >> 23);
  else static_cast<float*>(scales)[i] = s;
}
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}
template <bool E8>
__device__ __forceinline__ float load_scale(const void* scales, int64_t i) {
  if constexpr (E8) return e8m0_value(static_cast<const uint8_t*>(scales)[i]);
  else return static_cast<const float*>(scales)[i];
}

// A tile in global memory whose loads go straight into LDS: 16 bytes per
// lane, from the lane's byte offset plus a common one to 1024 consecutive
// bytes of LDS at a wave-uniform address.  Lanes at or beyond `bytes` give
// zeros.  Written out, because the compiler would wait for such a load before
// any later LDS read, of the other buffer too; the kernels wait for all of
// them (vmcnt) before the barrier that precedes their first use.
using TileSrc = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ TileSrc tile_src(const void* base, int bytes) {
  // both are the same in every lane; said so, or the loads may loop over lanes
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  base = reinterpret_cast<const void*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)at) |
                                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) << 32);
  bytes = __builtin_amdgcn_readfirstlane(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ uint32_t lds_address(const void* lds) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds;
}
__device__ __forceinline__ void load_lds16(TileSrc src, uint32_t lds, unsigned lane_offset, int offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(lane_offset), "s"(src),
                 "s"(__builtin_amdgcn_readfirstlane(offset))
               : "memory");
}
// The same for one word per lane: 4 bytes, or one byte widened.
template <int kBytes>
__device__ __forceinline__ void load_lds_word(TileSrc src, uint32_t lds, unsigned lane_offset, int offset) {
  const int at = __builtin_amdgcn_readfirstlane((int)lds), from = __builtin_amdgcn_readfirstlane(offset);
  if constexpr (kBytes == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(at), "v"(lane_offset), "s"(src), "s"(from)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                 :
                 : "s"(at), "v"(lane_offset), "s"(src), "s"(from)
                 : "memory");
}
// Loads of such a tile into registers.
__device__ __forceinline__ u32x4 load_16(TileSrc src, unsigned lane_offset) {
  return __builtin_amdgcn_raw_buffer_load_b128(src, lane_offset, 0, 0);
}
template <int kBytes>
__device__ __forceinline__ uint32_t load_word(TileSrc src, unsigned lane_offset) {
  if constexpr (kBytes == 4) return __builtin_amdgcn_raw_buffer_load_b32(src, lane_offset, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b8(src, lane_offset, 0, 0);
}

__device__ __forceinline__ void store_16(TileSrc dst, unsigned lane_offset, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, dst, lane_offset, 0, 0);
}

// How a product's rows are brought in.  kWhole: 16-byte aligned rows of whole
// 16-byte pieces, straight into LDS.  kCut: any alignment and length of 16
// bytes or more, through registers; the piece that a row's end cuts is loaded
// from 16 bytes before the end and shifted.  kNarrow: shorter rows, or strides
// beyond a descriptor, by elements.
enum Rows { kWhole, kCut, kNarrow };

// Which tile a workgroup computes: consecutive workgroups go to the 8 dies in
// turn, so each die takes one contiguous run of the tiles, ordered in groups
// of 8 tiles along m, and its 32 compute units share 8 + 4 panels in its L2.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int total = tiles_m * tiles_n, xcd = id & 7, q = total >> 3, r = total & 7;
  const int t = xcd * q + min(xcd, r) + (id >> 3);
  constexpr int kGroup = 8;
  const int per = kGroup * tiles_n, g = t / per, first = g * kGroup;
  const int gm = min(kGroup, tiles_m - first), in = t - g * per;
  // (the division is done per lane; the result is the same in all of them)
  *tn = __builtin_amdgcn_readfirstlane(in / gm);
  *tm = __builtin_amdgcn_readfirstlane(first + in - in / gm * gm);
}

// Tiles of one launch: its threads along x have to be less than 2^32, or it is
// refused or leaves out tiles; 2^30 columns by tiles of 64 and 256 threads are
// more.
constexpr int kTilesPerLaunch = 1 << 23;

// Lane offset that is beyond any tile.
constexpr unsigned kNoLoad = 0x7fffff00u;

// A scale as it is stored (E8M0: its byte), and its value.
template <bool E8>
__device__ __forceinline__ uint32_t scale_bits(const void* scales, int64_t i) {
  if constexpr (E8) return static_cast<const uint8_t*>(scales)[i];
  else return static_cast<const uint32_t*>(scales)[i];
}
template <bool E8>
__device__ __forceinline__ float scale_value(uint32_t bits) {
  return E8 ? e8m0_value(bits) : __uint_as_float(bits);
}

// Largest / sum over the 16 lanes that share a block (one DPP row), in every
// lane of it.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  return max(v, row_ror<1>(v));
}
__device__ __forceinline__ float row16_sum(float v) {
  v += __uint_as_float(row_ror<8>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<4>(__float_as_uint(v)));
  v += __uint_as_float(row_ror<2>(__float_as_uint(v)));
  return v + __uint_as_float(row_ror<1>(__float_as_uint(v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// -------------------------------------------------------------- host side
struct NormArgs {
  const void *x, *residual, *gamma;
  void* h;
  uint8_t *codes, *ckpt;
  void *scales, *ckpt_scales;
  float* rstd;
  int64_t ldx, ldr, ldh, ldc, ldk, rows;
  int d;
  float eps;
};
struct NormVjpArgs {
  const uint8_t* codes;
  const void *scales, *gamma, *dn, *dres;
  const float* rstd;
  void* dh;
  float *dgamma, *partial;
  int64_t ldc, lddn, lddres, lddh, rows;
  int d;
};
struct MatmulArgs {
  const uint8_t *a, *w;
  const void *a_scales, *w_scales;
  void* y;
  float* partial;
  int64_t lda, ldw, ldy;
  int rows, n, k, nkb;
};
struct WgradArgs {
  const uint16_t* dy;
  const uint8_t* x;
  const void* x_scales;
  void* dw;
  float* partial;
  int64_t lddy, ldx, lddw;
  int rows, n, k, nkb;
};

hipError_t launch_quantize_q8(const void* x, int64_t ldx, DT io, int64_t rows, int cols, bool tile, uint8_t* codes,
                              int64_t ldc, void* scales, bool e8, hipStream_t stream);
hipError_t launch_rmsnorm_q8(const NormArgs& a, DT io, bool e8, hipStream_t stream);
int64_t rmsnorm_q8_vjp_workspace(int64_t rows, int64_t d);
hipError_t launch_rmsnorm_q8_vjp(const NormVjpArgs& a, DT io, bool e8, hipStream_t stream);
int64_t matmul_q8_workspace(int64_t rows, int64_t n, int64_t k);
hipError_t launch_matmul_q8(const MatmulArgs& a, bool e8, DT out, hipStream_t stream);
int64_t matmul_q8_wgrad_workspace(int64_t rows, int64_t n, int64_t k);
hipError_t launch_matmul_q8_wgrad(const WgradArgs& a, bool e8, DT out, hipStream_t stream);

}  // namespace harp
