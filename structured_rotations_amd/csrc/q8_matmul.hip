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
#include "q8.h"

namespace harp {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kUnit = 0x7f7f7f7f;  // E8M0 1.0 in every byte

struct __attribute__((packed, aligned(1))) Raw16 { uint32_t w[4]; };

// 16 codes of a row, the ones past its end zero.
__device__ __forceinline__ u32x4 load16_codes(const uint8_t* p, int n) {
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

// A fragment: the two 16-byte pieces q and q + 4 of a 128-byte row in LDS,
// whose pieces are exchanged by the row's number (piece ^ (row & 7)) so that
// eight rows' reads of one piece cover all banks.
__device__ __forceinline__ i32x8 frag(const uint8_t* lds, int row, int q) {
  const uint8_t* p = lds + row * kQBlk;
  const i32x4 a = *reinterpret_cast<const i32x4*>(p + ((q ^ (row & 7)) << 4));
  const i32x4 b = *reinterpret_cast<const i32x4*>(p + (((q + 4) ^ (row & 7)) << 4));
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

// One BM x BN tile of y per workgroup of (BM / 64) (BN / 64) waves, each with
// 64 x 64 of it; one block of 128 per step through LDS.
template <int BM, int BN, bool E8, typename TO>
__global__ __launch_bounds__(BM * BN / 64) void matmul_tile_kernel(MatmulArgs g, int kb_per_split) {
  constexpr int T = BM * BN / 64, NA = BM * 8 / T, NW = BN * 8 / T;
  __shared__ __align__(16) uint8_t la[BM * kQBlk];
  __shared__ __align__(16) uint8_t lw[BN * kQBlk];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m0 = (int)blockIdx.y * BM, n0 = (int)blockIdx.x * BN;
  const int wm = (wave / (BN / 64)) * 64, wn = (wave % (BN / 64)) * 64;
  const int q = lane >> 4, i16 = lane & 15;
  const int kb0 = (int)blockIdx.z * kb_per_split, kb1 = min(g.nkb, kb0 + kb_per_split);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int64_t sw_row = (int64_t)((n0 + wn) / kQBlk < (g.n - 1) / kQBlk ? (n0 + wn) / kQBlk : (g.n - 1) / kQBlk) * g.nkb;
  // bf16 results with E8M0 scales: the instruction applies the scales
  constexpr bool kHwScale = E8 && sizeof(TO) == 2, kWide = sizeof(TO) == 4;
  for (int kb = kb0; kb < kb1; ++kb) {
    const int kk = kb * kQBlk;
    u32x4 va[NA], vw[NW];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int u = tid + i * T, r = u >> 3, c = u & 7;
      va[i] = load16_codes(g.a + (int64_t)(m0 + r) * g.lda + kk + c * 16, m0 + r < g.rows ? g.k - kk - c * 16 : 0);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int u = tid + i * T, r = u >> 3, c = u & 7;
      vw[i] = load16_codes(g.w + (int64_t)(n0 + r) * g.ldw + kk + c * 16, n0 + r < g.n ? g.k - kk - c * 16 : 0);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int u = tid + i * T, r = u >> 3, c = u & 7;
      *reinterpret_cast<u32x4*>(la + r * kQBlk + ((c ^ (r & 7)) << 4)) = va[i];
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int u = tid + i * T, r = u >> 3, c = u & 7;
      *reinterpret_cast<u32x4*>(lw + r * kQBlk + ((c ^ (r & 7)) << 4)) = vw[i];
    }
    __syncthreads();
    i32x8 fa[4];
    float s[4];
    int sb[4], swb = 0;
    if constexpr (kHwScale) swb = static_cast<const uint8_t*>(g.w_scales)[sw_row + kb];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = min(m0 + wm + j * 16 + i16, g.rows - 1);
      fa[j] = frag(la, wm + j * 16 + i16, q);
      if constexpr (kHwScale) sb[j] = static_cast<const uint8_t*>(g.a_scales)[m * g.nkb + kb];
      else s[j] = load_scale<E8>(g.a_scales, m * g.nkb + kb) * load_scale<E8>(g.w_scales, sw_row + kb);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const i32x8 fw = frag(lw, wn + i * 16 + i16, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kHwScale) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], acc[i][j], 0, 0, 0, swb, 0, sb[j]);
        } else {
          f32x4 p = {0, 0, 0, 0};
          if constexpr (kWide) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(fw, t), widen(fa[j], t), p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa[j], p, 0, 0, 0, kUnit, 0, kUnit);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s[j], acc[i][j][e]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = m0 + wm + j * 16 + i16;
    if (m >= g.rows) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + wn + i * 16 + q * 4;
      if (n >= g.n) continue;
      if (gridDim.z > 1)
        store4<float>(g.partial + ((int64_t)blockIdx.z * g.rows + m) * g.n + n, g.n - n, acc[i][j]);
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

// The reduction is split while the tiles leave compute units idle.
int splits_of(int64_t rows, int64_t n, int64_t k) {
  const int64_t tiles = ((rows + 127) / 128) * ((n + 127) / 128), nkb = q_nblk(k);
  int64_t s = 1;
  while (tiles * s < 256 && s * 2 <= nkb && s < 16) s *= 2;
  const int64_t per = (nkb + s - 1) / s;
  return (int)((nkb + per - 1) / per);
}

template <bool E8, typename TO>
hipError_t matmul_go(const MatmulArgs& g, hipStream_t stream) {
  const int s = splits_of(g.rows, g.n, g.k), per = (g.nkb + s - 1) / s;
  hipLaunchKernelGGL((matmul_tile_kernel<128, 128, E8, TO>), dim3((g.n + 127) / 128, (g.rows + 127) / 128, s),
                     dim3(256), 0, stream, g, per);
  if (s > 1) {
    const int64_t wg = ((int64_t)g.rows * g.n + 255) / 256;
    hipLaunchKernelGGL((matmul_join_kernel<TO>), dim3((unsigned)(wg < 4096 ? wg : 4096)), dim3(256), 0, stream, g, s);
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_q8_workspace(int64_t rows, int64_t n, int64_t k) {
  if (rows == 0) return 0;
  const int s = splits_of(rows, n, k);
  return s > 1 ? (int64_t)s * rows * n * 4 : 0;
}

hipError_t launch_matmul_q8(const MatmulArgs& g, bool e8, DT out, hipStream_t stream) {
  if (out == DT::F32) return e8 ? matmul_go<true, float>(g, stream) : matmul_go<false, float>(g, stream);
  return e8 ? matmul_go<true, uint16_t>(g, stream) : matmul_go<false, uint16_t>(g, stream);
}

}  // namespace harp
