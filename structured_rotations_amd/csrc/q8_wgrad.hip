// dW = dY^T X with X from an 8-bit checkpoint, on the bf16 matrix
// instructions.
//
//   dw[n][k] = sum_m dy[m][n] s[m][k/128] c[m][k]
//
// The scale changes along the reduction, so x is decoded before the product.
// A code has 4 significant bits: times a power of two (E8M0) it is exact in
// bf16 and so is every product.  Times an fp32 scale it has up to 28 bits;
// x = hi + lo in bf16 keeps 16 of them (two products), which fp32 results
// take; bf16 results take the rounded x alone, whose error (2^-9 of each
// term) is below the result's own rounding.
//
// Both operands are stored along the other axis than the one summed over:
// they stay that way in LDS ([m][n], [m][k]) and the transposing LDS read
// (ds_read_b64_tr_b16) gives a lane its neighbouring m.
#include "q8.h"

namespace harp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 32;  // rows (m) per step

// LDS tile of kStep rows of W bf16 values: 32-byte segments exchanged by the
// row's number so that neighbouring rows' reads of one segment cover all banks.
template <int W>
__device__ __forceinline__ int seg_off(int row, int seg) {
  constexpr int kSegs = W / 16;
  return row * W * 2 + ((seg ^ (row & (kSegs < 16 ? kSegs - 1 : 15))) << 5);
}

// The 8 values m = 8q .. 8q+7 of column seg * 16 + i16 for lane (q, i16).
template <int W>
__device__ __forceinline__ bf16x8_t frag_t(const uint8_t* lds, int seg, int lane) {
  const int q = lane >> 4, i = lane & 15;
  s16x4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * q + 4 * h + (i >> 2);
    v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(lds + seg_off<W>(row, seg) + (i & 3) * 8));
  }
  const s16x8 r = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8_t, r);
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int n, const f32x4& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) store1(p + i, v[i]);
}

// One 128 x 128 tile of dw per workgroup of 4 waves, each 64 (k) x 64 (n).
// PARTS: bf16 parts of x.
template <bool E8, int PARTS, typename TO>
__global__ __launch_bounds__(256) void wgrad_tile_kernel(WgradArgs g, int m_per_split) {
  constexpr int B = 128;
  __shared__ __align__(16) uint8_t ld[kStep * B * 2];
  __shared__ __align__(16) uint8_t lx[PARTS][kStep * B * 2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int k0 = (int)blockIdx.x * B, n0 = (int)blockIdx.y * B;
  const int wk = (wave & 1) * 4, wn = (wave >> 1) * 4;  // in segments of 16
  const int64_t mlo = (int64_t)blockIdx.z * m_per_split, mhi = min((int64_t)g.rows, mlo + m_per_split);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  for (int64_t m0 = mlo; m0 < mhi; m0 += kStep) {
    // 16 values (one segment) of each operand per thread: 32 rows x 8 segments
    const int r = tid >> 3, sg = tid & 7;
    const int64_t m = m0 + r;
    float dv[2][8], xv[2][8];
    float s = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int nn = m < mhi ? g.n - (n0 + sg * 16 + h * 8) : 0, nk = m < mhi ? g.k - (k0 + sg * 16 + h * 8) : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) dv[h][j] = xv[h][j] = 0.0f;
      if (nn > 0) load8_of<uint16_t>(g.dy + m * g.lddy + n0 + sg * 16 + h * 8, nn, dv[h]);
      if (nk > 0) load8_codes(g.x + m * g.ldx + k0 + sg * 16 + h * 8, nk, xv[h]);
    }
    if (m < mhi) s = load_scale<E8>(g.x_scales, m * g.nkb + k0 / kQBlk);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      store8(reinterpret_cast<uint16_t*>(ld + seg_off<B>(r, sg) + h * 16), dv[h]);
      float hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) hi[j] = xv[h][j] * s;
      store8(reinterpret_cast<uint16_t*>(lx[0] + seg_off<B>(r, sg) + h * 16), hi);
      if constexpr (PARTS == 2) {
        float lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) lo[j] = hi[j] - bf16_to_f32((uint16_t)pack_bf16x2_hw(hi[j], hi[j]));
        store8(reinterpret_cast<uint16_t*>(lx[PARTS - 1] + seg_off<B>(r, sg) + h * 16), lo);
      }
    }
    __syncthreads();
    bf16x8_t fd[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) fd[j] = frag_t<B>(ld, wn + j, lane);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8_t fx = frag_t<B>(lx[p], wk + i, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx, fd[j], acc[i][j], 0, 0, 0);
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + (wn + j) * 16 + (lane & 15);
    if (n >= g.n) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + (wk + i) * 16 + (lane >> 4) * 4;
      if (k >= g.k) continue;
      if (gridDim.z > 1) store4<float>(g.partial + ((int64_t)blockIdx.z * g.n + n) * g.k + k, g.k - k, acc[i][j]);
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

int wgrad_splits(int64_t rows, int64_t n, int64_t k, int64_t* per) {
  const int64_t tiles = ((n + 127) / 128) * ((k + 127) / 128), steps = (rows + kStep - 1) / kStep;
  int64_t s = 1;
  while (tiles * s < 256 && s * 2 * 4 <= steps && s < 64) s *= 2;
  const int64_t p = (steps + s - 1) / s;
  *per = p * kStep;
  return p > 0 ? (int)((steps + p - 1) / p) : 1;
}

template <bool E8, int PARTS, typename TO>
hipError_t wgrad_go(const WgradArgs& g, hipStream_t stream) {
  int64_t per;
  const int s = wgrad_splits(g.rows, g.n, g.k, &per);
  hipLaunchKernelGGL((wgrad_tile_kernel<E8, PARTS, TO>), dim3((g.k + 127) / 128, (g.n + 127) / 128, s), dim3(256), 0,
                     stream, g, (int)per);
  if (s > 1) {
    const int64_t wg = ((int64_t)g.n * g.k + 255) / 256;
    hipLaunchKernelGGL((wgrad_join_kernel<TO>), dim3((unsigned)(wg < 4096 ? wg : 4096)), dim3(256), 0, stream, g, s);
  }
  return hipGetLastError();
}

}  // namespace

int64_t matmul_q8_wgrad_workspace(int64_t rows, int64_t n, int64_t k) {
  int64_t per;
  const int s = wgrad_splits(rows, n, k, &per);
  return s > 1 ? (int64_t)s * n * k * 4 : 0;
}

hipError_t launch_matmul_q8_wgrad(const WgradArgs& g, bool e8, DT out, hipStream_t stream) {
  if (out == DT::F32) return e8 ? wgrad_go<true, 1, float>(g, stream) : wgrad_go<false, 2, float>(g, stream);
  return e8 ? wgrad_go<true, 1, uint16_t>(g, stream) : wgrad_go<false, 1, uint16_t>(g, stream);
}

}  // namespace harp
