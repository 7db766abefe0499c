// Row kernels of the 8-bit path: coding of rows and weights, the
// root-mean-square norm with the residual's addition and 8-bit output, and
// the norm's reverse mode from its 8-bit checkpoint.
//
// All of them are bound by HBM.  A thread holds chunks of 8 consecutive
// values (16 bytes of bf16), so a block of 128 columns is one DPP row of 16
// lanes and its maximum is four row rotations, with no LDS.
#include "q8.h"

namespace harp {
namespace {

// ---------------------------------------------------------------- coding
// Rows: a workgroup of 256 threads covers 2^sh blocks by 16 >> sh rows at a
// time and walks down the rows.
template <typename T, bool E8>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                            int cols, int nblk, int sh, uint8_t* __restrict__ codes,
                                                            int64_t ldc, void* __restrict__ scales) {
  const int unit = threadIdx.x >> 4;
  const int blk = (int)blockIdx.x * (1 << sh) + (unit & ((1 << sh) - 1));
  const int col = blk * kQBlk + (threadIdx.x & 15) * 8;
  const int n = blk < nblk ? cols - col : 0;
  const int64_t step = (int64_t)gridDim.y * (16 >> sh);
  for (int64_t r = (int64_t)blockIdx.y * (16 >> sh) + (unit >> sh); r < rows; r += step) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) load8_of<T>(x + r * ldx + col, n, v);
    const Coder<E8> code(row16_umax(amax8(v)), 1.0f);
    code.code8(v, v);
    if (n > 0) {
      store8_codes(codes + r * ldc + col, n, v);
      if ((threadIdx.x & 15) == 0) store_scale<E8>(scales, r * nblk + blk, code.scale);
    }
  }
}

// Weights: one 128 x 128 block per workgroup, 64 values per thread in
// registers between the maximum and the coding, so the weight is read once.
template <typename T, bool E8>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                            int cols, int nblk, uint8_t* __restrict__ codes,
                                                            int64_t ldc, void* __restrict__ scales) {
  __shared__ uint32_t part[4];
  const int blk = blockIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * kQBlk + (threadIdx.x >> 4);
  const int col = blk * kQBlk + (threadIdx.x & 15) * 8;
  const int n = cols - col;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && n > 0) load8_of<T>(x + r * ldx + col, n, v[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i]));
  m = row16_umax(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const Coder<E8> code(max(max(part[0], part[1]), max(part[2], part[3])), 1.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    code.code8(v[i], v[i]);
    if (r < rows && n > 0) store8_codes(codes + r * ldc + col, n, v[i]);
  }
  if (threadIdx.x == 0) store_scale<E8>(scales, (int64_t)blockIdx.y * nblk + blk, code.scale);
}

// ------------------------------------------------------------------ norm
// Sum over the workgroup, in a fixed order, in every thread.  `part` holds
// two sets of 16 slots, used in turn: a wave reaches the next use of a set
// only after a barrier that follows everyone's reads of it.
__device__ __forceinline__ float block_sum(float v, float (&part)[2][16], int set) {
  v = wave_sum(v);
  const int nw = (int)blockDim.x >> 6;
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) part[set][threadIdx.x >> 6] = v;
  __syncthreads();
  const int l = threadIdx.x & 15;
  return row16_sum(l < nw ? part[set][l] : 0.0f);
}

// One row per workgroup; the row stays in registers between the sum of
// squares and the coding (NCH chunks of 8 per thread).
template <typename T, int NCH, bool E8>
__global__ __launch_bounds__(1024) void rmsnorm_q8_kernel(NormArgs a) {
  __shared__ float part[2][16];
  const int nblk = (a.d + kQBlk - 1) / kQBlk;
  const T* gamma = static_cast<const T*>(a.gamma);
  int set = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* res = static_cast<const T*>(a.residual) + (a.residual ? r * a.ldr : 0);
    float v[NCH][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
      if (n > 0) load8_of<T>(x + col, n, v[c]);
    }
    if (a.residual) {
      float w[NCH][8];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
        if (n > 0) load8_of<T>(res + col, n, w[c]);
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
        if (n <= 0) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] += w[c][j];
        if (a.h) store8_of<T>(static_cast<T*>(a.h) + r * a.ldh + col, n, v[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[c][j] * v[c][j];
    ss = block_sum(ss, part, set);
    const float rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int chunk = (int)threadIdx.x + c * (int)blockDim.x;
      const int col = chunk * 8, n = a.d - col;
float o[8];
      if (gamma) {
        if (a.ckpt) {
          const Coder<E8> code(row16_umax(amax8(v[c])), rstd);
          code.code8(v[c], o);
          if (n > 0) {
            store8_codes(a.ckpt + r * a.ldk + col, n, o);
            if ((threadIdx.x & 15) == 0) store_scale<E8>(a.ckpt_scales, r * nblk + (chunk >> 4), code.scale);
          }
        }
        float g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n > 0) load8_of<T>(gamma + col, n, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] *= g[j];
      }
      const Coder<E8> code(row16_umax(amax8(v[c])), rstd);
      code.code8(v[c], o);
      if (n > 0) {
        store8_codes(a.codes + r * a.ldc + col, n, o);
        if ((threadIdx.x & 15) == 0) store_scale<E8>(a.scales, r * nblk + (chunk >> 4), code.scale);
      }
    }
  }
}

// --------------------------------------------------------- norm, backward
// A workgroup walks over rows, keeping gamma and its share of dgamma's sum
// for its columns in registers; the partial sums of the workgroups are added
// in order by the second kernel.
template <typename T, int NCH, bool E8>
__global__ __launch_bounds__(1024) void rmsnorm_q8_vjp_kernel(NormVjpArgs a) {
  __shared__ float part[2][16];
  const int nblk = (a.d + kQBlk - 1) / kQBlk;
  float g[NCH][8], dg[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[c][j] = 1.0f;
      dg[c][j] = 0.0f;
    }
    if (a.gamma && n > 0) load8_of<T>(static_cast<const T*>(a.gamma) + col, n, g[c]);
  }
  int set = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
    float xn[NCH][8], u[NCH][8], dr[NCH][8];
    float dot = 0.0f;
    const float rstd = a.rstd[r];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int chunk = (int)threadIdx.x + c * (int)blockDim.x;
      const int col = chunk * 8, n = a.d - col;
#pragma unroll
      for (int j = 0; j < 8; ++j) xn[c][j] = u[c][j] = dr[c][j] = 0.0f;
      if (n > 0) {
        load8_codes(a.codes + r * a.ldc + col, n, xn[c]);
        load8_of<T>(static_cast<const T*>(a.dn) + r * a.lddn + col, n, u[c]);
        if (a.dres) load8_of<T>(static_cast<const T*>(a.dres) + r * a.lddres + col, n, dr[c]);
        const float s = load_scale<E8>(a.scales, r * nblk + (chunk >> 4));
#pragma unroll
        for (int j = 0; j < 8; ++j) xn[c][j] = j < n ? xn[c][j] * s : 0.0f;  // 0 past the end, whatever the scale
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dg[c][j] += u[c][j] * xn[c][j];
        u[c][j] *= g[c][j];
        dot += u[c][j] * xn[c][j];
      }
    const float mean = block_sum(dot, part, set) / (float)a.d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
      if (n <= 0) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = dr[c][j] + rstd * (u[c][j] - xn[c][j] * mean);
      store8_of<T>(static_cast<T*>(a.dh) + r * a.lddh + col, n, o);
    }
  }
  if (a.partial) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = ((int)threadIdx.x + c * (int)blockDim.x) * 8, n = a.d - col;
      if (n > 0) store8_of<float>(a.partial + (int64_t)blockIdx.x * a.d + col, n, dg[c]);
    }
  }
}

// dgamma = the partial sums added in order: 16 columns by 16 slices of them
// per workgroup.  parts == 0 writes zeros.
__global__ __launch_bounds__(256) void dgamma_kernel(const float* __restrict__ partial, int parts, int d,
                                                     float* __restrict__ dgamma) {
  __shared__ float sum[16][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int col = (int)blockIdx.x * 16 + c;
  float s = 0.0f;
  if (col < d)
    for (int p = slice; p < parts; p += 16) s += partial[(int64_t)p * d + col];
  sum[slice][c] = s;
  __syncthreads();
  if (slice == 0 && col < d) {
    float t = 0.0f;
    for (int i = 0; i < 16; ++i) t += sum[i][c];
    dgamma[col] = t;
  }
}

// Threads and chunks per thread for a row of d values: the row is held by one
// workgroup of whole waves.
struct RowShape {
  int threads, nch;
};
RowShape row_shape(int d) {
  const int nch = d <= 2048 ? 1 : d <= 16384 ? 2 : 4;
  const int chunks = (d + 7) / 8;
  return {((chunks + nch - 1) / nch + 63) / 64 * 64, nch};
}

template <typename T, bool E8>
hipError_t norm_go(const NormArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.d);
  const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20)));
  if (s.nch == 1) hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 1, E8>), grid, dim3(s.threads), 0, stream, a);
  else if (s.nch == 2) hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 2, E8>), grid, dim3(s.threads), 0, stream, a);
  else hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 4, E8>), grid, dim3(s.threads), 0, stream, a);
  return hipGetLastError();
}

int vjp_groups(int64_t rows) { return (int)(rows < 1024 ? rows : 1024); }

template <typename T, bool E8>
hipError_t norm_vjp_go(const NormVjpArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.d);
  const int groups = vjp_groups(a.rows);
  if (groups > 0) {
    const dim3 grid(groups);
    if (s.nch == 1) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 1, E8>), grid, dim3(s.threads), 0, stream, a);
    else if (s.nch == 2) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 2, E8>), grid, dim3(s.threads), 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 4, E8>), grid, dim3(s.threads), 0, stream, a);
  }
  if (a.dgamma)
    hipLaunchKernelGGL(dgamma_kernel, dim3((a.d + 15) / 16), dim3(256), 0, stream, a.partial, groups, a.d, a.dgamma);
  return hipGetLastError();
}

template <typename T, bool E8>
hipError_t quantize_go(const T* x, int64_t ldx, int64_t rows, int cols, bool tile, uint8_t* codes, int64_t ldc,
                       void* scales, hipStream_t stream) {
  const int nblk = (int)q_nblk(cols);
  if (tile) {
    // 65535 row blocks per launch (the grid's second dimension)
    const int64_t span = 65535LL * kQBlk;
    for (int64_t r = 0; r < rows; r += span) {
      const int64_t n = rows - r < span ? rows - r : span;
      void* sc = static_cast<char*>(scales) + r / kQBlk * nblk * (E8 ? 1 : 4);
      hipLaunchKernelGGL((quantize_tile_kernel<T, E8>), dim3(nblk, (unsigned)q_nblk(n)), dim3(256), 0, stream,
                         x + r * ldx, ldx, n, cols, nblk, codes + r * ldc, ldc, sc);
    }
    return hipGetLastError();
  }
  int sh = 0;
  while (sh < 4 && (1 << sh) < nblk) ++sh;
  const int64_t gx = (nblk + (1 << sh) - 1) >> sh, units = (rows + (16 >> sh) - 1) / (16 >> sh);
  // about 8 workgroups a CU in flight, each walking down the rows
  int64_t gy = (256 * 8 * 2 + gx - 1) / gx;
  if (gy > units) gy = units;
  if (gy > 65535) gy = 65535;
  hipLaunchKernelGGL((quantize_rows_kernel<T, E8>), dim3((unsigned)gx, (unsigned)gy), dim3(256), 0, stream, x, ldx,
                     rows, cols, nblk, sh, codes, ldc, scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_q8(const void* x, int64_t ldx, DT io, int64_t rows, int cols, bool tile, uint8_t* codes,
                              int64_t ldc, void* scales, bool e8, hipStream_t stream) {
  if (io == DT::F32) {
    const float* p = static_cast<const float*>(x);
    return e8 ? quantize_go<float, true>(p, ldx, rows, cols, tile, codes, ldc, scales, stream)
              : quantize_go<float, false>(p, ldx, rows, cols, tile, codes, ldc, scales, stream);
  }
  const uint16_t* p = static_cast<const uint16_t*>(x);
  return e8 ? quantize_go<uint16_t, true>(p, ldx, rows, cols, tile, codes, ldc, scales, stream)
            : quantize_go<uint16_t, false>(p, ldx, rows, cols, tile, codes, ldc, scales, stream);
}

hipError_t launch_rmsnorm_q8(const NormArgs& a, DT io, bool e8, hipStream_t stream) {
  if (io == DT::F32) return e8 ? norm_go<float, true>(a, stream) : norm_go<float, false>(a, stream);
  return e8 ? norm_go<uint16_t, true>(a, stream) : norm_go<uint16_t, false>(a, stream);
}

int64_t rmsnorm_q8_vjp_workspace(int64_t rows, int64_t d) { return (int64_t)vjp_groups(rows) * d * 4; }

hipError_t launch_rmsnorm_q8_vjp(const NormVjpArgs& a, DT io, bool e8, hipStream_t stream) {
  if (io == DT::F32) return e8 ? norm_vjp_go<float, true>(a, stream) : norm_vjp_go<float, false>(a, stream);
  return e8 ? norm_vjp_go<uint16_t, true>(a, stream) : norm_vjp_go<uint16_t, false>(a, stream);
}

}  // namespace harp
