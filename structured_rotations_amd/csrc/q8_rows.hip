// Row kernels of the 8-bit path: coding of rows and weights, the
// root-mean-square norm with the residual's addition and 8-bit output, and
// the norm's reverse mode from its 8-bit checkpoint.
//
// All of them are bound by HBM.  A thread holds chunks of 8 consecutive
// values (16 bytes of bf16), so a block of 128 columns is one DPP row of 16
// lanes and its maximum is four row rotations, with no LDS.
#include <algorithm>

#include "q8.h"

namespace harp {
namespace {

// ---------------------------------------------------------------- coding
// Rows: a workgroup of 256 threads covers 2^sh blocks by 16 >> sh rows at a
// time and walks down the rows.  16384 x 4096 bf16: 38 to 40 us over buffers in
// turn, as a copy of as many bytes (39); one buffer again and again stays in the
// cache, 33 us (a copy 29).
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
    Raw8<T> w;
    w.fill(0);
    if (n > 0) w.load(x + r * ldx + col, n);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i];
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
// 13824 x 5120 bf16: 42 us (a copy 41).
template <typename T, bool E8>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                            int cols, int nblk, uint8_t* __restrict__ codes,
                                                            int64_t ldc, void* __restrict__ scales) {
  __shared__ uint32_t part[4];
  const int blk = blockIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * kQBlk + (threadIdx.x >> 4);
  const int col = blk * kQBlk + (threadIdx.x & 15) * 8;
  const int n = cols - col;
  Raw8<T> w[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    w[i].fill(0);
    if (r < rows && n > 0) w[i].load(x + r * ldx + col, n);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(w[i][j]) & 0x7fffffffu);
  m = row16_umax(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  const Coder<E8> code(max(max(part[0], part[1]), max(part[2], part[3])), 1.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = w[i][j];
    code.code8(v, v);
    if (r < rows && n > 0) store8_codes(codes + r * ldc + col, n, v);
  }
  if (threadIdx.x == 0) store_scale<E8>(scales, (int64_t)blockIdx.y * nblk + blk, code.scale);
}

// ------------------------------------------------------------------ norm
// Sum over the workgroup, in a fixed order, in every thread.  `part` holds
// sets of 16 slots, used in turn: a wave reaches the next use of a set only
// after a barrier that follows everyone's reads of it.
template <int kSets>
__device__ __forceinline__ float block_sum(float v, float (&part)[kSets][16], int set) {
  v = wave_sum(v);
  const int nw = (int)blockDim.x >> 6;
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) part[set][threadIdx.x >> 6] = v;
  __syncthreads();
  const int l = threadIdx.x & 15;
  return row16_sum(l < nw ? part[set][l] : 0.0f);
}

// How a row is held.  One workgroup (kLanes 0), or, rows of one or two blocks
// (the norms of attention heads), 16 or 32 lanes of a workgroup of 256.
template <int kLanes>
struct RowMap {
  static constexpr int kRows = kLanes ? 256 / kLanes : 1;
  int tid, threads, row;
  int64_t first, step;
  __device__ __forceinline__ RowMap() {
    tid = kLanes ? threadIdx.x & (kLanes - 1) : threadIdx.x;
    threads = kLanes ? kLanes : blockDim.x;
    row = kLanes ? (int)threadIdx.x / kLanes : 0;
    first = (int64_t)blockIdx.x * kRows + row;
    step = (int64_t)gridDim.x * kRows;
  }
};
template <int kLanes, int kSets>
__device__ __forceinline__ float row_sum(float v, float (&part)[kSets][16], int set) {
  if constexpr (kLanes == 0) return block_sum(v, part, set);
  v = row16_sum(v);
  return kLanes == 32 ? v + __shfl_xor(v, 16) : v;
}

// A workgroup walks over rows; a row stays in registers between the sum of
// squares and the coding (NCH chunks of 8 per thread), and (kAhead: rows up to
// 8192, which leave registers for it) the next row is on its way meanwhile.
// 16384 x 5120 bf16, residual, checkpoint: 674 MB in 135 us, 5.0 TB/s (a copy 125;
// 175 us without the next row's loads); 4096 x 16384: 90 us, with gamma and its
// second coding 114.  One row of 4096: 2.8 us of the call's 8, the rest is the
// launch and the host's checks.  Rows of 64 (16 lanes each), 100000 of them: 11 us
// with E8M0 scales and one coding to 17 with fp32 scales and two, against 46 us
// with a workgroup per row; 60000 of 160 (32 lanes): 19 us, against 39.
template <typename T, int NCH, bool E8, int kLanes = 0>
__global__ __launch_bounds__(NCH <= 2 ? 512 : 1024) void rmsnorm_q8_kernel(NormArgs a) {
  constexpr bool kAhead = NCH <= 2;
  const RowMap<kLanes> map;
  __shared__ float part[3][16];
  const int nblk = (a.d + kQBlk - 1) / kQBlk;
  const T* gamma = static_cast<const T*>(a.gamma);
  int col[NCH], n[NCH];
  Raw8<T> x[NCH], res[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    col[c] = (map.tid + c * map.threads) * 8;
    n[c] = a.d - col[c];
    x[c].fill(0);
    res[c].fill(0);
  }
  auto load = [&](int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if (n[c] <= 0) continue;
      x[c].load(static_cast<const T*>(a.x) + r * a.ldx + col[c], n[c]);
      if (a.residual) res[c].load(static_cast<const T*>(a.residual) + r * a.ldr + col[c], n[c]);
    }
  };
  if (kAhead) load(map.first);
  const float least = a.eps < 0x1p-100f ? 0x1p-80f : 0.0f;
  int set = 0;
  for (int64_t r = map.first; r < a.rows; r += map.step, set ^= 1) {
    if (!kAhead) load(r);
    float v[NCH][8], ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[c][j] = a.residual ? x[c][j] + res[c][j] : x[c][j];
        ss += v[c][j] * v[c][j];
      }
      if (a.h && n[c] > 0) store8_of<T>(static_cast<T*>(a.h) + r * a.ldh + col[c], n[c], v[c]);
    }
    if (kAhead) load(r + map.step);
    ss = row_sum<kLanes>(ss, part, set);
    float rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
    // Squares beyond fp32's range (rows around 2^64 / sqrt(d) and more, or, if
    // eps does not outweigh them, below 2^-40): again with the sum in other
    // units.  The sum is the same in every thread of the row.
    if (!(ss >= least && ss < __uint_as_float(0x7f800000u))) {
      const float unit = ss < least ? 0x1p80f : 0x1p-80f;
      ss = 0.0f;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (v[c][j] * unit) * (v[c][j] * unit);
      ss = row_sum<kLanes>(ss, part, 2);
      rstd = unit / sqrtf(ss / (float)a.d + a.eps * unit * unit);
    }
    if (a.rstd && map.tid == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int blk = col[c] / kQBlk;
      float o[8];
      if (gamma) {
        if (a.ckpt) {
          const Coder<E8> code(row16_umax(amax8(v[c])), rstd);
          code.code8(v[c], o);
          if (n[c] > 0) {
            store8_codes(a.ckpt + r * a.ldk + col[c], n[c], o);
            if ((threadIdx.x & 15) == 0) store_scale<E8>(a.ckpt_scales, r * nblk + blk, code.scale);
          }
        }
        Raw8<T> g;
        g.fill(0);
        if (n[c] > 0) g.load(gamma + col[c], n[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] *= g[j];
      }
      const Coder<E8> code(row16_umax(amax8(v[c])), rstd);
      code.code8(v[c], o);
      if (n[c] > 0) {
        store8_codes(a.codes + r * a.ldc + col[c], n[c], o);
        if ((threadIdx.x & 15) == 0) store_scale<E8>(a.scales, r * nblk + blk, code.scale);
      }
    }
  }
}

// --------------------------------------------------------- norm, backward
// A workgroup walks over rows, keeping gamma and its share of dgamma's sum
// for its columns in registers, and the row as it came: the values are made
// from it once for the sum and once for dh, which takes fewer registers than
// keeping them.  The next row is on its way meanwhile (kAhead: rows up to 8192;
// longer ones read gamma and dres when they are used instead).  The partial sums of the
// workgroups are added in order by the second kernel (6 us at 16384 x 5120; atomics would
// change the result from run to run).  16384 x 5120 bf16 with dres, both kernels: 126 us,
// 4.7 TB/s (a copy 110); 4096 x 16384: 111 us; 100000 x 64: 16 us (a workgroup per row 51),
// 60000 x 160: 19 us (36).
// Rows beyond 16384 spill, dgamma's share and four chunks of the row in registers: 305 us
// at 2234 x 30000, 3.5 times what its 469 MB take.
template <typename T, int NCH, bool E8, int kLanes = 0>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void rmsnorm_q8_vjp_kernel(NormVjpArgs a) {
  constexpr bool kAhead = NCH == 1;
  const RowMap<kLanes> map;
  __shared__ float part[2][16];
  const int nblk = (a.d + kQBlk - 1) / kQBlk;
  int col[NCH], n[NCH];
  Raw8<T> g[NCH];
  float dg[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    col[c] = (map.tid + c * map.threads) * 8;
    n[c] = a.d - col[c];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[c][j] = 0.0f;
  }
  auto load_g = [&](int c) {
    g[c].fill(0x3f800000u);
    if (a.gamma && n[c] > 0) g[c].load(static_cast<const T*>(a.gamma) + col[c], n[c]);
  };
  if (kAhead)
#pragma unroll
    for (int c = 0; c < NCH; ++c) load_g(c);
  struct Row {
    Raw8<T> dn[NCH], dr[NCH];
    RawCodes cd[NCH];
    float sc[NCH], rstd;
  } now, next;
  auto load_dr = [&](Row& w, int64_t r, int c) {
    w.dr[c].fill(0);
    if (a.dres && r < a.rows && n[c] > 0)
      w.dr[c].load(static_cast<const T*>(a.dres) + r * a.lddres + col[c], n[c]);
  };
  auto load = [&](Row& w, int64_t r) {
    w.rstd = r < a.rows ? a.rstd[r] : 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      w.dn[c].fill(0);
      if (kAhead) load_dr(w, r, c);
      w.cd[c].w[0] = w.cd[c].w[1] = 0;
      w.sc[c] = 0.0f;
      if (r >= a.rows || n[c] <= 0) continue;
      w.cd[c].load(a.codes + r * a.ldc + col[c], n[c]);
      w.dn[c].load(static_cast<const T*>(a.dn) + r * a.lddn + col[c], n[c]);
      w.sc[c] = load_scale<E8>(a.scales, r * nblk + col[c] / kQBlk);
    }
  };
  if (kAhead) load(now, map.first);
  int set = 0;
  for (int64_t r = map.first; r < a.rows; r += map.step, set ^= 1) {
    if (kAhead) load(next, r + map.step);
    else load(now, r);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float xn[8];
      now.cd[c].values(xn);
      if (!kAhead) load_g(c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xn[j] = j < n[c] ? xn[j] * now.sc[c] : 0.0f;  // 0 past the row's end, whatever the scale
        const float u = now.dn[c][j];
        dg[c][j] += u * xn[j];
        dot += u * g[c][j] * xn[j];
      }
    }
    const float mean = row_sum<kLanes>(dot, part, set) / (float)a.d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if (n[c] <= 0) continue;
      float xn[8], o[8];
      now.cd[c].values(xn);
      if (!kAhead) {
        load_g(c);
        load_dr(now, r, c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = now.dr[c][j] + now.rstd * (now.dn[c][j] * g[c][j] - xn[j] * now.sc[c] * mean);
      store8_of<T>(static_cast<T*>(a.dh) + r * a.lddh + col[c], n[c], o);
    }
    if (kAhead) now = next;
  }
  if constexpr (kLanes > 0) {
    // the rows' shares in order
    __shared__ float share[256 / kLanes][kLanes * 8 + 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) share[map.row][map.tid * 8 + j] = dg[0][j];
    __syncthreads();
    if (a.partial && (int)threadIdx.x < a.d) {
      float t = 0.0f;
      for (int i = 0; i < 256 / kLanes; ++i) t += share[i][threadIdx.x];
      a.partial[(int64_t)blockIdx.x * a.d + threadIdx.x] = t;
    }
  } else if (a.partial) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (n[c] > 0) store8_of<float>(a.partial + (int64_t)blockIdx.x * a.d + col[c], n[c], dg[c]);
  }
}

// dgamma = the partial sums added in a fixed order: 16 columns by 64 slices of
// them per workgroup, four loads in flight each.  parts == 0 writes zeros.
__global__ __launch_bounds__(1024) void dgamma_kernel(const float* __restrict__ partial, int parts, int d,
                                                      float* __restrict__ dgamma) {
  __shared__ float sum[64][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int col = (int)blockIdx.x * 16 + c;
  float s[4] = {0, 0, 0, 0};
  if (col < d)
    for (int p = slice; p < parts; p += 256)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p + 64 * i < parts) s[i] += partial[(int64_t)(p + 64 * i) * d + col];
  sum[slice][c] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (slice == 0 && col < d) {
    float t = 0.0f;
    for (int i = 0; i < 64; ++i) t += sum[i][c];
    dgamma[col] = t;
  }
}

// Threads for a row of d values with nch chunks of 8 each: whole waves.
int row_threads(int d, int nch) { return ((d + 7) / 8 + nch * 64 - 1) / (nch * 64) * 64; }

// Workgroups for rows of one or two blocks.
int short_groups(int64_t rows, int64_t d) {
  const int64_t per = d <= kQBlk ? 16 : 8;
  return (int)std::min((rows + per - 1) / per, (int64_t)2048);
}

// Chunks per thread of the norm: two from 4096 on (16384 x 5120 bf16 with a
// checkpoint: one chunk 165 us, two 134 us; a row of 4096 is then 8 waves or
// 4, and one row alone is faster with 8).
template <typename T, bool E8>
hipError_t norm_go(const NormArgs& a, hipStream_t stream) {
  if (a.d <= 2 * kQBlk) {
    const dim3 grid(short_groups(a.rows, a.d));
    if (a.d <= kQBlk) hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 1, E8, 16>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 1, E8, 32>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  const int nch = a.d <= 4096 ? 1 : a.d <= 8192 ? 2 : 4, threads = row_threads(a.d, nch);
  // about as many workgroups as fit the compute units at once
  const int64_t fit = 256 * (int64_t)std::max(1, 1024 / threads);
  const dim3 grid((unsigned)std::min(a.rows, fit));
  if (nch == 1) hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 1, E8>), grid, dim3(threads), 0, stream, a);
  else if (nch == 2) hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 2, E8>), grid, dim3(threads), 0, stream, a);
  else hipLaunchKernelGGL((rmsnorm_q8_kernel<T, 4, E8>), grid, dim3(threads), 0, stream, a);
  return hipGetLastError();
}

// Chunks per thread of the backward pass (16384 x 5120: two 186 us against 127,
// for want of registers).
int vjp_chunks(int64_t d) { return d <= 8192 ? 1 : d <= 16384 ? 2 : 4; }
// Lanes of a row, 0: a workgroup.  Up to 64 rows of two blocks take a workgroup
// each (16 rows of 256: 4.84 us against 5.01; 256 rows: 5.99 against 5.25).
int vjp_lanes(int64_t rows, int64_t d) { return d <= kQBlk ? 16 : d <= 2 * kQBlk && rows > 64 ? 32 : 0; }
// Workgroups of the backward pass.  Each writes a row of partial sums, which the
// second kernel reads with d / 16 workgroups, so no more than keep the compute
// units busy: about 512 threads each (1000 values x 30000 rows: 42 us, with 1024
// threads 48), 1024 where rows are no whole pieces of 8 and take more
// instructions (999 x 30000: 86 us, with 512 threads 124), with 8 or 4 rows
// for each workgroup (1000 x 2048: 11.4 us, 21.6 with one).  16384 x 5120: 512
// workgroups 127 us, 1024 135 us.  Rows of one or two blocks, 16 or 8 at a time:
// 512 (200 x 30000: 14 us, 2048 workgroups 21).
int vjp_groups(int64_t rows, int64_t d) {
  if (vjp_lanes(rows, d)) return std::min(short_groups(rows, d), 512);
  const int threads = row_threads((int)d, vjp_chunks(d));
  const bool whole = d % 8 == 0;
  const int per_unit = whole ? (512 + threads - 1) / threads : 1024 / threads;
  const int64_t most = 256 * (int64_t)std::min(8, std::max(2, per_unit));
  return (int)std::min(rows, std::max<int64_t>(512, std::min(rows / (whole ? 8 : 4), most)));
}

template <typename T, bool E8>
hipError_t norm_vjp_go(const NormVjpArgs& a, hipStream_t stream) {
  const int groups = vjp_groups(a.rows, a.d), nch = vjp_chunks(a.d), threads = row_threads(a.d, nch);
  const int lanes = vjp_lanes(a.rows, a.d);
  if (groups > 0) {
    const dim3 grid(groups);
    if (lanes == 16) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 1, E8, 16>), grid, dim3(256), 0, stream, a);
    else if (lanes == 32) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 1, E8, 32>), grid, dim3(256), 0, stream, a);
    else if (nch == 1) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 1, E8>), grid, dim3(threads), 0, stream, a);
    else if (nch == 2) hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 2, E8>), grid, dim3(threads), 0, stream, a);
    else hipLaunchKernelGGL((rmsnorm_q8_vjp_kernel<T, 4, E8>), grid, dim3(threads), 0, stream, a);
  }
  if (a.dgamma)
    hipLaunchKernelGGL(dgamma_kernel, dim3((a.d + 15) / 16), dim3(1024), 0, stream, a.partial, groups, a.d, a.dgamma);
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

int64_t rmsnorm_q8_vjp_workspace(int64_t rows, int64_t d) { return (int64_t)vjp_groups(rows, d) * d * 4; }

hipError_t launch_rmsnorm_q8_vjp(const NormVjpArgs& a, DT io, bool e8, hipStream_t stream) {
  if (io == DT::F32) return e8 ? norm_vjp_go<float, true>(a, stream) : norm_vjp_go<float, false>(a, stream);
  return e8 ? norm_vjp_go<uint16_t, true>(a, stream) : norm_vjp_go<uint16_t, false>(a, stream);
}

}  // namespace harp
