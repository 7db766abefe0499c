// The 4-bit cache as it is written and as it is read back.
//
// Both are bound by HBM.  A thread holds 8 consecutive values of a head: 16
// bytes of bf16 and one word of 8 codes; the 4 lanes of a quad share a block
// of 32 and find its maximum by two lane exchanges.
#include <algorithm>

#include "kv4.h"
#include "q8.h"

namespace harp {
namespace {

// The scale byte of a block whose largest magnitude has the bits `top`: the
// smallest power of two of which it is at most 6 times, by its bits: the
// exponent less 2 if the mantissa is at most 1.5, less 1 if not.  2^-120 at
// least; 255 for NaN, infinities and magnitudes of 1.75 * 2^127 and more, whose
// codes would stand for more than fp32 holds.
__device__ __forceinline__ uint32_t scale4(uint32_t top) {
  if (top >= 0x7f600000u) return 255;
  const int e = (int)((top + 0x003fffffu) >> 23) - 2;
  return (uint32_t)max(e, 127 - 120);
}

// Where the tokens of a call lie.  Waves walk over tokens; `threads` lanes of
// a wave's 64 at a time over a token's keys and values, 8 values each.
struct Place {
  int64_t page;  // -1: none
  int in_page;   // -1: before the sequence's beginning or behind the last one
};
__device__ __forceinline__ Place place_of(const Cache4& c, const Plan4& p, int64_t row) {
  const int b = sequence_of(p, row);
  const int64_t first = p.starts[b], end = p.starts[b + 1];
  const int64_t pos = (int64_t)p.lengths[b] - (end - row);
  if (row < first || row >= end) return {-1, -2};
  if (pos < 0) return {-1, -1};
  const int64_t page = pos >> c.page_log2;
  return {page_of(c, p, b, page), (int)(pos - (page << c.page_log2))};
}

// The u-th 8 values of a token: keys first, then values.
struct Unit {
  bool is_k;
  int head, col;
  __device__ __forceinline__ Unit(const Cache4& c, int u) {
    const int per_head = c.d >> 3, side = c.heads * per_head;
    is_k = u < side;
    const int in = is_k ? u : u - side;
    head = in / per_head;
    col = (in - head * per_head) * 8;
  }
};
__device__ __forceinline__ int64_t row_in_page(const Cache4& c, int head, int in_page) {
  return ((int64_t)head << c.page_log2) + in_page;
}

template <typename T>
__global__ __launch_bounds__(256) void kv4_write_kernel(Cache4 c, Plan4 p, Heads k, Heads v, int tokens, int parts) {
  const int units = c.heads * (c.d >> 2), lane = threadIdx.x & 63;
  const int per = ((units + 63) / 64 + parts - 1) / parts * 64;
  const int64_t all = (int64_t)tokens * parts;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < all; unit += (int64_t)gridDim.x * 4) {
    const int64_t row = unit / parts;
    const int first = (int)(unit - row * parts) * per, end = min(units, first + per);
    const Place at = place_of(c, p, row);
    if (at.page < 0) continue;
    for (int u0 = first; u0 < end; u0 += 64) {
      const int u = u0 + lane;
      if (u >= end) continue;  // quads stay whole: end and u0 are multiples of 4
      const Unit w(c, u);
      const Heads& s = w.is_k ? k : v;
      Raw8<T> x;
      x.load(static_cast<const T*>(s.p) + row * s.token + w.head * s.head + w.col, 8);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = x[i];
      uint32_t top = amax8(f);
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
      const uint32_t e = scale4(top);
      const float scale = __uint_as_float(e << 23);
      uint32_t codes = 0;
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0], f[1], scale, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2], f[3], scale, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4], f[5], scale, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6], f[7], scale, 3);
      if (e == 255) codes = 0;
      const Side4& o = w.is_k ? c.k : c.v;
      const int64_t to = row_in_page(c, w.head, at.in_page);
      *reinterpret_cast<uint32_t*>(o.codes + at.page * o.codes_page + to * (c.d >> 1) + (w.col >> 1)) = codes;
      if ((lane & 3) == 0) o.scales[at.page * o.scales_page + to * (c.d >> 5) + (w.col >> 5)] = (uint8_t)e;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void kv4_read_kernel(Cache4 c, Plan4 p, Heads k, Heads v, int tokens, int parts) {
  const int units = c.heads * (c.d >> 2), lane = threadIdx.x & 63;
  const int per = ((units + 63) / 64 + parts - 1) / parts * 64;
  const int64_t all = (int64_t)tokens * parts;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < all; unit += (int64_t)gridDim.x * 4) {
    const int64_t row = unit / parts;
    const int first = (int)(unit - row * parts) * per, end = min(units, first + per);
    const Place at = place_of(c, p, row);
    if (at.in_page == -2) continue;
    for (int u = first + lane; u < end; u += 64) {
      const Unit w(c, u);
      uint32_t codes = 0, e = at.in_page < 0 ? 127 : 255;
      if (at.page >= 0) {
        const Side4& o = w.is_k ? c.k : c.v;
        const int64_t from = row_in_page(c, w.head, at.in_page);
        codes = *reinterpret_cast<const uint32_t*>(o.codes + at.page * o.codes_page + from * (c.d >> 1) + (w.col >> 1));
        e = o.scales[at.page * o.scales_page + from * (c.d >> 5) + (w.col >> 5)];
      }
      const float scale = __uint_as_float(e << 23);  // the conversion reads the exponent only; 255 gives NaN
      float f[8];
      const f32x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
      const f32x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
      const f32x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
      const f32x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
      f[0] = a0[0]; f[1] = a0[1]; f[2] = a1[0]; f[3] = a1[1];
      f[4] = a2[0]; f[5] = a2[1]; f[6] = a3[0]; f[7] = a3[1];
      const Heads& s = w.is_k ? k : v;
      store8(static_cast<T*>(s.p) + row * s.token + w.head * s.head + w.col, f);
    }
  }
}

// Parts of a token, a wave each: one where there are tokens enough, else as
// many as the chip has room for.
int parts_of(const Cache4& c, int tokens) {
  const int rounds = (c.heads * (c.d >> 2) + 63) / 64;
  return std::min(rounds, std::max(1, 8192 / std::max(1, tokens)));
}

template <typename K>
hipError_t go(K kernel, const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, hipStream_t stream) {
  const int parts = parts_of(c, tokens);
  const dim3 grid((unsigned)std::min<int64_t>(((int64_t)tokens * parts + 3) / 4, 1 << 20));
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, c, p, k, v, tokens, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_write(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                            hipStream_t stream) {
  return io == DT::F32 ? go(kv4_write_kernel<float>, c, p, k, v, tokens, stream)
                       : go(kv4_write_kernel<uint16_t>, c, p, k, v, tokens, stream);
}
hipError_t launch_kv4_read(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                           hipStream_t stream) {
  return io == DT::F32 ? go(kv4_read_kernel<float>, c, p, k, v, tokens, stream)
                       : go(kv4_read_kernel<uint16_t>, c, p, k, v, tokens, stream);
}

}  // namespace harp
