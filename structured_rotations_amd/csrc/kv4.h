// The operators of attention over a cache in 4 bits: E2M1 codes with one E8M0
// scale per 32 values of a head.  The format, a cache's and a plan's places,
// and the host launchers that the C entry points call after every argument has
// been checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "kernels.h"
#include "q8.h"

namespace harp {

constexpr int kBlk4 = 32;  // values per scale

// From so many bytes on an array of heads is streamed, past the caches: the 8
// L2s hold 4 MiB each, so little of it would be left there for its next reader,
// and it would push out what is (norm_rope of 16384 x 32+8 x 128: 72 us, streamed
// 64; reading 41 million values of a cache: 61 us, streamed 38).  Less is left
// to the caches, from which its reader gets it.
constexpr int64_t kStreamBytes = 32LL << 20;

// An array of tokens x heads x d values: distances in elements.
struct Heads {
  void* p;
  int64_t token, head;
  int heads;
};

struct QkArgs {
  Heads q, k;        // inputs
  Heads yq, yk;      // results (their gradients in the reverse mode)
  Heads dq, dk;      // reverse mode: results
  const void *positions, *gamma_q, *gamma_k;
  const double* freqs;
  const int8_t* signs;
  float *dgamma_q, *dgamma_k, *partial;
  int64_t tokens;
  int d, pairs;
  float eps;
  bool wide, interleaved;
};

// Keys or values of a cache: bytes between pages.
struct Side4 {
  uint8_t *codes, *scales;
  int64_t codes_page, scales_page;
};
struct Cache4 {
  Side4 k, v;
  int pages, heads, d, page_log2;
};
struct Plan4 {
  const int32_t *starts, *lengths, *table;
  int64_t ld_table;
  int sequences, width;
};

struct Attn4Args {
  Cache4 cache;
  Plan4 plan;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* partial;
  int64_t q_token, q_head, out_token, out_head;
  int tokens, q_heads, group;
  float scale;
  bool causal;
  int window;  // 0: none
};

hipError_t launch_qk_norm_rope(const QkArgs& a, DT io, hipStream_t stream);
int64_t qk_norm_rope_vjp_workspace(int64_t tokens, int64_t heads, int64_t d);
hipError_t launch_qk_norm_rope_vjp(const QkArgs& a, DT io, hipStream_t stream);
hipError_t launch_kv4_write(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                            hipStream_t stream);
hipError_t launch_kv4_read(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                           hipStream_t stream);
int64_t kv4_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size,
                                int64_t sequences, int64_t width);
hipError_t launch_kv4_attention(const Attn4Args& a, hipStream_t stream);

// ------------------------------------------------------------ device side
// Eight values that are not read again before the caches have seen as much
// again as they hold: loads and stores that do not take their place there.
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
template <bool kStream>
__device__ __forceinline__ void load8(Raw8<uint16_t>& w, const uint16_t* p) {
  if constexpr (!kStream) return w.load(p, 8);
  const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_at2*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) w.w[i] = x[i];
}
template <bool kStream>
__device__ __forceinline__ void load8(Raw8<float>& w, const float* p) {
  if constexpr (!kStream) return w.load(p, 8);
  const u32x4_at4* q = reinterpret_cast<const u32x4_at4*>(p);
  const u32x4 x = __builtin_nontemporal_load(q), y = __builtin_nontemporal_load(q + 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w.w[i] = x[i];
    w.w[i + 4] = y[i];
  }
}
template <bool kStream>
__device__ __forceinline__ void put8(uint16_t* p, const float (&v)[8]) {
  if constexpr (!kStream) return store8(p, v);
  u32x4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack_bf16x2_hw(v[2 * i], v[2 * i + 1]);
  __builtin_nontemporal_store(x, reinterpret_cast<u32x4_at2*>(p));
}
template <bool kStream>
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  if constexpr (!kStream) return store8(p, v);
  u32x4 x, y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = __float_as_uint(v[i]);
    y[i] = __float_as_uint(v[i + 4]);
  }
  __builtin_nontemporal_store(x, reinterpret_cast<u32x4_at4*>(p));
  __builtin_nontemporal_store(y, reinterpret_cast<u32x4_at4*>(p) + 1);
}

// The last b of 0 .. n - 1 with f(b) <= value, or 0: f does not decrease, and
// value is the same in every lane of the wave, which looks at 64 places at a time.
// Whatever f gives, the result is in range.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int64_t value, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0;  // the answer is in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) >> 6, at = (lane + 1) * step;
    const bool past = at < n && f(lo + at) <= value;
    const int skip = __popcll(__ballot(past));
    lo += skip * step;
    n = min(step, n - skip * step);
  }
  return lo;
}

// The sequence whose rows include `row`, or the last one before it.
__device__ __forceinline__ int sequence_of(const Plan4& p, int64_t row) {
  return last_at_most(p.sequences, row, [&](int b) { return (int64_t)p.starts[b]; });
}

// The page of a sequence's tokens (page << page_log2) and on, -1 if it has none.
__device__ __forceinline__ int page_of(const Cache4& c, const Plan4& p, int seq, int64_t page) {
  if (page >= p.width) return -1;
  const int at = p.table[(int64_t)seq * p.ld_table + page];
  return at >= 0 && at < c.pages ? at : -1;
}

}  // namespace harp
