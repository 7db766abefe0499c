// The 4-bit cache as it is written and as it is read back.
//
// Both are bound by HBM.  A thread holds 8 consecutive values of a head: 16
// bytes of bf16 and one word of 8 codes; the 4 lanes of a quad share a block
// of 32 and find its maximum by two lane exchanges.  24000 tokens of 8 x 128,
// written: 30 us, 4.1 TB/s; read back: 25 us, 4.9 TB/s; 41 million values read:
// 38 us, 5.6 TB/s (the codes, a sixth of it, come from the caches).  In fp32 24000
// tokens written and read take 151 us, 3.1 TB/s.
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

// Where a wave's tokens lie.  It goes from token to token of one sequence; what
// it knows of the sequence and of the page serves while they last.
struct Walker {
  const Cache4& c;
  const Plan4& p;
  int seq = -1;
  int64_t first = 0, end = 0, len = 0;
  int64_t page = -1;   // the sequence's
  int64_t at = -1;     // the cache's; -1: none
  int in_page = 0;     // place in it; -1: before the sequence's beginning, -2: not of the call
  __device__ __forceinline__ Walker(const Cache4& c_, const Plan4& p_) : c(c_), p(p_) {}
  __device__ __forceinline__ void go(int64_t row) {
    if (row >= end || row < first) {
      seq = __builtin_amdgcn_readfirstlane(sequence_of(p, row));
      first = p.starts[seq];
      end = p.starts[seq + 1];
      len = p.lengths[seq];
      page = -1;
      if (row >= end || row < first) {
        in_page = -2;
        first = end = 0;
        return;
      }
    }
    const int64_t pos = len - (end - row);
    if (pos < 0) {
      in_page = -1;
      at = -1;
      return;
    }
    const int64_t now = pos >> c.page_log2;
    if (now != page) {
      page = now;
      at = page_of(c, p, seq, now);
    }
    in_page = (int)(pos - (now << c.page_log2));
  }
};

// A lane's 8 values of every token: the u-th of the token's, keys first.
template <typename T>
struct Unit {
  bool has, is_k;
  uint64_t io, codes, scales;  // addresses of token 0, of the page's first place
  Unit() = default;
  __device__ __forceinline__ Unit(const Cache4& c, const Heads& k, const Heads& v, int u) {
    const int per_head = c.d >> 3, side = c.heads * per_head;
    has = u < 2 * side;
    is_k = u < side;
    const int in = has ? is_k ? u : u - side : 0, head = in / per_head, col = (in - head * per_head) * 8;
    const Heads& s = is_k ? k : v;
    const Side4& o = is_k ? c.k : c.v;
    const int64_t row = (int64_t)head << c.page_log2;
    io = reinterpret_cast<uint64_t>(s.p) + (uint64_t)(head * s.head + col) * sizeof(T);
    codes = reinterpret_cast<uint64_t>(o.codes) + (uint64_t)(row * (c.d >> 1) + (col >> 1));
    scales = reinterpret_cast<uint64_t>(o.scales) + (uint64_t)(row * (c.d >> 5) + (col >> 5));
  }
  __device__ __forceinline__ T* row(const Heads& k, const Heads& v, int64_t row) const {
    return reinterpret_cast<T*>(io + (uint64_t)(row * (is_k ? k.token : v.token)) * sizeof(T));
  }
  __device__ __forceinline__ uint32_t* code(const Cache4& c, const Walker& w) const {
    return reinterpret_cast<uint32_t*>(codes + (uint64_t)(w.at * (is_k ? c.k.codes_page : c.v.codes_page) +
                                                          (int64_t)w.in_page * (c.d >> 1)));
  }
  __device__ __forceinline__ uint8_t* scale(const Cache4& c, const Walker& w) const {
    return reinterpret_cast<uint8_t*>(scales + (uint64_t)(w.at * (is_k ? c.k.scales_page : c.v.scales_page) +
                                                          (int64_t)w.in_page * (c.d >> 5)));
  }
};

// How the work is cut: a wave takes kRounds times 64 units of each of `run`
// tokens that follow one another, the next token's loads under way while it
// turns the present one's.
struct Cut {
  int parts, run;
  int64_t waves;
};

template <typename T, int kRounds, bool kStream>
__global__ __launch_bounds__(256) void kv4_write_kernel(Cache4 c, Plan4 p, Heads k, Heads v, int tokens, Cut cut) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (wave >= cut.waves) return;
  const uint32_t group = wave / (uint32_t)cut.parts, part = wave - group * cut.parts;
  const int64_t row0 = (int64_t)group * cut.run, row1 = min(row0 + cut.run, (int64_t)tokens);
  Unit<T> unit[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) unit[r] = Unit<T>(c, k, v, (part * kRounds + r) * 64 + lane);
  Walker walk(c, p);
  Raw8<T> next[kRounds];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (unit[r].has) load8<kStream>(next[r], unit[r].row(k, v, row));
  };
#pragma unroll
  for (int r = 0; r < kRounds; ++r) next[r].fill(0);
  load(row0);
  for (int64_t row = row0; row < row1; ++row) {
    walk.go(row);
    float f[kRounds][8];
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) f[r][i] = next[r][i];
    if (row + 1 < row1) load(row + 1);
    if (walk.in_page < 0 || walk.at < 0) continue;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      uint32_t top = amax8(f[r]);
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
      const uint32_t e = scale4(top);
      const float scale = __uint_as_float(e << 23);
      uint32_t codes = 0;
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][0], f[r][1], scale, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][2], f[r][3], scale, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][4], f[r][5], scale, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][6], f[r][7], scale, 3);
      if (e == 255) codes = 0;
      if (unit[r].has) {
        *unit[r].code(c, walk) = codes;
        if ((lane & 3) == 0) *unit[r].scale(c, walk) = (uint8_t)e;
      }
    }
  }
}

template <typename T, int kRounds, bool kStream>
__global__ __launch_bounds__(256) void kv4_read_kernel(Cache4 c, Plan4 p, Heads k, Heads v, int tokens, Cut cut) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (wave >= cut.waves) return;
  const uint32_t group = wave / (uint32_t)cut.parts, part = wave - group * cut.parts;
  const int64_t row0 = (int64_t)group * cut.run, row1 = min(row0 + cut.run, (int64_t)tokens);
  Unit<T> unit[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) unit[r] = Unit<T>(c, k, v, (part * kRounds + r) * 64 + lane);
  Walker walk(c, p);
  uint32_t codes[kRounds], e[kRounds];
  int kind = 0;  // of the token whose codes are held: Walker's in_page
  auto load = [&](int64_t row) {
    walk.go(row);
    kind = walk.in_page;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      codes[r] = 0;
      e[r] = kind < 0 ? 127 : 255;
      if (kind >= 0 && walk.at >= 0 && unit[r].has) {
        codes[r] = *unit[r].code(c, walk);
        e[r] = *unit[r].scale(c, walk);
      }
    }
  };
  load(row0);
  for (int64_t row = row0; row < row1; ++row) {
    uint32_t w[kRounds], s[kRounds];
    const int now = kind;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      w[r] = codes[r];
      s[r] = e[r];
    }
    if (row + 1 < row1) load(row + 1);
    if (now == -2) continue;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const float scale = __uint_as_float(s[r] << 23);  // the conversion reads the exponent only; 255 gives NaN
      const f32x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r], scale, 0);
      const f32x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r], scale, 1);
      const f32x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r], scale, 2);
      const f32x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[r], scale, 3);
      const float f[8] = {a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
      if (unit[r].has) put8<kStream>(unit[r].row(k, v, row), f);
    }
  }
}

// A wave for every 64 units of a token where tokens are few; four times as many
// where they are not, then runs of tokens, until the chip is about twice full.
template <int kRounds>
Cut cut_of(const Cache4& c, int tokens) {
  Cut r;
  const int rounds = (c.heads * (c.d >> 2) + 63) / 64;
  r.parts = (rounds + kRounds - 1) / kRounds;
  const int64_t all = (int64_t)tokens * r.parts;
  r.run = kRounds == 1 ? 1 : (int)std::min<int64_t>(std::max<int64_t>(1, all / 8192), 64);
  // launches are of up to 2^25 waves
  while ((((int64_t)tokens + r.run - 1) / r.run) * r.parts > (1 << 25)) r.run *= 2;
  r.waves = (((int64_t)tokens + r.run - 1) / r.run) * r.parts;
  return r;
}
bool few(const Cache4& c, int tokens) { return (int64_t)tokens * ((c.heads * (c.d >> 2) + 63) / 64) <= 8192; }

template <typename K>
hipError_t go(K kernel, const Cut& cut, const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens,
              hipStream_t stream) {
  hipLaunchKernelGGL(kernel, dim3((unsigned)((cut.waves + 3) / 4)), dim3(256), 0, stream, c, p, k, v, tokens, cut);
  return hipGetLastError();
}
template <typename T>
hipError_t write_go(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, hipStream_t stream) {
  if (few(c, tokens)) return go(kv4_write_kernel<T, 1, false>, cut_of<1>(c, tokens), c, p, k, v, tokens, stream);
  const bool streamed = 2LL * tokens * c.heads * c.d * (int)sizeof(T) >= kStreamBytes;
  return go(streamed ? kv4_write_kernel<T, 4, true> : kv4_write_kernel<T, 4, false>, cut_of<4>(c, tokens), c, p, k, v, tokens,
            stream);
}
template <typename T>
hipError_t read_go(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, hipStream_t stream) {
  if (few(c, tokens)) return go(kv4_read_kernel<T, 1, false>, cut_of<1>(c, tokens), c, p, k, v, tokens, stream);
  const bool streamed = 2LL * tokens * c.heads * c.d * (int)sizeof(T) >= kStreamBytes;
  return go(streamed ? kv4_read_kernel<T, 4, true> : kv4_read_kernel<T, 4, false>, cut_of<4>(c, tokens), c, p, k, v, tokens,
            stream);
}

}  // namespace

hipError_t launch_kv4_write(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                            hipStream_t stream) {
  return io == DT::F32 ? write_go<float>(c, p, k, v, tokens, stream) : write_go<uint16_t>(c, p, k, v, tokens, stream);
}
hipError_t launch_kv4_read(const Cache4& c, const Plan4& p, const Heads& k, const Heads& v, int tokens, DT io,
                           hipStream_t stream) {
  return io == DT::F32 ? read_go<float>(c, p, k, v, tokens, stream) : read_go<uint16_t>(c, p, k, v, tokens, stream);
}

}  // namespace harp
