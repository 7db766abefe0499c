// Heads of queries and keys: root-mean-square norm, position rotation and
// signed Hadamard rotation in one pass over them, and its reverse mode.
//
// All of it is bound by HBM at many tokens: a head is read once and written
// once.  A head of d values lies in 8, 16, 32 or 64 lanes with 8 consecutive
// values each (16-byte loads of bf16), so that its sums, the partners of a
// turn and the Hadamard stages are exchanges between lanes, with no LDS.  A
// wave holds 64 / lanes heads at a time and walks over the heads of one token,
// whose angles it computes once.
#include <algorithm>

#include "kv4.h"
#include "q8.h"

namespace harp {
namespace {

// v of another lane of the same 16: a DPP control.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xf, 0xf, true));
}
// Sum over the kLanes lanes of a head, in every one of them.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp<0xb1>(v);                            // lane ^ 1
  v += dpp<0x4e>(v);                            // lane ^ 2
  v += dpp<0x141>(v);                           // the other 4 of 8 (mirrored)
  if constexpr (kLanes >= 16) v += dpp<0x140>(v);  // the other 8 of 16 (mirrored)
  if constexpr (kLanes >= 32) v += __shfl_xor(v, 16);
  if constexpr (kLanes >= 64) v += __shfl_xor(v, 32);
  return v;
}

// One stage between lanes, but for a sign: with p the partner's value, lanes of
// bit 0 get v + p and those of bit 1 get v - p, where a - b = p - v is meant.
// The sign left out is the same in both partners of every later stage, so all
// of them are made good at the end, by the parity of the lane's bits.
//
// Written out: the exchange is an operand of the multiply-add, which the
// compiler makes two instructions of, with waits between them.  A value may be
// read that way two instructions after it is written, hence the waits in front;
// eight values one after the other keep that distance from stage to stage.
#define HARP_STAGE(ctrl)                                                              \
  asm("s_nop 1\n\t"                                                                  \
      "v_fmac_f32_dpp %0, %0, %8 " ctrl "\n\tv_fmac_f32_dpp %1, %1, %8 " ctrl "\n\t" \
      "v_fmac_f32_dpp %2, %2, %8 " ctrl "\n\tv_fmac_f32_dpp %3, %3, %8 " ctrl "\n\t" \
      "v_fmac_f32_dpp %4, %4, %8 " ctrl "\n\tv_fmac_f32_dpp %5, %5, %8 " ctrl "\n\t" \
      "v_fmac_f32_dpp %6, %6, %8 " ctrl "\n\tv_fmac_f32_dpp %7, %7, %8 " ctrl         \
      : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]) \
      : "v"(other))
// The same onto values of their own, for an exchange that takes two controls.
#define HARP_STAGE_ONTO(ctrl)                                                           \
  asm("s_nop 1\n\t"                                                                    \
      "v_fmac_f32_dpp %0, %8, %16 " ctrl "\n\tv_fmac_f32_dpp %1, %9, %16 " ctrl "\n\t"  \
      "v_fmac_f32_dpp %2, %10, %16 " ctrl "\n\tv_fmac_f32_dpp %3, %11, %16 " ctrl "\n\t" \
      "v_fmac_f32_dpp %4, %12, %16 " ctrl "\n\tv_fmac_f32_dpp %5, %13, %16 " ctrl "\n\t" \
      "v_fmac_f32_dpp %6, %14, %16 " ctrl "\n\tv_fmac_f32_dpp %7, %15, %16 " ctrl          \
      : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(w[4]), "+v"(w[5]), "+v"(w[6]), "+v"(w[7]) \
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "v"(other))
template <int kMask>
__device__ __forceinline__ void butterfly(float (&v)[8], int lane) {
  const float other = lane & kMask ? -1.0f : 1.0f;
  if constexpr (kMask == 1) {
    HARP_STAGE("quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf");
  } else if constexpr (kMask == 2) {
    HARP_STAGE("quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf");
  } else if constexpr (kMask == 4) {  // by banks of 4 lanes: from 4 above, from 4 below
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i];
    HARP_STAGE_ONTO("row_ror:12 row_mask:0xf bank_mask:0x5");
    HARP_STAGE_ONTO("row_ror:4 row_mask:0xf bank_mask:0xa");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i];
  } else if constexpr (kMask == 8) {
    HARP_STAGE("row_ror:8 row_mask:0xf bank_mask:0xf");
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(__shfl_xor(v[i], kMask), other, v[i]);
  }
}
#undef HARP_STAGE
#undef HARP_STAGE_ONTO
// Sylvester matrix of order d, not normalised: stages between lanes, then three
// within a lane, of which the last one takes the sign.
template <int kLanes>
__device__ __forceinline__ void hadamard(float (&v)[8], int lane, int d) {
  if constexpr (kLanes == 8) {  // d = 8 to 64
    if (d > 8) butterfly<1>(v, lane);
    if (d > 16) butterfly<2>(v, lane);
    if (d > 32) butterfly<4>(v, lane);
  } else {  // d = 8 lanes: a power of two, of half that it would have half the lanes
    butterfly<1>(v, lane);
    butterfly<2>(v, lane);
    butterfly<4>(v, lane);
    butterfly<8>(v, lane);
    if constexpr (kLanes >= 32) butterfly<16>(v, lane);
    if constexpr (kLanes >= 64) butterfly<32>(v, lane);
  }
#pragma unroll
  for (int m = 1; m < 4; m *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & m)) {
        const float a = v[i], b = v[i + m];
        v[i] = a + b;
        v[i + m] = a - b;
      }
  const float sign = __popc(lane & (d / 8 - 1)) & 1 ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = v[i], b = v[i + 4] * sign;
    v[i] = fmaf(a, sign, b);
    v[i + 4] = fmaf(a, sign, -b);
  }
}

// The angle pos times freq (radians) in turns, less whole ones.  It reaches 2^31
// times a frequency of 8, and 2^-53 of that is not little: 1 / 2 pi is the sum of
// two fp64 numbers, and what each product leaves off is kept until the whole turns
// are gone, which leaves an error of 2^-53 turns.  (Products are not to be joined
// with what follows them, or what they leave off would count twice.)
__device__ __forceinline__ double fraction_of_turn(double pos, double freq) {
#pragma clang fp contract(off)
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnRest = -0x1.6b01ec5417056p-57;
  const double per = freq * kTurn, per_rest = fma(freq, kTurn, -per) + freq * kTurnRest;
  const double turns = pos * per, rest = fma(pos, per, -turns) + pos * per_rest;
  return (turns - rint(turns)) + rest;
}

// A lane's share of a token's turn: out = c v + s partner(v), with the partner
// in lane `from` (pairs j, j + pairs) or in the same lane (interleaved pairs).
template <int kLanes, bool kInter>
struct Turn {
  float c[8], s[8];
  int from;

  // Each lane computes every 64th pair's angle, and gets what it needs from the
  // others.  What the rounding of a fraction of a turn to fp32 leaves off turns sine
  // and cosine once more.
  __device__ __forceinline__ void make(const QkArgs& a, int64_t token, int lane, float back) {
    constexpr int kRounds = kLanes <= 16 ? 1 : kLanes / 16;  // pairs are at most 4 to a lane of a head
    const int self = threadIdx.x & 63;
    const double pos = a.pairs == 0 ? 0.0  // no positions either
                       : a.wide     ? (double)static_cast<const int64_t*>(a.positions)[token]
                                    : (double)static_cast<const int32_t*>(a.positions)[token];
    float sn[kRounds], cs[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      sn[r] = 0.0f;
      cs[r] = 1.0f;
      if (64 * r + self < a.pairs) {
        const double t = fraction_of_turn(pos, a.freqs[64 * r + self]);
        const float near = (float)t, off = 6.28318530717958648f * (float)(t - (double)near);
        float x, y;
        sincospif(2.0f * near, &x, &y);
        sn[r] = fmaf(y, off, x) * back;
        cs[r] = fmaf(-x, off, y);
      }
    }
    const int e = 8 * lane;
    const bool turned = e < 2 * a.pairs, second = !kInter && e >= a.pairs;
    const int j0 = !turned ? 0 : kInter ? e / 2 : second ? e - a.pairs : e;
#pragma unroll
    for (int i = 0; i < (kInter ? 4 : 8); ++i) {
      float x = __shfl(sn[0], (j0 + i) & 63), y = __shfl(cs[0], (j0 + i) & 63);
#pragma unroll
      for (int r = 1; r < kRounds; ++r) {
        const float xr = __shfl(sn[r], (j0 + i) & 63), yr = __shfl(cs[r], (j0 + i) & 63);
        if (j0 >= 64 * r) {
          x = xr;
          y = yr;
        }
      }
      if (!turned) {
        x = 0.0f;
        y = 1.0f;
      }
      if constexpr (kInter) {
        c[2 * i] = c[2 * i + 1] = y;
        s[2 * i] = -x;
        s[2 * i + 1] = x;
      } else {
        c[i] = y;
        s[i] = second ? x : -x;
      }
    }
    from = self + (!turned || kInter ? 0 : (second ? -a.pairs : a.pairs) / 8);
  }
  // What the turned values are multiplied by next.
  __device__ __forceinline__ void times(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] *= f[i];
      s[i] *= f[i];
    }
  }
  __device__ __forceinline__ void apply(float (&v)[8]) const {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = kInter ? v[i ^ 1] : __shfl(v[i], from);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], c[i], s[i] * o[i]);
  }
};

// 1 / sqrt(x) of an x from 2^-100 on: the hardware's estimate (an ulp off) and
// one step of Newton's method, with what x r^2 is off 1 to twice fp32's width.
__device__ __forceinline__ float rsqrt_of(float x) {
  const float r = __builtin_amdgcn_rsqf(x), t = x * r;
  const float e = fmaf(-t, r, 1.0f) - fmaf(x, r, -t) * r;
  return fmaf(0.5f * r, e, r);
}

// 1 / sqrt(mean(x^2) + eps).  A head whose squares leave fp32's range is brought
// into it first, by a power of two that `unit` tells (1 for all others): v and the
// result are then of the head in those units, of which v times the result does not
// depend.  The smallest heads' 1 / rms is more than fp32 holds.
// (0x1p100: squares from 2^-298 on become 2^-98, and their sum, below 2^-80, 2^120;
// eps is below 2^-100 where they are taken for small.)
template <int kLanes>
__device__ __forceinline__ float head_rstd(float (&v)[8], float d, float eps, float least, float* unit) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += v[i] * v[i];
  ss = head_sum<kLanes>(ss);
  const float mean = fmaf(ss, 1.0f / d, eps);
  float r = rsqrt_of(mean);
  const bool far = !(ss >= least && mean < __uint_as_float(0x7f800000u));
  *unit = 1.0f;
  if (__any(far)) {  // the whole wave, so that every lane has its partners
    if (far) *unit = ss < least ? 0x1p100f : 0x1p-80f;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= *unit;
      t += v[i] * v[i];
    }
    t = head_sum<kLanes>(t);
    if (far) r = 1.0f / sqrtf(t / d + eps * *unit * *unit);
  }
  return r;
}

// Where a wave's heads lie: lane `lane` of the `slot`th of kPar heads at a time.
template <int kLanes>
struct HeadMap {
  static constexpr int kPar = 64 / kLanes;
  int lane, slot;
  bool has;
  __device__ __forceinline__ explicit HeadMap(int d) {
    lane = threadIdx.x & (kLanes - 1);
    slot = (threadIdx.x & 63) / kLanes;
    has = 8 * lane < d;
  }
};
// The places of a wave's heads in one pair of arrays, which go from head to head
// by additions.  (Where a head is none of the one array its address there is not
// used.)
template <typename T, int kPar>
struct Walk {
  uint64_t q, k, q_step, k_step;
  __device__ __forceinline__ Walk(const Heads& sq, const Heads& sk, int64_t token, int h, int col) {
    q = reinterpret_cast<uint64_t>(sq.p) + (uint64_t)(token * sq.token + h * sq.head + col) * sizeof(T);
    k = reinterpret_cast<uint64_t>(sk.p) + (uint64_t)(token * sk.token + (h - sq.heads) * sk.head + col) * sizeof(T);
    q_step = (uint64_t)sq.head * (kPar * sizeof(T));
    k_step = (uint64_t)sk.head * (kPar * sizeof(T));
  }
  __device__ __forceinline__ T* at(bool is_q) const { return reinterpret_cast<T*>(is_q ? q : k); }
  __device__ __forceinline__ void next() {
    q += q_step;
    k += k_step;
  }
};
__device__ __forceinline__ void load_signs(const QkArgs& a, int lane, bool has, float (&sg)[8]) {
  const float unit = rsqrt_of((float)a.d);
  RawCodes w;  // 8 bytes
  w.w[0] = w.w[1] = 0;
  if (has) w.load(reinterpret_cast<const uint8_t*>(a.signs) + 8 * lane, 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) sg[i] = unit * (float)(int8_t)(w.w[i >> 2] >> (8 * (i & 3)));
}
template <typename T>
__device__ __forceinline__ void load_gamma(const void* gamma, int col, bool has, float (&g)[8]) {
  Raw8<T> w;
  w.fill(0x3f800000u);
  if (gamma && has) w.load(static_cast<const T*>(gamma) + col, 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = w[i];
}
__device__ __forceinline__ float least_of(float eps) { return eps < 0x1p-100f ? 0x1p-80f : 0.0f; }

// A wave takes `per` heads of a token.  16384 x 32+8 x 128 in bf16, 336 MB: 63 to 66
// us, 5.1 to 5.3 TB/s, which is a copy's rate; the vector unit is busy 86% of it.  In
// fp32 148 us, 4.5 TB/s.
// One token: 3.7 us.
template <typename T, int kLanes, bool kInter, bool kStream>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkArgs a, int per, int parts) {
  const HeadMap<kLanes> map(a.d);
  // (units of a launch are less than 2^26)
  const uint32_t unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int token = (int)(unit / (uint32_t)parts);
  if (token >= a.tokens) return;
  const int heads = a.q.heads + a.k.heads, first = ((int)unit - token * parts) * per;
  const int end = min(heads, first + per), col = 8 * map.lane;
  Raw8<T> next;
  Walk<const T, map.kPar> in(a.q, a.k, token, first + map.slot, col);
  Walk<T, map.kPar> to(a.yq, a.yk, token, first + map.slot, col);
  auto load = [&](int h) {
    next.fill(0);
    if (map.has && h < end) load8<kStream>(next, in.at(h < a.q.heads));
    in.next();
  };
  load(first + map.slot);
  Turn<kLanes, kInter> turn;
  turn.make(a, token, map.lane, 1.0f);
  float gq[8], gk[8];
  load_gamma<T>(a.gamma_q, col, map.has, gq);
  load_gamma<T>(a.gamma_k, col, map.has, gk);
  if (a.signs) {
    float sg[8];
    load_signs(a, map.lane, map.has, sg);
    turn.times(sg);
  }
  const float d = (float)a.d, least = least_of(a.eps);
  for (int h0 = first; h0 < end; h0 += map.kPar) {
    const int h = h0 + map.slot;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = next[i];
    load(h + map.kPar);
    float in_units;  // v times r does not depend on it
    const float r = head_rstd<kLanes>(v, d, a.eps, least, &in_units);
    const bool is_q = h < a.q.heads;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (is_q ? gq[i] : gk[i]);
    turn.apply(v);
    if (a.signs) hadamard<kLanes>(v, map.lane, a.d);
    if (map.has && h < end) put8<kStream>(to.at(is_q), v);
    to.next();
  }
}

// The reverse mode: workgroups walk over the parts of tokens, keeping their
// lanes' shares of the two dgammas in registers; the shares of a workgroup are
// added in order through LDS, those of the workgroups by the second kernel.  16384
// x 32+8 x 128 in bf16, 503 MB: 100 to 106 us with it, 4.7 to 5.0 TB/s; in fp32, 1007
// MB, 216 us, 4.7 TB/s, though 13 of its 128 registers spill.
template <typename T, int kLanes, bool kInter, bool kStream>
__global__ __launch_bounds__(256, 4) void qk_norm_rope_vjp_kernel(QkArgs a, int per, int parts) {
  const HeadMap<kLanes> map(a.d);
  const int heads = a.q.heads + a.k.heads, col = 8 * map.lane;
  // tokens up to 2^30 in one part, or up to 4096 in several
  const uint32_t units = (uint32_t)(a.tokens * parts), step = gridDim.x * 4;
  float gq[8], gk[8], sg[8], sum_q[8], sum_k[8];
  load_gamma<T>(a.gamma_q, col, map.has, gq);
  load_gamma<T>(a.gamma_k, col, map.has, gk);
  if (a.signs) load_signs(a, map.lane, map.has, sg);
#pragma unroll
  for (int i = 0; i < 8; ++i) sum_q[i] = sum_k[i] = 0.0f;
  const float d = (float)a.d, least = least_of(a.eps);
  for (uint32_t unit = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6)); unit < units; unit += step) {
    const int token = (int)(unit / (uint32_t)parts);
    const int first = ((int)unit - token * parts) * per, end = min(heads, first + per);
    Raw8<T> xn, gn;
    Walk<const T, map.kPar> x_at(a.q, a.k, token, first + map.slot, col), g_at(a.yq, a.yk, token, first + map.slot, col);
    Walk<T, map.kPar> to(a.dq, a.dk, token, first + map.slot, col);
    auto load = [&](int h) {
      xn.fill(0);
      gn.fill(0);
      if (map.has && h < end) {
        load8<kStream>(xn, x_at.at(h < a.q.heads));
        load8<kStream>(gn, g_at.at(h < a.q.heads));
      }
      x_at.next();
      g_at.next();
    };
    load(first + map.slot);
    Turn<kLanes, kInter> turn;
    turn.make(a, token, map.lane, -1.0f);
    for (int h0 = first; h0 < end; h0 += map.kPar) {
      const int h = h0 + map.slot;
      float x[8], g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = xn[i];  // zeros where there is no head: nothing is added for it
        g[i] = gn[i];
      }
      load(h + map.kPar);
      float in_units;
      const float r = head_rstd<kLanes>(x, d, a.eps, least, &in_units);
      if (a.signs) {
        hadamard<kLanes>(g, map.lane, a.d);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= sg[i];
      }
      turn.apply(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = h < end ? x[i] * r : 0.0f;
      const bool is_q = h < a.q.heads;
      if (a.partial) {
        if (h0 + map.kPar <= a.q.heads) {  // all of the wave's heads are queries'
#pragma unroll
          for (int i = 0; i < 8; ++i) sum_q[i] = fmaf(g[i], x[i], sum_q[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // (no product with 0: a gradient may be infinite or NaN)
            const float sum = fmaf(g[i], x[i], is_q ? sum_q[i] : sum_k[i]);
            sum_q[i] = is_q ? sum : sum_q[i];
            sum_k[i] = is_q ? sum_k[i] : sum;
          }
        }
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] *= is_q ? gq[i] : gk[i];
        dot = fmaf(g[i], x[i], dot);
      }
      const float mean = head_sum<kLanes>(dot) * (1.0f / d);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * fmaf(x[i], -mean, g[i]);
      if (__any(in_units != 1.0f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= in_units;
      }
      if (map.has && h < end) put8<kStream>(to.at(is_q), g);
      to.next();
    }
  }
  if (a.partial == nullptr) return;
  constexpr int kRows = 256 / kLanes, kWidth = kLanes * 8;
  __shared__ float share[kRows][kWidth + 1];
  const int row = threadIdx.x / kLanes;
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) share[row][col + i] = side ? sum_k[i] : sum_q[i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += 256) {
      float t = 0.0f;
      for (int i = 0; i < kRows; ++i) t += share[i][c];
      a.partial[((int64_t)blockIdx.x * 2 + side) * a.d + c] = t;
    }
  }
}

// dgamma_q and dgamma_k = the workgroups' partial sums added in a fixed order:
// 16 columns by 64 slices of them per workgroup, then a wave for each column.
// parts == 0 writes zeros.  (1024 parts of 256 columns: 7 us with four loads in
// flight and the slices added by one thread.)
__global__ __launch_bounds__(1024) void qk_dgamma_kernel(const float* __restrict__ partial, int parts, int d,
                                                         float* __restrict__ dgamma_q, float* __restrict__ dgamma_k) {
  __shared__ float sum[64][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  float s[4] = {0, 0, 0, 0};
  {
    const int col = (int)blockIdx.x * 16 + c;
    if (col < 2 * d)
      for (int p = slice; p < parts; p += 1024) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = p + 64 * i < parts ? partial[(int64_t)(p + 64 * i) * 2 * d + col] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i & 3] += x[i];
      }
  }
  sum[slice][c] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  const int col = (int)blockIdx.x * 16 + (threadIdx.x >> 6);
  const float t = wave_sum(sum[threadIdx.x & 63][threadIdx.x >> 6]);
  if ((threadIdx.x & 63) == 0 && col < 2 * d) {
    float* out = col < d ? dgamma_q : dgamma_k;
    if (out) out[col < d ? col : col - d] = t;
  }
}

// Heads per wave: all of a token's where there are tokens enough to fill the
// chip (its angles are then computed once), fewer down to one round where not.
struct Split {
  int per, parts;
};
Split split_of(int64_t tokens, int heads, int lanes) {
  const int par = 64 / lanes, rounds = (heads + par - 1) / par;
  int parts = (int)std::min<int64_t>(rounds, std::max<int64_t>(1, 4096 / std::max<int64_t>(1, tokens)));
  const int per = (rounds + parts - 1) / parts * par;
  return {per, (heads + per - 1) / per};
}
int lanes_of(int64_t d) { return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : 64; }

int64_t vjp_groups(int64_t tokens, int64_t heads, int64_t d) {
  const Split s = split_of(tokens, (int)heads, lanes_of(d));
  return std::min<int64_t>((tokens * s.parts + 3) / 4, 1024);
}

template <typename T>
bool streamed(const QkArgs& a) {
  return a.tokens * (a.q.heads + a.k.heads) * a.d * (int)sizeof(T) >= kStreamBytes;
}

template <typename T, int kLanes>
void go(const QkArgs& a, hipStream_t stream) {
  const Split s = split_of(a.tokens, a.q.heads + a.k.heads, kLanes);
  // 2^22 workgroups a launch
  const int64_t most = (int64_t)(1 << 24) / s.parts;
  for (int64_t t = 0; t < a.tokens; t += most) {
    QkArgs b = a;
    b.tokens = std::min(most, a.tokens - t);
    const int eb = (int)sizeof(T);
    for (Heads* h : {&b.q, &b.k, &b.yq, &b.yk})
      if (h->p) h->p = static_cast<char*>(h->p) + t * h->token * eb;
    if (a.positions) b.positions = static_cast<const char*>(a.positions) + t * (a.wide ? 8 : 4);
    const dim3 grid((unsigned)((b.tokens * s.parts + 3) / 4));
    const auto kernel = a.interleaved ? streamed<T>(a) ? qk_norm_rope_kernel<T, kLanes, true, true>
                                                       : qk_norm_rope_kernel<T, kLanes, true, false>
                        : streamed<T>(a) ? qk_norm_rope_kernel<T, kLanes, false, true>
                                         : qk_norm_rope_kernel<T, kLanes, false, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, b, s.per, s.parts);
  }
}
template <typename T, int kLanes>
void vjp_go(const QkArgs& a, hipStream_t stream) {
  const Split s = split_of(a.tokens, a.q.heads + a.k.heads, kLanes);
  const int64_t groups = vjp_groups(a.tokens, a.q.heads + a.k.heads, a.d);
  if (groups > 0) {
    const dim3 grid((unsigned)groups);
    const auto kernel = a.interleaved ? streamed<T>(a) ? qk_norm_rope_vjp_kernel<T, kLanes, true, true>
                                                       : qk_norm_rope_vjp_kernel<T, kLanes, true, false>
                        : streamed<T>(a) ? qk_norm_rope_vjp_kernel<T, kLanes, false, true>
                                         : qk_norm_rope_vjp_kernel<T, kLanes, false, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, s.per, s.parts);
  }
  if (a.dgamma_q || a.dgamma_k)
    hipLaunchKernelGGL(qk_dgamma_kernel, dim3((2 * a.d + 15) / 16), dim3(1024), 0, stream, a.partial, (int)groups, a.d,
                       a.dgamma_q, a.dgamma_k);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkArgs& a, DT io, hipStream_t stream) {
  const bool f = io == DT::F32;
  switch (lanes_of(a.d)) {
    case 8: f ? go<float, 8>(a, stream) : go<uint16_t, 8>(a, stream); break;
    case 16: f ? go<float, 16>(a, stream) : go<uint16_t, 16>(a, stream); break;
    case 32: f ? go<float, 32>(a, stream) : go<uint16_t, 32>(a, stream); break;
    default: f ? go<float, 64>(a, stream) : go<uint16_t, 64>(a, stream); break;
  }
  return hipGetLastError();
}

int64_t qk_norm_rope_vjp_workspace(int64_t tokens, int64_t heads, int64_t d) {
  return vjp_groups(tokens, heads, d) * 2 * d * 4;
}

hipError_t launch_qk_norm_rope_vjp(const QkArgs& a, DT io, hipStream_t stream) {
  const bool f = io == DT::F32;
  switch (lanes_of(a.d)) {
    case 8: f ? vjp_go<float, 8>(a, stream) : vjp_go<uint16_t, 8>(a, stream); break;
    case 16: f ? vjp_go<float, 16>(a, stream) : vjp_go<uint16_t, 16>(a, stream); break;
    case 32: f ? vjp_go<float, 32>(a, stream) : vjp_go<uint16_t, 32>(a, stream); break;
    default: f ? vjp_go<float, 64>(a, stream) : vjp_go<uint16_t, 64>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace harp
