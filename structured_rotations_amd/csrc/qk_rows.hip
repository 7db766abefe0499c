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
template <int kCtrl, int kBanks = 0xf>
__device__ __forceinline__ float dpp(float v, float old = 0.0f) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v),
                                                               kCtrl, 0xf, kBanks, kBanks == 0xf));
}
// v of lane ^ kMask.
template <int kMask>
__device__ __forceinline__ float lane_xor(float v) {
  if constexpr (kMask == 1) return dpp<0xb1>(v);        // quad_perm [1, 0, 3, 2]
  else if constexpr (kMask == 2) return dpp<0x4e>(v);   // quad_perm [2, 3, 0, 1]
  else if constexpr (kMask == 4) return dpp<0x124, 0xa>(v, dpp<0x12c, 0x5>(v));  // row_ror 4 and 12, by banks of 4
  else if constexpr (kMask == 8) return dpp<0x128>(v);  // row_ror 8
  else return __shfl_xor(v, kMask);
}
// Sum over the kLanes lanes of a head, in every one of them.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += dpp<0x141>(v);                           // the other 4 of 8 (mirrored)
  if constexpr (kLanes >= 16) v += dpp<0x140>(v);  // the other 8 of 16 (mirrored)
  if constexpr (kLanes >= 32) v += lane_xor<16>(v);
  if constexpr (kLanes >= 64) v += lane_xor<32>(v);
  return v;
}

template <int kMask>
__device__ __forceinline__ void butterfly(float (&v)[8], int lane, int d) {
  if (8 * kMask >= d) return;
  const float own = lane & kMask ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], own, lane_xor<kMask>(v[i]));
}
// Sylvester matrix of order d, not normalised: three stages within a lane, the
// others between lanes.
template <int kLanes>
__device__ __forceinline__ void hadamard(float (&v)[8], int lane, int d) {
#pragma unroll
  for (int m = 1; m < 8; m *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & m)) {
        const float a = v[i], b = v[i + m];
        v[i] = a + b;
        v[i + m] = a - b;
      }
  butterfly<1>(v, lane, d);
  butterfly<2>(v, lane, d);
  butterfly<4>(v, lane, d);
  if constexpr (kLanes >= 16) butterfly<8>(v, lane, d);
  if constexpr (kLanes >= 32) butterfly<16>(v, lane, d);
  if constexpr (kLanes >= 64) butterfly<32>(v, lane, d);
}

// A lane's share of a token's turn: out = c v + s partner(v), with the partner
// in lane `from` (pairs j, j + pairs) or in the same lane (interleaved pairs).
template <bool kInter>
struct Turn {
  float c[8], s[8];
  int from;

  // Angles reach 2^31 times a frequency: in turns and 64 bits until the whole
  // turns are gone.  What fp64 leaves off is 2^-53 of the angle.
  __device__ __forceinline__ void make(const QkArgs& a, int64_t token, int lane, float back) {
    const double pos = a.pairs == 0 ? 0.0  // no positions either
                       : a.wide     ? (double)static_cast<const int64_t*>(a.positions)[token]
                                    : (double)static_cast<const int32_t*>(a.positions)[token];
    const int e = 8 * lane;
    const bool turned = e < 2 * a.pairs, second = !kInter && e >= a.pairs;
    const int j0 = !turned ? 0 : kInter ? e / 2 : second ? e - a.pairs : e;
#pragma unroll
    for (int i = 0; i < (kInter ? 4 : 8); ++i) {
      float sn = 0.0f, cs = 1.0f;
      if (turned) {
        double t = pos * (a.freqs[j0 + i] * 0.15915494309189533577);
        t -= rint(t);
        sincospif(2.0f * (float)t, &sn, &cs);
      }
      sn *= back;
      if constexpr (kInter) {
        c[2 * i] = c[2 * i + 1] = cs;
        s[2 * i] = -sn;
        s[2 * i + 1] = sn;
      } else {
        c[i] = cs;
        s[i] = second ? sn : -sn;
      }
    }
    from = (threadIdx.x & 63) + (!turned || kInter ? 0 : (second ? -a.pairs : a.pairs) / 8);
  }
  __device__ __forceinline__ void apply(float (&v)[8]) const {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = kInter ? v[i ^ 1] : __shfl(v[i], from);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], c[i], s[i] * o[i]);
  }
};

// 1 / sqrt(mean(x^2) + eps), of any finite head: squares beyond fp32's range
// are summed again in other units.
template <int kLanes>
__device__ __forceinline__ float head_rstd(const float (&v)[8], float d, float eps, float least) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += v[i] * v[i];
  ss = head_sum<kLanes>(ss);
  float r = 1.0f / sqrtf(ss / d + eps);
  const bool far = !(ss >= least && ss < __uint_as_float(0x7f800000u));
  if (__any(far)) {  // the whole wave, so that every lane has its partners
    const float unit = ss < least ? 0x1p80f : 0x1p-80f;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += (v[i] * unit) * (v[i] * unit);
    t = head_sum<kLanes>(t);
    if (far) r = unit / sqrtf(t / d + eps * unit * unit);
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
template <typename T>
__device__ __forceinline__ T* head_at(const Heads& q, const Heads& k, int64_t token, int h, int col) {
  const bool is_q = h < q.heads;
  const Heads& s = is_q ? q : k;
  return static_cast<T*>(s.p) + token * s.token + (int64_t)(is_q ? h : h - q.heads) * s.head + col;
}
__device__ __forceinline__ void load_signs(const QkArgs& a, int lane, bool has, float (&sg)[8]) {
  const float unit = 1.0f / sqrtf((float)a.d);
#pragma unroll
  for (int i = 0; i < 8; ++i) sg[i] = has ? unit * (float)a.signs[8 * lane + i] : 0.0f;
}
__device__ __forceinline__ float least_of(float eps) { return eps < 0x1p-100f ? 0x1p-80f : 0.0f; }

// A wave takes `per` heads of a token.
template <typename T, int kLanes, bool kInter>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkArgs a, int per, int parts) {
  const HeadMap<kLanes> map(a.d);
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t token = unit / parts;
  if (token >= a.tokens) return;
  const int heads = a.q.heads + a.k.heads, first = (int)(unit - token * parts) * per;
  const int end = min(heads, first + per), col = 8 * map.lane;
  Raw8<T> next;
  auto load = [&](int h) {
    next.fill(0);
    if (map.has && h < end) next.load(head_at<const T>(a.q, a.k, token, h, col), 8);
  };
  load(first + map.slot);
  Turn<kInter> turn;
  turn.make(a, token, map.lane, 1.0f);
  Raw8<T> gq, gk;
  gq.fill(0x3f800000u);
  gk.fill(0x3f800000u);
  if (a.gamma_q && map.has) gq.load(static_cast<const T*>(a.gamma_q) + col, 8);
  if (a.gamma_k && map.has) gk.load(static_cast<const T*>(a.gamma_k) + col, 8);
  float sg[8];
  if (a.signs) load_signs(a, map.lane, map.has, sg);
  const float d = (float)a.d, least = least_of(a.eps);
  for (int h0 = first; h0 < end; h0 += map.kPar) {
    const int h = h0 + map.slot;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = next[i];
    load(h + map.kPar);
    const float r = head_rstd<kLanes>(v, d, a.eps, least);
    const bool is_q = h < a.q.heads;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (is_q ? gq[i] : gk[i]);
    turn.apply(v);
    if (a.signs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= sg[i];
      hadamard<kLanes>(v, map.lane, a.d);
    }
    if (map.has && h < end) store8(head_at<T>(a.yq, a.yk, token, h, col), v);
  }
}

// The reverse mode: workgroups walk over the parts of tokens, keeping their
// lanes' shares of the two dgammas in registers; the shares of a workgroup are
// added in order through LDS, those of the workgroups by the second kernel.
template <typename T, int kLanes, bool kInter>
__global__ __launch_bounds__(256) void qk_norm_rope_vjp_kernel(QkArgs a, int per, int parts) {
  const HeadMap<kLanes> map(a.d);
  const int heads = a.q.heads + a.k.heads, col = 8 * map.lane;
  const int64_t units = a.tokens * parts, step = (int64_t)gridDim.x * 4;
  Raw8<T> gq, gk;
  gq.fill(0x3f800000u);
  gk.fill(0x3f800000u);
  if (a.gamma_q && map.has) gq.load(static_cast<const T*>(a.gamma_q) + col, 8);
  if (a.gamma_k && map.has) gk.load(static_cast<const T*>(a.gamma_k) + col, 8);
  float sg[8], sum_q[8], sum_k[8];
  if (a.signs) load_signs(a, map.lane, map.has, sg);
#pragma unroll
  for (int i = 0; i < 8; ++i) sum_q[i] = sum_k[i] = 0.0f;
  const float d = (float)a.d, least = least_of(a.eps);
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < units; unit += step) {
    const int64_t token = unit / parts;
    const int first = (int)(unit - token * parts) * per, end = min(heads, first + per);
    Raw8<T> xn, gn;
    auto load = [&](int h) {
      xn.fill(0);
      gn.fill(0);
      if (map.has && h < end) {
        xn.load(head_at<const T>(a.q, a.k, token, h, col), 8);
        gn.load(head_at<const T>(a.yq, a.yk, token, h, col), 8);
      }
    };
    load(first + map.slot);
    Turn<kInter> turn;
    turn.make(a, token, map.lane, -1.0f);
    for (int h0 = first; h0 < end; h0 += map.kPar) {
      const int h = h0 + map.slot;
      float x[8], g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = xn[i];
        g[i] = gn[i];
      }
      load(h + map.kPar);
      const float r = head_rstd<kLanes>(x, d, a.eps, least);
      if (a.signs) {
        hadamard<kLanes>(g, map.lane, a.d);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= sg[i];
      }
      turn.apply(g);
      const bool is_q = h < a.q.heads, counts = h < end;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= r;
        const float t = counts ? g[i] * x[i] : 0.0f;
        sum_q[i] += is_q ? t : 0.0f;
        sum_k[i] += is_q ? 0.0f : t;
        g[i] *= is_q ? gq[i] : gk[i];
        dot += g[i] * x[i];
      }
      const float mean = head_sum<kLanes>(dot) / d;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * (g[i] - x[i] * mean);
      if (map.has && counts) store8(head_at<T>(a.dq, a.dk, token, h, col), g);
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
// 16 columns by 64 slices of them per workgroup.  parts == 0 writes zeros.
__global__ __launch_bounds__(1024) void qk_dgamma_kernel(const float* __restrict__ partial, int parts, int d,
                                                         float* __restrict__ dgamma_q, float* __restrict__ dgamma_k) {
  __shared__ float sum[64][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int col = (int)blockIdx.x * 16 + c;
  float s[4] = {0, 0, 0, 0};
  if (col < 2 * d)
    for (int p = slice; p < parts; p += 256)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p + 64 * i < parts) s[i] += partial[(int64_t)(p + 64 * i) * 2 * d + col];
  sum[slice][c] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (slice == 0 && col < 2 * d) {
    float t = 0.0f;
    for (int i = 0; i < 64; ++i) t += sum[i][c];
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
    if (a.interleaved)
      hipLaunchKernelGGL((qk_norm_rope_kernel<T, kLanes, true>), grid, dim3(256), 0, stream, b, s.per, s.parts);
    else
      hipLaunchKernelGGL((qk_norm_rope_kernel<T, kLanes, false>), grid, dim3(256), 0, stream, b, s.per, s.parts);
  }
}
template <typename T, int kLanes>
void vjp_go(const QkArgs& a, hipStream_t stream) {
  const Split s = split_of(a.tokens, a.q.heads + a.k.heads, kLanes);
  const int64_t groups = vjp_groups(a.tokens, a.q.heads + a.k.heads, a.d);
  if (groups > 0) {
    const dim3 grid((unsigned)groups);
    if (a.interleaved)
      hipLaunchKernelGGL((qk_norm_rope_vjp_kernel<T, kLanes, true>), grid, dim3(256), 0, stream, a, s.per, s.parts);
    else
      hipLaunchKernelGGL((qk_norm_rope_vjp_kernel<T, kLanes, false>), grid, dim3(256), 0, stream, a, s.per, s.parts);
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
