// extern "C" entry points of attention over a 4-bit cache (include/harp.h):
// every argument is checked on the host, before any HIP call, then the
// launchers run.
#include <cmath>
#include <cstdint>

#include "args.h"
#include "harp.h"
#include "kv4.h"

using namespace harp;

namespace {

constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxPlan = 1LL << 24;  // sequences, pages of one

// An array of tokens x heads x d values as the matrix that it is part of: its
// rows are tokens if a token's heads lie within the distance of tokens, else
// heads.
harp_status as_mat(const char* name, const void* p, int64_t token, int64_t head, int64_t tokens, int64_t heads,
                   int64_t d, int eb, Mat* m) {
  if (heads == 1) head = d;
  if (tokens == 1) token = head > INT64_MAX / heads ? head : head * heads;
  if (token < d || head < d)
    return fail(HARP_ERR_INVALID_ARG, "%s: tokens or heads are less than a head's length %lld apart", name, (long long)d);
  if (head <= (INT64_MAX - d) / heads && token >= (heads - 1) * head + d)
    *m = {name, p, token, tokens, (heads - 1) * head + d, eb};
  else if (token <= (INT64_MAX - d) / tokens && head >= (tokens - 1) * token + d)
    *m = {name, p, head, heads, (tokens - 1) * token + d, eb};
  else
    return fail(HARP_ERR_INVALID_ARG, "%s: tokens and heads overlap (distances %lld and %lld)", name, (long long)token,
                (long long)head);
  return check(*m);
}

// A heads argument.
struct HeadsArg {
  const char* name;
  const void* p;
  int64_t token, head, heads;
  Mat m;
};
harp_status check(HeadsArg* a, int64_t tokens, int64_t d, int eb) {
  return as_mat(a->name, a->p, a->token, a->head, tokens, a->heads, d, eb, &a->m);
}
harp_status apart(const HeadsArg& out, const HeadsArg& in, bool same, int64_t tokens) {
  if (same && out.p == in.p && out.heads == in.heads && (tokens == 1 || out.token == in.token) &&
      (out.heads == 1 || out.head == in.head))
    return HARP_OK;
  return check_apart(out.m, in.m, false);
}
Heads heads_of(const HeadsArg& a) { return {const_cast<void*>(a.p), a.token, a.head, (int)a.heads}; }

harp_status check_vec(const char* name, const void* p, int64_t n, int eb, Mat* m) {
  *m = {name, p, n, 1, n, eb};
  return check(*m);
}

// ------------------------------------------------------------ norm and turn
struct QkIn {
  HeadsArg q, k;
  int64_t tokens, d;
  harp_dtype io;
  const void* positions;
  int32_t wide;
  const double* freqs;
  int64_t pairs;
  const void *gamma_q, *gamma_k;
  float eps;
  const int8_t* signs;
  Mat small[5];  // positions, freqs, gammas, signs
  int n_small = 0;
  bool has_k() const { return k.heads > 0; }
};
harp_status check_sizes(QkIn* a) {
  if (!io_ok(a->io)) return fail(HARP_ERR_UNSUPPORTED, "io_dtype must be HARP_F32 or HARP_BF16");
  TRY(check_size("tokens", a->tokens, 0, kMaxSize));
  TRY(check_size("q_heads", a->q.heads, 1, kMaxHeads));
  TRY(check_size("k_heads", a->k.heads, 0, kMaxHeads));
  TRY(check_size("d", a->d, 8, 512));
  if (a->d % 8) return fail(HARP_ERR_UNSUPPORTED, "d must be a multiple of 8, got %lld", (long long)a->d);
  TRY(check_size("pairs", a->pairs, 0, a->d / 2));
  if (a->pairs % 8) return fail(HARP_ERR_UNSUPPORTED, "pairs must be a multiple of 8, got %lld", (long long)a->pairs);
  if (a->signs && !is_pow2(a->d))
    return fail(HARP_ERR_UNSUPPORTED, "with signs d must be a power of two, got %lld", (long long)a->d);
  if (!(a->eps >= 0.0f)) return fail(HARP_ERR_INVALID_ARG, "eps must be at least 0");
  if (a->k.heads == 0 && (a->k.p || a->gamma_k))
    return fail(HARP_ERR_INVALID_ARG, "k and gamma_k go with k_heads > 0 only");
  return HARP_OK;
}
harp_status check_inputs(QkIn* a) {
  const int eb = size_of(a->io);
  TRY(check(&a->q, a->tokens, a->d, eb));
  if (a->has_k()) TRY(check(&a->k, a->tokens, a->d, eb));
  auto small = [&](const char* name, const void* p, int64_t n, int bytes) {
    return check_vec(name, p, n, bytes, &a->small[a->n_small++]);
  };
  if (a->pairs > 0) {
    TRY(small("positions", a->positions, a->tokens, a->wide ? 8 : 4));
    TRY(small("freqs", a->freqs, a->pairs, 8));
  }
  if (a->gamma_q) TRY(small("gamma_q", a->gamma_q, a->d, eb));
  if (a->gamma_k) TRY(small("gamma_k", a->gamma_k, a->d, eb));
  if (a->signs) TRY(small("signs", a->signs, a->d, 1));
  return HARP_OK;
}
QkArgs args_of(const QkIn& a, bool interleaved) {
  QkArgs g{};
  g.q = heads_of(a.q);
  g.k = heads_of(a.k);
  g.positions = a.positions;
  g.freqs = a.freqs;
  g.gamma_q = a.gamma_q;
  g.gamma_k = a.gamma_k;
  g.signs = a.signs;
  g.tokens = a.tokens;
  g.d = (int)a.d;
  g.pairs = (int)a.pairs;
  g.eps = a.eps;
  g.wide = a.wide != 0;
  g.interleaved = interleaved;
  return g;
}

// ---------------------------------------------------------- cache and plan
struct CacheArg {
  const uint8_t* p[4];  // k codes, k scales, v codes, v scales
  int64_t page[4];      // bytes between pages
  int64_t pages, heads, page_size, d;
  const int32_t *starts, *lengths, *table;
  int64_t ld_table, sequences, width;
  Mat m[4], plan[3];
};
harp_status check_sizes(const CacheArg& c) {
  TRY(check_size("pages", c.pages, 1, kMaxSize));
  TRY(check_size("kv_heads", c.heads, 1, kMaxHeads));
  TRY(check_size("page_size", c.page_size, 16, 1 << 20));
  if (!is_pow2(c.page_size))
    return fail(HARP_ERR_UNSUPPORTED, "page_size must be a power of two, got %lld", (long long)c.page_size);
  TRY(check_size("d", c.d, 32, 256));
  if (c.d % kBlk4) return fail(HARP_ERR_UNSUPPORTED, "d must be a multiple of 32, got %lld", (long long)c.d);
  TRY(check_size("sequences", c.sequences, 0, kMaxPlan));
  TRY(check_size("width", c.width, 1, kMaxPlan));
  return check_size("sequences x kv_heads", c.sequences * c.heads, 0, kMaxSize);
}
harp_status check(CacheArg* c) {
  const char* names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
  for (int i = 0; i < 4; ++i) {
    const int64_t bytes = c->heads * c->page_size * (c->d / (i % 2 ? kBlk4 : 2));
    if (c->pages == 1) c->page[i] = bytes;
    c->m[i] = {names[i], c->p[i], c->page[i], c->pages, bytes, 1};
    TRY(harp::check(c->m[i]));
    if (c->m[i].at() % 16 || c->page[i] % 16)
      return fail(HARP_ERR_INVALID_ARG, "%s and the distance of its pages must be multiples of 16 bytes", names[i]);
  }
  TRY(check_vec("starts", c->starts, c->sequences + 1, 4, &c->plan[0]));
  TRY(check_vec("lengths", c->lengths, c->sequences, 4, &c->plan[1]));
  c->plan[2] = {"table", c->table, c->sequences == 1 ? c->width : c->ld_table, c->sequences, c->width, 4};
  return harp::check(c->plan[2]);
}
Cache4 cache_of(const CacheArg& c) {
  Cache4 r{};
  r.k = {const_cast<uint8_t*>(c.p[0]), const_cast<uint8_t*>(c.p[1]), c.page[0], c.page[1]};
  r.v = {const_cast<uint8_t*>(c.p[2]), const_cast<uint8_t*>(c.p[3]), c.page[2], c.page[3]};
  r.pages = (int)c.pages;
  r.heads = (int)c.heads;
  r.d = (int)c.d;
  while ((1 << r.page_log2) < c.page_size) ++r.page_log2;
  return r;
}
Plan4 plan_of(const CacheArg& c) {
  return {c.starts, c.lengths, c.table, c.ld_table, (int)c.sequences, (int)c.width};
}

}  // namespace

extern "C" {

harp_status harp_qk_norm_rope(const void* q, int64_t q_token, int64_t q_head, int64_t q_heads, const void* k,
                              int64_t k_token, int64_t k_head, int64_t k_heads, int64_t tokens, int64_t d,
                              harp_dtype io_dtype, const void* positions, int32_t wide_positions,
                              const double* freqs, int64_t pairs, int32_t interleaved, const void* gamma_q,
                              const void* gamma_k, float eps, const int8_t* signs, void* q_out, int64_t qo_token,
                              int64_t qo_head, void* k_out, int64_t ko_token, int64_t ko_head, hipStream_t stream) {
  QkIn a{{"q", q, q_token, q_head, q_heads, {}}, {"k", k, k_token, k_head, k_heads, {}}, tokens, d, io_dtype, positions,
         wide_positions, freqs, pairs, gamma_q, gamma_k, eps, signs, {}, 0};
  TRY(check_sizes(&a));
  if (tokens == 0) return HARP_OK;
  TRY(check_inputs(&a));
  HeadsArg oq{"q_out", q_out, qo_token, qo_head, q_heads, {}}, ok{"k_out", k_out, ko_token, ko_head, k_heads, {}};
  const int eb = size_of(io_dtype);
  HeadsArg* outs[2] = {&oq, &ok};
  const HeadsArg* ins[2] = {&a.q, &a.k};
  const int sides = a.has_k() ? 2 : 1;
  for (int i = 0; i < sides; ++i) {
    TRY(check(outs[i], tokens, d, eb));
    for (int j = 0; j < sides; ++j) TRY(apart(*outs[i], *ins[j], i == j, tokens));
    for (int j = 0; j < a.n_small; ++j) TRY(check_apart(outs[i]->m, a.small[j], false));
  }
  if (sides == 2) TRY(apart(ok, oq, false, tokens));
  QkArgs g = args_of(a, interleaved != 0);
  g.yq = heads_of(oq);
  g.yk = heads_of(ok);
  return launched(launch_qk_norm_rope(g, dt(io_dtype), stream), "harp_qk_norm_rope");
}

int64_t harp_qk_norm_rope_vjp_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t d) {
  if (tokens < 0 || tokens > kMaxSize || q_heads < 1 || q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads ||
      d < 8 || d > 512 || d % 8)
    return -1;
  return qk_norm_rope_vjp_workspace(tokens, q_heads + k_heads, d);
}

harp_status harp_qk_norm_rope_vjp(const void* q, int64_t q_token, int64_t q_head, int64_t q_heads, const void* k,
                                  int64_t k_token, int64_t k_head, int64_t k_heads, int64_t tokens, int64_t d,
                                  harp_dtype io_dtype, const void* positions, int32_t wide_positions,
                                  const double* freqs, int64_t pairs, int32_t interleaved, const void* gamma_q,
                                  const void* gamma_k, float eps, const int8_t* signs, const void* dyq,
                                  int64_t dyq_token, int64_t dyq_head, const void* dyk, int64_t dyk_token,
                                  int64_t dyk_head, void* dq, int64_t dq_token, int64_t dq_head, void* dk,
                                  int64_t dk_token, int64_t dk_head, float* dgamma_q, float* dgamma_k,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  QkIn a{{"q", q, q_token, q_head, q_heads, {}}, {"k", k, k_token, k_head, k_heads, {}}, tokens, d, io_dtype, positions,
         wide_positions, freqs, pairs, gamma_q, gamma_k, eps, signs, {}, 0};
  TRY(check_sizes(&a));
  if (k_heads == 0 && dgamma_k) return fail(HARP_ERR_INVALID_ARG, "dgamma_k goes with k_heads > 0 only");
  Mat mg[2] = {{"dgamma_q", nullptr, d, 1, d, 4}, {"dgamma_k", nullptr, d, 1, d, 4}};
  if (dgamma_q) TRY(check_vec("dgamma_q", dgamma_q, d, 4, &mg[0]));
  if (dgamma_k) TRY(check_vec("dgamma_k", dgamma_k, d, 4, &mg[1]));
  TRY(check_apart(mg[1], mg[0], false));
  const bool sums = dgamma_q || dgamma_k;
  if (tokens == 0 && !sums) return HARP_OK;
  QkArgs g = args_of(a, interleaved != 0);
  g.dgamma_q = dgamma_q;
  g.dgamma_k = dgamma_k;
  if (tokens > 0) {
    TRY(check_inputs(&a));
    const int eb = size_of(io_dtype), sides = a.has_k() ? 2 : 1;
    HeadsArg gy[2] = {{"dyq", dyq, dyq_token, dyq_head, q_heads, {}}, {"dyk", dyk, dyk_token, dyk_head, k_heads, {}}};
    HeadsArg gx[2] = {{"dq", dq, dq_token, dq_head, q_heads, {}}, {"dk", dk, dk_token, dk_head, k_heads, {}}};
    const HeadsArg* ins[2] = {&a.q, &a.k};
    for (int i = 0; i < sides; ++i) TRY(check(&gy[i], tokens, d, eb));
    const int64_t need = sums ? qk_norm_rope_vjp_workspace(tokens, q_heads + k_heads, d) : 0;
    TRY(check_workspace(need, workspace, workspace_bytes, 4));
    const Mat mw{"workspace", need > 0 ? workspace : nullptr, need / 4, 1, need / 4, 4};
    for (int i = 0; i < 2; ++i) TRY(check_apart(mw, mg[i], false));
    for (int i = 0; i < sides; ++i) {
      TRY(check(&gx[i], tokens, d, eb));
      for (int j = 0; j < sides; ++j) {
        TRY(apart(gx[i], gy[j], i == j, tokens));
        TRY(apart(gx[i], *ins[j], i == j, tokens));
      }
      for (const Mat& o : {mg[0], mg[1], mw}) {
        TRY(check_apart(o, gx[i].m, false));
        TRY(check_apart(o, gy[i].m, false));
        TRY(check_apart(o, ins[i]->m, false));
      }
      for (int j = 0; j < a.n_small; ++j) TRY(check_apart(gx[i].m, a.small[j], false));
    }
    for (const Mat& o : {mg[0], mg[1], mw})
      for (int j = 0; j < a.n_small; ++j) TRY(check_apart(o, a.small[j], false));
    if (sides == 2) TRY(apart(gx[1], gx[0], false, tokens));
    g.yq = heads_of(gy[0]);
    g.yk = heads_of(gy[1]);
    g.dq = heads_of(gx[0]);
    g.dk = heads_of(gx[1]);
    g.partial = need > 0 ? static_cast<float*>(workspace) : nullptr;
  }
  return launched(launch_qk_norm_rope_vjp(g, dt(io_dtype), stream), "harp_qk_norm_rope_vjp");
}

harp_status harp_kv4_write(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                           int64_t v_head, int64_t tokens, harp_dtype io_dtype, uint8_t* k_codes, int64_t kc_page,
                           uint8_t* k_scales, int64_t ks_page, uint8_t* v_codes, int64_t vc_page, uint8_t* v_scales,
                           int64_t vs_page, int64_t pages, int64_t kv_heads, int64_t page_size, int64_t d,
                           const int32_t* starts, const int32_t* lengths, const int32_t* table, int64_t ld_table,
                           int64_t sequences, int64_t width, hipStream_t stream) {
  CacheArg c{{k_codes, k_scales, v_codes, v_scales}, {kc_page, ks_page, vc_page, vs_page}, pages, kv_heads, page_size, d,
             starts, lengths, table, ld_table, sequences, width, {}, {}};
  if (!io_ok(io_dtype)) return fail(HARP_ERR_UNSUPPORTED, "io_dtype must be HARP_F32 or HARP_BF16");
  TRY(check_sizes(c));
  TRY(check_size("tokens", tokens, 0, kMaxSize));
  if (tokens == 0 || sequences == 0) return HARP_OK;
  HeadsArg x[2] = {{"k", k, k_token, k_head, kv_heads, {}}, {"v", v, v_token, v_head, kv_heads, {}}};
  for (HeadsArg& a : x) TRY(check(&a, tokens, d, size_of(io_dtype)));
  TRY(check(&c));
  for (int i = 0; i < 4; ++i) {
    for (const HeadsArg& a : x) TRY(check_apart(c.m[i], a.m, false));
    for (const Mat& p : c.plan) TRY(check_apart(c.m[i], p, false));
    for (int j = 0; j < i; ++j) TRY(check_apart(c.m[i], c.m[j], false));
  }
  return launched(launch_kv4_write(cache_of(c), plan_of(c), heads_of(x[0]), heads_of(x[1]), (int)tokens, dt(io_dtype),
                                   stream),
                  "harp_kv4_write");
}

harp_status harp_kv4_read(const uint8_t* k_codes, int64_t kc_page, const uint8_t* k_scales, int64_t ks_page,
                          const uint8_t* v_codes, int64_t vc_page, const uint8_t* v_scales, int64_t vs_page,
                          int64_t pages, int64_t kv_heads, int64_t page_size, int64_t d, const int32_t* starts,
                          const int32_t* lengths, const int32_t* table, int64_t ld_table, int64_t sequences,
                          int64_t width, void* k, int64_t k_token, int64_t k_head, void* v, int64_t v_token,
                          int64_t v_head, int64_t tokens, harp_dtype io_dtype, hipStream_t stream) {
  CacheArg c{{k_codes, k_scales, v_codes, v_scales}, {kc_page, ks_page, vc_page, vs_page}, pages, kv_heads, page_size, d,
             starts, lengths, table, ld_table, sequences, width, {}, {}};
  if (!io_ok(io_dtype)) return fail(HARP_ERR_UNSUPPORTED, "io_dtype must be HARP_F32 or HARP_BF16");
  TRY(check_sizes(c));
  TRY(check_size("tokens", tokens, 0, kMaxSize));
  if (tokens == 0 || sequences == 0) return HARP_OK;
  TRY(check(&c));
  HeadsArg x[2] = {{"k", k, k_token, k_head, kv_heads, {}}, {"v", v, v_token, v_head, kv_heads, {}}};
  for (HeadsArg& a : x) {
    TRY(check(&a, tokens, d, size_of(io_dtype)));
    for (const Mat& m : c.m) TRY(check_apart(a.m, m, false));
    for (const Mat& m : c.plan) TRY(check_apart(a.m, m, false));
  }
  TRY(check_apart(x[1].m, x[0].m, false));
  return launched(launch_kv4_read(cache_of(c), plan_of(c), heads_of(x[0]), heads_of(x[1]), (int)tokens, dt(io_dtype),
                                  stream),
                  "harp_kv4_read");
}

int64_t harp_kv4_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size,
                                     int64_t sequences, int64_t width) {
  if (tokens < 0 || tokens > kMaxSize || kv_heads < 1 || q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads ||
      d < kBlk4 || d > 256 || d % kBlk4 || page_size < 16 || page_size > 1 << 20 || !is_pow2(page_size) ||
      sequences < 0 || sequences > kMaxPlan || width < 1 || width > kMaxPlan)
    return -1;
  if (tokens * q_heads > kMaxSize || sequences * kv_heads > kMaxSize) return -1;
  return kv4_attention_workspace(tokens, q_heads, kv_heads, d, page_size, sequences, width);
}

harp_status harp_kv4_attention(const void* q, int64_t q_token, int64_t q_head, int64_t tokens, int64_t q_heads,
                               const uint8_t* k_codes, int64_t kc_page, const uint8_t* k_scales, int64_t ks_page,
                               const uint8_t* v_codes, int64_t vc_page, const uint8_t* v_scales, int64_t vs_page,
                               int64_t pages, int64_t kv_heads, int64_t page_size, int64_t d, const int32_t* starts,
                               const int32_t* lengths, const int32_t* table, int64_t ld_table, int64_t sequences,
                               int64_t width, float scale, int32_t causal, int64_t window, void* out,
                               int64_t out_token, int64_t out_head, float* lse, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  CacheArg c{{k_codes, k_scales, v_codes, v_scales}, {kc_page, ks_page, vc_page, vs_page}, pages, kv_heads, page_size, d,
             starts, lengths, table, ld_table, sequences, width, {}, {}};
  TRY(check_sizes(c));
  TRY(check_size("tokens", tokens, 0, kMaxSize));
  TRY(check_size("q_heads", q_heads, 1, kMaxHeads));
  if (q_heads % kv_heads)
    return fail(HARP_ERR_INVALID_ARG, "q_heads = %lld is not a multiple of kv_heads = %lld", (long long)q_heads,
                (long long)kv_heads);
  TRY(check_size("tokens x q_heads", tokens * q_heads, 0, kMaxSize));
  if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(HARP_ERR_INVALID_ARG, "scale must be positive and finite");
  TRY(check_size("window", window, 0, INT32_MAX));
  if (tokens == 0 || sequences == 0) return HARP_OK;
  HeadsArg mq{"q", q, q_token, q_head, q_heads, {}}, mo{"out", out, out_token, out_head, q_heads, {}};
  TRY(check(&mq, tokens, d, 2));
  TRY(check(&c));
  TRY(check(&mo, tokens, d, 2));
  Mat ml{"lse", nullptr, 1, 1, 1, 4};
  if (lse) TRY(check_vec("lse", lse, tokens * q_heads, 4, &ml));
  const int64_t need = kv4_attention_workspace(tokens, q_heads, kv_heads, d, page_size, sequences, width);
  TRY(check_workspace(need, workspace, workspace_bytes, 16));
  const Mat mw{"workspace", need > 0 ? workspace : nullptr, need / 4, 1, need / 4, 4};
  for (const Mat& o : {mo.m, ml, mw}) {
    TRY(check_apart(o, mq.m, false));
    for (const Mat& m : c.m) TRY(check_apart(o, m, false));
    for (const Mat& m : c.plan) TRY(check_apart(o, m, false));
  }
  TRY(check_apart(ml, mo.m, false));
  TRY(check_apart(mw, mo.m, false));
  TRY(check_apart(mw, ml, false));
  Attn4Args a{};
  a.cache = cache_of(c);
  a.plan = plan_of(c);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.partial = need > 0 ? static_cast<float*>(workspace) : nullptr;
  a.q_token = q_token;
  a.q_head = q_head;
  a.out_token = out_token;
  a.out_head = out_head;
  a.tokens = (int)tokens;
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / kv_heads);
  a.scale = scale;
  a.causal = causal != 0;
  a.window = (int)window;
  return launched(launch_kv4_attention(a, stream), "harp_kv4_attention");
}

}  // extern "C"
