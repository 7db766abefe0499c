// extern "C" entry points of the 8-bit path (include/harp.h): every argument
// is checked on the host, before any HIP call, then the launchers run.
#include <cstdint>

#include "args.h"
#include "harp.h"
#include "q8.h"

using namespace harp;

namespace {

bool scale_ok(harp_dtype t) { return t == HARP_F32 || t == HARP_E8M0; }

Mat scale_mat(const char* name, const void* p, harp_dtype t, int64_t brows, int64_t cols) {
  const int64_t nb = harp::q_nblk(cols);
  return {name, p, nb, brows, nb, size_of(t)};
}

bool sizes_ok(int64_t rows, int64_t n, int64_t k) {
  return rows >= 0 && rows <= kMaxSize && n >= 1 && n <= kMaxSize && k >= 1 && k <= kMaxSize;
}

constexpr const char* kBadScale = "scale_dtype must be HARP_F32 or HARP_E8M0";

}  // namespace

extern "C" {

harp_status harp_quantize_q8(const void* x, int64_t ldx, harp_dtype x_dtype, int64_t rows, int64_t cols,
                             int32_t block_rows, uint8_t* codes, int64_t ldc, void* scales, harp_dtype scale_dtype,
                             hipStream_t stream) {
  if (!io_ok(x_dtype)) return fail(HARP_ERR_UNSUPPORTED, "x_dtype must be HARP_F32 or HARP_BF16");
  if (!scale_ok(scale_dtype)) return fail(HARP_ERR_UNSUPPORTED, kBadScale);
  if (block_rows != 1 && block_rows != harp::kQBlk)
    return fail(HARP_ERR_UNSUPPORTED, "block_rows must be 1 or %d", harp::kQBlk);
  TRY(check_size("rows", rows, 0, kMaxSize));
  TRY(check_size("cols", cols, 1, kMaxSize));
  if (rows == 0) return HARP_OK;
  const Mat mx{"x", x, ldx, rows, cols, size_of(x_dtype)}, mc{"codes", codes, ldc, rows, cols, 1};
  const Mat ms = scale_mat("scales", scales, scale_dtype, (rows + block_rows - 1) / block_rows, cols);
  for (const Mat* m : {&mx, &mc, &ms}) TRY(check(*m));
  TRY(check_apart(mc, mx, false));
  TRY(check_apart(ms, mx, false));
  TRY(check_apart(ms, mc, false));
  return launched(harp::launch_quantize_q8(x, ldx, dt(x_dtype), rows, (int)cols, block_rows != 1, codes, ldc, scales,
                                           scale_dtype == HARP_E8M0, stream),
                  "harp_quantize_q8");
}

harp_status harp_rmsnorm_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* gamma,
                            float eps, void* h_out, int64_t ldh, uint8_t* codes, int64_t ldc, void* scales,
                            float* rstd, uint8_t* ckpt_codes, int64_t ldk, void* ckpt_scales,
                            harp_dtype scale_dtype, int64_t rows, int64_t d, harp_dtype io_dtype,
                            hipStream_t stream) {
  if (!io_ok(io_dtype)) return fail(HARP_ERR_UNSUPPORTED, "io_dtype must be HARP_F32 or HARP_BF16");
  if (!scale_ok(scale_dtype)) return fail(HARP_ERR_UNSUPPORTED, kBadScale);
  TRY(check_size("rows", rows, 0, kMaxSize));
  TRY(check_size("d", d, 1, HARP_MAX_D));
  if (!(eps >= 0.0f)) return fail(HARP_ERR_INVALID_ARG, "eps must be at least 0");
  if (h_out != nullptr && residual == nullptr) return fail(HARP_ERR_INVALID_ARG, "h_out goes with a residual only");
  if ((ckpt_codes != nullptr) != (ckpt_scales != nullptr))
    return fail(HARP_ERR_INVALID_ARG, "ckpt_codes and ckpt_scales go together");
  if (ckpt_codes != nullptr && gamma == nullptr)
    return fail(HARP_ERR_INVALID_ARG, "ckpt_codes go with gamma only (without it codes are the checkpoint)");
  if (rows == 0) return HARP_OK;
  const int eb = size_of(io_dtype);
  const Mat in[3] = {{"x", x, ldx, rows, d, eb}, {"residual", residual, ldr, rows, d, eb}, {"gamma", gamma, d, 1, d, eb}};
  const Mat out[6] = {{"h_out", h_out, ldh, rows, d, eb},
                      {"codes", codes, ldc, rows, d, 1},
                      scale_mat("scales", scales, scale_dtype, rows, d),
                      {"rstd", rstd, 1, rows, 1, 4},
                      {"ckpt_codes", ckpt_codes, ldk, rows, d, 1},
                      scale_mat("ckpt_scales", ckpt_scales, scale_dtype, rows, d)};
  for (int i = 0; i < 3; ++i)
    if (i == 0 || in[i].p) TRY(check(in[i]));
  for (int i = 0; i < 6; ++i)
    if (i == 1 || i == 2 || out[i].p) TRY(check(out[i]));
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 3; ++j) TRY(check_apart(out[i], in[j], i == 0 && j < 2));
    for (int j = 0; j < i; ++j) TRY(check_apart(out[i], out[j], false));
  }
  // h_out in place over one input still must not touch the other in part:
  // check_apart above rejects that (same base or no common byte).
  harp::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.h = h_out;
  a.codes = codes;
  a.ckpt = ckpt_codes;
  a.scales = scales;
  a.ckpt_scales = ckpt_scales;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldc = ldc;
  a.ldk = ldk;
  a.rows = rows;
  a.d = (int)d;
  a.eps = eps;
  return launched(harp::launch_rmsnorm_q8(a, dt(io_dtype), scale_dtype == HARP_E8M0, stream), "harp_rmsnorm_q8");
}

int64_t harp_rmsnorm_q8_vjp_workspace(int64_t rows, int64_t d) {
  if (rows < 0 || rows > kMaxSize || d < 1 || d > HARP_MAX_D) return -1;
  return harp::rmsnorm_q8_vjp_workspace(rows, d);
}

harp_status harp_rmsnorm_q8_vjp(const uint8_t* codes, int64_t ldc, const void* scales, harp_dtype scale_dtype,
                                const float* rstd, const void* gamma, const void* dn, int64_t lddn, const void* dres,
                                int64_t lddres, void* dh, int64_t lddh, float* dgamma, int64_t rows, int64_t d,
                                harp_dtype io_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!io_ok(io_dtype)) return fail(HARP_ERR_UNSUPPORTED, "io_dtype must be HARP_F32 or HARP_BF16");
  if (!scale_ok(scale_dtype)) return fail(HARP_ERR_UNSUPPORTED, kBadScale);
  TRY(check_size("rows", rows, 0, kMaxSize));
  TRY(check_size("d", d, 1, HARP_MAX_D));
  const int eb = size_of(io_dtype);
  const Mat mg{"dgamma", dgamma, d, 1, d, 4};
  if (dgamma) TRY(check(mg));
  if (rows == 0 && dgamma == nullptr) return HARP_OK;
  if (rows > 0) {
    const Mat in[6] = {{"codes", codes, ldc, rows, d, 1},   scale_mat("scales", scales, scale_dtype, rows, d),
                       {"rstd", rstd, 1, rows, 1, 4},       {"dn", dn, lddn, rows, d, eb},
                       {"dres", dres, lddres, rows, d, eb}, {"gamma", gamma, d, 1, d, eb}};
    const Mat mh{"dh", dh, lddh, rows, d, eb};
    for (int i = 0; i < 6; ++i)
      if (i < 4 || in[i].p) TRY(check(in[i]));
    TRY(check(mh));
    for (int i = 0; i < 6; ++i) {
      TRY(check_apart(mh, in[i], i == 3 || i == 4));
      TRY(check_apart(mg, in[i], false));
    }
    TRY(check_apart(mg, mh, false));
    if (dgamma) {
      const int64_t need = harp::rmsnorm_q8_vjp_workspace(rows, d);
      TRY(check_workspace(need, workspace, workspace_bytes, 4));
      const Mat mw{"workspace", workspace, need / 4, 1, need / 4, 4};
      for (int i = 0; i < 6; ++i) TRY(check_apart(mw, in[i], false));
      TRY(check_apart(mw, mh, false));
      TRY(check_apart(mw, mg, false));
    }
  }
  harp::NormVjpArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.gamma = gamma;
  a.dn = dn;
  a.dres = dres;
  a.rstd = rstd;
  a.dh = dh;
  a.dgamma = dgamma;
  a.partial = dgamma ? static_cast<float*>(workspace) : nullptr;
  a.ldc = ldc;
  a.lddn = lddn;
  a.lddres = lddres;
  a.lddh = lddh;
  a.rows = rows;
  a.d = (int)d;
  return launched(harp::launch_rmsnorm_q8_vjp(a, dt(io_dtype), scale_dtype == HARP_E8M0, stream),
                  "harp_rmsnorm_q8_vjp");
}

int64_t harp_matmul_q8_workspace(int64_t rows, int64_t n, int64_t k) {
  return sizes_ok(rows, n, k) ? harp::matmul_q8_workspace(rows, n, k) : -1;
}

harp_status harp_matmul_q8(const uint8_t* a, int64_t lda, const void* a_scales, const uint8_t* w, int64_t ldw,
                           const void* w_scales, harp_dtype scale_dtype, int64_t rows, int64_t n, int64_t k, void* y,
                           int64_t ldy, harp_dtype y_dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  if (!io_ok(y_dtype)) return fail(HARP_ERR_UNSUPPORTED, "y_dtype must be HARP_F32 or HARP_BF16");
  if (!scale_ok(scale_dtype)) return fail(HARP_ERR_UNSUPPORTED, kBadScale);
  TRY(check_size("rows", rows, 0, kMaxSize));
  TRY(check_size("n", n, 1, kMaxSize));
  TRY(check_size("k", k, 1, kMaxSize));
  if (rows == 0) return HARP_OK;
  const Mat in[4] = {{"a", a, lda, rows, k, 1},
                     scale_mat("a_scales", a_scales, scale_dtype, rows, k),
                     {"w", w, ldw, n, k, 1},
                     scale_mat("w_scales", w_scales, scale_dtype, harp::q_nblk(n), k)};
  const Mat my{"y", y, ldy, rows, n, size_of(y_dtype)};
  for (const Mat& m : in) TRY(check(m));
  TRY(check(my));
  for (const Mat& m : in) TRY(check_apart(my, m, false));
  const int64_t need = harp::matmul_q8_workspace(rows, n, k);
  TRY(check_workspace(need, workspace, workspace_bytes, 16));
  if (need > 0) {
    const Mat mw{"workspace", workspace, need / 4, 1, need / 4, 4};
    for (const Mat& m : in) TRY(check_apart(mw, m, false));
    TRY(check_apart(mw, my, false));
  }
  harp::MatmulArgs g{};
  g.a = a;
  g.w = w;
  g.a_scales = a_scales;
  g.w_scales = w_scales;
  g.y = y;
  g.partial = static_cast<float*>(workspace);
  g.lda = lda;
  g.ldw = ldw;
  g.ldy = ldy;
  g.rows = (int)rows;
  g.n = (int)n;
  g.k = (int)k;
  g.nkb = (int)harp::q_nblk(k);
  return launched(harp::launch_matmul_q8(g, scale_dtype == HARP_E8M0, dt(y_dtype), stream), "harp_matmul_q8");
}

int64_t harp_matmul_q8_wgrad_workspace(int64_t rows, int64_t n, int64_t k) {
  return sizes_ok(rows, n, k) ? harp::matmul_q8_wgrad_workspace(rows, n, k) : -1;
}

harp_status harp_matmul_q8_wgrad(const void* dy, int64_t lddy, const uint8_t* x, int64_t ldx, const void* x_scales,
                                 harp_dtype scale_dtype, int64_t rows, int64_t n, int64_t k, void* dw, int64_t lddw,
                                 harp_dtype dw_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!io_ok(dw_dtype)) return fail(HARP_ERR_UNSUPPORTED, "dw_dtype must be HARP_F32 or HARP_BF16");
  if (!scale_ok(scale_dtype)) return fail(HARP_ERR_UNSUPPORTED, kBadScale);
  TRY(check_size("rows", rows, 0, kMaxSize));
  TRY(check_size("n", n, 1, kMaxSize));
  TRY(check_size("k", k, 1, kMaxSize));
  const Mat md{"dw", dw, lddw, n, k, size_of(dw_dtype)};
  TRY(check(md));
  const int64_t need = harp::matmul_q8_wgrad_workspace(rows, n, k);
  TRY(check_workspace(need, workspace, workspace_bytes, 16));
  const Mat mw{"workspace", need > 0 ? workspace : nullptr, need / 4, 1, need / 4, 4};
  TRY(check_apart(mw, md, false));
  if (rows > 0) {
    const Mat in[3] = {{"dy", dy, lddy, rows, n, 2},
                       {"x", x, ldx, rows, k, 1},
                       scale_mat("x_scales", x_scales, scale_dtype, rows, k)};
    for (const Mat& m : in) {
      TRY(check(m));
      TRY(check_apart(md, m, false));
      TRY(check_apart(mw, m, false));
    }
  }
  harp::WgradArgs g{};
  g.dy = static_cast<const uint16_t*>(dy);
  g.x = x;
  g.x_scales = x_scales;
  g.dw = dw;
  g.partial = static_cast<float*>(workspace);
  g.lddy = lddy;
  g.ldx = ldx;
  g.lddw = lddw;
  g.rows = (int)rows;
  g.n = (int)n;
  g.k = (int)k;
  g.nkb = (int)harp::q_nblk(k);
  return launched(harp::launch_matmul_q8_wgrad(g, scale_dtype == HARP_E8M0, dt(dw_dtype), stream),
                  "harp_matmul_q8_wgrad");
}

}  // extern "C"
