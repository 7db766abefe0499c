"""Host-side tests of the 8-bit operators (no GPU needed): the oracle against
other routes, the C ABI's refusals before any HIP call, and the checks of the
Python binding before the library is reached.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from structured_rotations_amd import _lib, q8

F32, BF16, I8, F64, E8 = _lib.HARP_F32, _lib.HARP_BF16, _lib.HARP_I8, _lib.HARP_F64, _lib.HARP_E8M0
OK, BAD, UNSUP = _lib.HARP_OK, _lib.HARP_ERR_INVALID_ARG, _lib.HARP_ERR_UNSUPPORTED


# ------------------------------------------------------------------ oracle
def test_e4m3_table_against_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(Q.E4M3, t.astype(np.float64), equal_nan=True)
    assert Q.E4M3[0x7e] == 448 and Q.E4M3[1] == 2.0 ** -9


def test_encode_against_torch():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.01,
                        (Q.E4M3[:126] + Q.E4M3[1:127]) / 2, -(Q.E4M3[:126] + Q.E4M3[1:127]) / 2]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.encode(v), want)


def test_scales_by_hand():
    x = np.zeros((2, 130), dtype=np.float32)
    x[0, 3], x[0, 129], x[1, 0] = -7.0, 448.0, 500.0
    c, s = Q.quantize(x, 1, "f32")
    assert s.shape == (2, 2) and s[0, 0] == np.float32(7 / 448) and s[0, 1] == 1 and s[1, 1] == np.float32(2.0 ** -120)
    assert Q.decode(c)[0, 3] == -448 and Q.decode(c)[0, 129] == 448
    c, s = Q.quantize(x, 1, "e8m0")
    assert s[0, 0] == 2.0 ** -6 and s[0, 1] == 1 and s[1, 0] == 2 and s[1, 1] == 2.0 ** -120
    c, s = Q.quantize(x, 128, "f32")
    assert s.shape == (1, 2) and s[0, 0] == np.float32(500 / 448)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    h, g = rng.standard_normal((3, 7)), rng.standard_normal(7)
    dn, dr = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    _, _, r, xn = Q.rmsnorm(h, None, g, 0.1)
    dh, dg = Q.rmsnorm_vjp(xn, r, dn, g, dr)

    def loss(hh, gg):
        return np.sum(Q.rmsnorm(hh, None, gg, 0.1)[0] * dn) + np.sum(hh * dr)

    e = 1e-6
    for idx in np.ndindex(3, 7):
        d = np.zeros((3, 7))
        d[idx] = e
        assert abs((loss(h + d, g) - loss(h - d, g)) / (2 * e) - dh[idx]) < 1e-7
    for j in range(7):
        d = np.zeros(7)
        d[j] = e
        assert abs((loss(h, g + d) - loss(h, g - d)) / (2 * e) - dg[j]) < 1e-7


def test_products_against_single_elements_and_differences():
    rng = np.random.default_rng(2)
    ac, as_ = Q.quantize(rng.standard_normal((3, 200)), 1)
    wc, ws = Q.quantize(rng.standard_normal((130, 200)), 128)
    y = Q.matmul(ac, as_, wc, ws)
    one = sum(float(Q.E4M3[ac[2, k]]) * float(as_[2, k // 128]) * float(Q.E4M3[wc[129, k]]) * float(ws[1, k // 128])
              for k in range(200))
    assert abs(y[2, 129] - one) < 1e-9
    dy, w = rng.standard_normal((3, 4)), rng.standard_normal((4, 200))
    x = Q.dequantize(ac, as_)
    dw = Q.wgrad(dy, ac, as_)
    for j, k in ((0, 0), (3, 199), (2, 128)):
        d = np.zeros_like(w)
        d[j, k] = 1.0
        assert abs(np.sum(dy * (x @ (w + d).T)) - np.sum(dy * (x @ w.T)) - dw[j, k]) < 1e-9


# --------------------------------------------------------------------- ABI
@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def P(v):
    return ctypes.c_void_p(v)


X, Y, Z, V, W, U = (P(0x1000000 * (i + 1)) for i in range(6))     # never dereferenced


def quantize(lib, x=X, ldx=256, xdt=F32, rows=4, cols=256, br=1, codes=Y, ldc=256, scales=Z, sdt=F32):
    return lib.harp_quantize_q8(x, ldx, xdt, rows, cols, br, codes, ldc, scales, sdt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xdt=I8), UNSUP), (dict(xdt=E8), UNSUP), (dict(sdt=BF16), UNSUP), (dict(br=64), UNSUP), (dict(br=0), UNSUP),
    (dict(rows=-1), BAD), (dict(rows=(1 << 30) + 1), BAD), (dict(cols=0), BAD), (dict(ldx=255), BAD),
    (dict(ldc=255), BAD), (dict(x=None), BAD), (dict(codes=None), BAD), (dict(scales=None), BAD),
    (dict(x=P(0x1000002)), BAD), (dict(scales=P(0x3000001)), BAD), (dict(codes=X), BAD), (dict(scales=Y), BAD),
    (dict(codes=P(0x1000000 + 100)), BAD), (dict(ldx=1 << 61), BAD), (dict(ldc=1 << 62), BAD)])
def test_quantize_rejects_on_host(lib, kw, status):
    assert quantize(lib, **kw) == status
    assert lib.harp_last_error().decode()


def norm(lib, x=X, ldx=256, res=Y, ldr=256, gamma=None, eps=1e-6, h=None, ldh=256, codes=Z, ldc=256, scales=V,
         rstd=None, ck=None, ldk=256, cks=None, sdt=F32, rows=4, d=256, io=F32):
    return lib.harp_rmsnorm_q8(x, ldx, res, ldr, gamma, eps, h, ldh, codes, ldc, scales, rstd, ck, ldk, cks, sdt,
                               rows, d, io, None)


@pytest.mark.parametrize("kw,status", [
    (dict(io=F64), UNSUP), (dict(sdt=I8), UNSUP), (dict(rows=-1), BAD), (dict(d=0), BAD), (dict(d=32769, ldx=40000), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(x=None), BAD), (dict(codes=None), BAD),
    (dict(scales=None), BAD), (dict(ldx=255), BAD), (dict(ldr=255), BAD), (dict(ldc=10), BAD),
    (dict(h=W, res=None), BAD), (dict(h=W, ldh=3), BAD), (dict(ck=W), BAD), (dict(ck=W, cks=U), BAD),
    (dict(gamma=U, cks=W), BAD), (dict(h=P(0x1000000 + 1024)), BAD), (dict(h=X, ldh=512, ldx=256), BAD),
    (dict(codes=X), BAD), (dict(gamma=P(0x5000002)), BAD), (dict(rstd=Z), BAD),
    (dict(gamma=U, h=U), BAD)])
def test_rmsnorm_rejects_on_host(lib, kw, status):
    assert norm(lib, **kw) == status
    assert lib.harp_last_error().decode()


def norm_vjp(lib, codes=X, ldc=256, scales=Y, sdt=F32, rstd=Z, gamma=None, dn=V, lddn=256, dres=None, lddres=256, dh=W,
             lddh=256, dgamma=None, rows=4, d=256, io=F32, ws=U, wsb=1 << 20):
    return lib.harp_rmsnorm_q8_vjp(codes, ldc, scales, sdt, rstd, gamma, dn, lddn, dres, lddres, dh, lddh, dgamma, rows,
                                   d, io, ws, wsb, None)


DG = P(0x10000000)


@pytest.mark.parametrize("kw,status", [
    (dict(io=I8), UNSUP), (dict(sdt=BF16), UNSUP), (dict(rows=-1), BAD), (dict(d=0), BAD), (dict(d=32769), BAD),
    (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(rstd=None), BAD), (dict(dn=None), BAD),
    (dict(dh=None), BAD), (dict(lddn=1), BAD), (dict(lddh=1), BAD), (dict(dres=U, lddres=1), BAD),
    (dict(dgamma=DG, ws=None), BAD), (dict(dgamma=DG, wsb=4 * 256 * 4 - 1), BAD), (dict(dgamma=DG, ws=P(0x6000002)), BAD),
    (dict(dgamma=W), BAD), (dict(dgamma=DG, ws=V), BAD), (dict(dh=X), BAD), (dict(dh=V, lddh=512), BAD),
    (dict(dh=P(0x4000000 + 4)), BAD)])
def test_rmsnorm_vjp_rejects_on_host(lib, kw, status):
    assert norm_vjp(lib, **kw) == status
    assert lib.harp_last_error().decode()


def matmul(lib, a=X, lda=256, sa=Y, w=Z, ldw=256, sw=V, sdt=F32, rows=200, n=300, k=256, y=W, ldy=300, ydt=F32, ws=DG,
           wsb=1 << 30):
    return lib.harp_matmul_q8(a, lda, sa, w, ldw, sw, sdt, rows, n, k, y, ldy, ydt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ydt=I8), UNSUP), (dict(ydt=E8), UNSUP), (dict(sdt=BF16), UNSUP), (dict(rows=-1), BAD), (dict(n=0), BAD),
    (dict(k=0), BAD), (dict(k=(1 << 30) + 1), BAD), (dict(a=None), BAD), (dict(w=None), BAD), (dict(sa=None), BAD),
    (dict(sw=None), BAD), (dict(y=None), BAD), (dict(lda=255), BAD), (dict(ldw=255), BAD), (dict(ldy=299), BAD),
    (dict(sa=P(0x2000002)), BAD), (dict(y=P(0x5000002)), BAD), (dict(y=X), BAD), (dict(y=V), BAD)])
def test_matmul_rejects_on_host(lib, kw, status):
    assert matmul(lib, **kw) == status
    assert lib.harp_last_error().decode()


def wgrad(lib, dy=X, lddy=300, x=Y, ldx=256, sx=Z, sdt=F32, rows=4000, n=300, k=256, dw=V, lddw=256, wdt=F32, ws=DG,
          wsb=1 << 30):
    return lib.harp_matmul_q8_wgrad(dy, lddy, x, ldx, sx, sdt, rows, n, k, dw, lddw, wdt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(wdt=I8), UNSUP), (dict(sdt=F64), UNSUP), (dict(rows=-1), BAD), (dict(n=0), BAD), (dict(k=0), BAD),
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(sx=None), BAD), (dict(dw=None), BAD), (dict(lddy=1), BAD),
    (dict(ldx=1), BAD), (dict(lddw=1), BAD), (dict(dw=X), BAD), (dict(dy=P(0x1000001)), BAD)])
def test_wgrad_rejects_on_host(lib, kw, status):
    assert wgrad(lib, **kw) == status
    assert lib.harp_last_error().decode()


# x and residual side by side in rows of 4000 bytes, 1024 bytes each; h may lie in the 1952 bytes behind them, or be
# the residual
@pytest.mark.parametrize("at,free", [(2048, True), (2500, True), (2976, True), (4000 + 2048, True), (-4000 + 2976, True),
                                     (1024, True), (2980, False), (2044, False), (512, False), (4000, False),
                                     (8000 + 512, False), (-4, False)])
def test_rows_side_by_side(lib, at, free):
    # rstd over scales is refused last: the message says whether h was let through
    base = 0x1000000
    kw = dict(x=P(base), ldx=1000, res=P(base + 1024), ldr=1000, h=P(base + at), rstd=V)
    assert norm(lib, ldh=1000, **kw) == BAD
    assert lib.harp_last_error().decode().startswith("rstd overlaps" if free else "h_out overlaps")
    assert norm(lib, ldh=999, **kw) == BAD                        # other distances: apart as a whole only
    assert lib.harp_last_error().decode().startswith("h_out overlaps")


def test_a_single_row_beside_others(lib):
    # gamma (1024 bytes) within the rows' 4000 bytes, codes (256 of 4000) over it or not
    base = 0x1000000
    for at, free in ((0, True), (1024, False), (1024 + 2976, True), (800, False), (745, False), (744, True)):
        assert norm(lib, x=Y, gamma=P(base + 1000), res=None, codes=P(base + at), ldc=4000, rstd=V) == BAD
        got = lib.harp_last_error().decode()
        assert got.startswith("rstd overlaps" if free else "codes overlaps gamma"), (at, got)


def test_products_reject_short_workspaces(lib):
    for call, size in ((matmul, lambda: lib.harp_matmul_q8_workspace(200, 300, 4096)),
                       (wgrad, lambda: lib.harp_matmul_q8_wgrad_workspace(4000, 300, 256))):
        need = size()
        kw = dict(k=4096, lda=4096, ldw=4096) if call is matmul else {}
        if need > 0:
            assert call(lib, ws=None, **kw) == BAD
            assert call(lib, wsb=need - 1, **kw) == BAD
            assert call(lib, ws=P(0x10000004), **kw) == BAD
            assert "workspace" in lib.harp_last_error().decode()


def test_sizes_out_of_range(lib):
    for fn in (lib.harp_matmul_q8_workspace, lib.harp_matmul_q8_wgrad_workspace):
        assert fn(-1, 1, 1) == -1 and fn(1, 0, 1) == -1 and fn(1, 1, 0) == -1 and fn(1, 1, 1 << 31) == -1
        assert fn(1 << 30, 1 << 30, 1 << 30) >= 0
    assert lib.harp_rmsnorm_q8_vjp_workspace(-1, 5) == -1 and lib.harp_rmsnorm_q8_vjp_workspace(1, 32769) == -1
    assert lib.harp_rmsnorm_q8_vjp_workspace(1 << 30, 32768) > 0


def test_no_rows_is_a_noop(lib):
    assert quantize(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert norm(lib, rows=0, x=None, res=None, codes=None, scales=None) == OK
    assert norm_vjp(lib, rows=0, codes=None, scales=None, rstd=None, dn=None, dh=None) == OK
    assert matmul(lib, rows=0, a=None, w=None, sa=None, sw=None, y=None) == OK


# ----------------------------------------------------------------- binding
class _Guard:
    """The real library's size helpers; any launching entry point fails the test."""

    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return getattr(self._real, name)

        def reached(*a, **k):
            raise AssertionError(f"{name} reached the library")
        return reached


@pytest.fixture
def guard(monkeypatch):
    real = q8.lib()
    monkeypatch.setattr(q8, "lib", lambda: _Guard(real))


E4 = torch.float8_e4m3fn
E8T = torch.float8_e8m0fnu


def c(rows, cols):
    return torch.zeros(rows, cols, dtype=torch.uint8).view(E4)


def s(rows, cols, dtype=torch.float32):
    return torch.ones(rows, cols).to(dtype)


def gpu_only(fn):
    with pytest.raises(TypeError, match="GPU tensor"):
        fn()


def refuses(exc, match, fn):
    with pytest.raises(exc, match=match):
        fn()


def test_quantize_checks(guard):
    x = torch.zeros(3, 200)
    gpu_only(lambda: q8.harp_quantize_q8(x))
    gpu_only(lambda: q8.harp_quantize_q8(x, 128, "e8m0", c(3, 200), s(1, 2, E8T)))
    refuses(TypeError, "x must be", lambda: q8.harp_quantize_q8(x.double()))
    refuses(TypeError, "tensor", lambda: q8.harp_quantize_q8([1.0]))
    refuses(ValueError, "2-D", lambda: q8.harp_quantize_q8(x[0]))
    refuses(ValueError, "contiguous", lambda: q8.harp_quantize_q8(torch.zeros(200, 3).t()))
    refuses(ValueError, "row stride", lambda: q8.harp_quantize_q8(torch.zeros(1, 200).expand(3, 200)))
    refuses(ValueError, "block_rows", lambda: q8.harp_quantize_q8(x, 64))
    refuses(ValueError, "scale_dtype", lambda: q8.harp_quantize_q8(x, 1, "bf16"))
    refuses(ValueError, "codes must be", lambda: q8.harp_quantize_q8(x, codes=c(2, 200)))
    refuses(TypeError, "codes must be", lambda: q8.harp_quantize_q8(x, codes=torch.zeros(3, 200, dtype=torch.uint8)))
    refuses(ValueError, "scales must be", lambda: q8.harp_quantize_q8(x, scales=s(3, 1)))
    refuses(TypeError, "scales must be", lambda: q8.harp_quantize_q8(x, scales=s(3, 2, E8T)))
    refuses(ValueError, "contiguous", lambda: q8.harp_quantize_q8(x, scales=torch.ones(2, 3).t()))


def test_rmsnorm_checks(guard):
    x = torch.zeros(3, 200, dtype=torch.bfloat16)
    g = torch.ones(200, dtype=torch.bfloat16)
    gpu_only(lambda: q8.harp_rmsnorm_q8(x))
    gpu_only(lambda: q8.harp_rmsnorm_q8(x, x, g, checkpoint=True))
    refuses(TypeError, "residual", lambda: q8.harp_rmsnorm_q8(x, x.float()))
    refuses(ValueError, "residual", lambda: q8.harp_rmsnorm_q8(x, x[:2]))
    refuses(TypeError, "gamma", lambda: q8.harp_rmsnorm_q8(x, None, g.float()))
    refuses(ValueError, "gamma", lambda: q8.harp_rmsnorm_q8(x, None, g[:-1]))
    refuses(ValueError, "residual only", lambda: q8.harp_rmsnorm_q8(x, h=x))
    refuses(ValueError, "h must be", lambda: q8.harp_rmsnorm_q8(x, x, h=x[:2]))
    refuses(ValueError, "checkpoint", lambda: q8.harp_rmsnorm_q8(x, rstd=torch.zeros(3)))
    refuses(ValueError, "ckpt", lambda: q8.harp_rmsnorm_q8(x, checkpoint=True, ckpt_codes=c(3, 200)))
    refuses(ValueError, "rstd", lambda: q8.harp_rmsnorm_q8(x, checkpoint=True, rstd=torch.zeros(2)))
    refuses(ValueError, "scales", lambda: q8.harp_rmsnorm_q8(x, scales=s(3, 3)))


def test_rmsnorm_vjp_checks(guard):
    dn, g, r = torch.zeros(3, 200), torch.ones(200), torch.ones(3)

    def call(codes=c(3, 200), scales=s(3, 2), rstd=r, dn=dn, **kw):
        return q8.harp_rmsnorm_q8_vjp(codes, scales, rstd, dn, **kw)

    gpu_only(call)
    gpu_only(lambda: call(gamma=g, dres=dn, dgamma=torch.zeros(200)))
    refuses(ValueError, "ckpt_codes", lambda: call(codes=c(2, 200)))
    refuses(ValueError, "ckpt_scales", lambda: call(scales=s(3, 1)))
    refuses(ValueError, "rstd", lambda: call(rstd=r[:2]))
    refuses(TypeError, "gamma", lambda: call(gamma=g.to(torch.bfloat16)))
    refuses(ValueError, "dres", lambda: call(dres=dn[:, :100]))
    refuses(TypeError, "dh", lambda: call(dh=dn.to(torch.bfloat16)))
    refuses(ValueError, "dgamma", lambda: call(dgamma=torch.zeros(199)))
    refuses(ValueError, "want_dgamma", lambda: call(want_dgamma=False, dgamma=torch.zeros(200)))
    refuses(TypeError, "dn must be", lambda: call(dn=dn.half()))


def test_matmul_checks(guard):
    def call(a=c(3, 200), sa=s(3, 2), w=c(300, 200), sw=s(3, 2), **kw):
        return q8.harp_matmul_q8(a, sa, w, sw, **kw)

    gpu_only(call)
    gpu_only(lambda: call(sa=s(3, 2, E8T), sw=s(3, 2, E8T), out="f32", y=torch.zeros(3, 300)))
    refuses(TypeError, "a_codes", lambda: call(a=torch.zeros(3, 200)))
    refuses(ValueError, "w_codes", lambda: call(w=c(300, 199)))
    refuses(ValueError, "a_scales", lambda: call(sa=s(3, 1)))
    refuses(ValueError, "w_scales", lambda: call(sw=s(300, 2)))
    refuses(TypeError, "w_scales", lambda: call(sw=s(3, 2, E8T)))
    refuses(ValueError, "out must be", lambda: call(out="f16"))
    refuses(TypeError, "y must be", lambda: call(y=torch.zeros(3, 300)))
    refuses(ValueError, "y must be", lambda: call(y=torch.zeros(3, 299, dtype=torch.bfloat16)))
    refuses(ValueError, "no rows", lambda: call(w=c(0, 200)))
    refuses(ValueError, "workspace", lambda: call(workspace=torch.zeros(8, 8).t()))


def test_wgrad_checks(guard):
    dy = torch.zeros(5, 64, dtype=torch.bfloat16)

    def call(dy=dy, x=c(5, 200), sx=s(5, 2), **kw):
        return q8.harp_matmul_q8_wgrad(dy, x, sx, **kw)

    gpu_only(call)
    refuses(TypeError, "dy must be", lambda: call(dy=dy.float()))
    refuses(ValueError, "x_codes", lambda: call(x=c(4, 200)))
    refuses(ValueError, "x_scales", lambda: call(sx=s(5, 3)))
    refuses(TypeError, "dw must be", lambda: call(dw=torch.zeros(64, 200, dtype=torch.bfloat16)))
    refuses(ValueError, "dw must be", lambda: call(dw=torch.zeros(200, 64)))
    refuses(ValueError, "out must be", lambda: call(out="i8"))
