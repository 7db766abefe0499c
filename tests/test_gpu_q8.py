"""The 8-bit operators against the fp64 oracle (oracle/q8_oracle.py).

Tolerances, fixed by the arithmetic:
  - coding: scales are one fp32 division and compared for equality.  A code is
    the rounding of an fp32 quotient, 2^-23 at most from the true one: it has
    to be the nearest one (ties to even) except for quotients nearer than that
    to the middle of two codes, but not on it;
  - norm: its values reach the coding with an fp32 error.  A row's sum of
    squares is added in a tree of at most 5 + 32 fp32 additions of positive
    terms, so it is off by at most 40 * 2^-24, and 1/rms and the products by
    less than that: 2^-18 relative bounds the whole.  A scale may be off by
    that much, a code must be a nearest one up to that much;
  - gradients and products: per row relative l2 error 1e-5 for fp32 results and
    4e-3 for bf16 ones (one rounding, 2^-8 at most per element), the bounds of
    the other transforms.
"""
import numpy as np
import pytest
import torch

import structured_rotations_amd as H
from oracle import q8_oracle as Q

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
SCALE = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}
TOL = {"f32": 1e-5, "bf16": 4e-3}
SLACK = 2.0 ** -18


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes_np(t):
    return t.view(torch.uint8).cpu().numpy()


def scales_np(t):
    if t.dtype == torch.float32:
        return t.cpu().numpy()
    return Q.e8m0(t.view(torch.uint8).cpu().numpy()).astype(np.float32)


def to_codes(c):
    return torch.from_numpy(np.ascontiguousarray(c)).cuda().view(torch.float8_e4m3fn)


def to_scales(s, kind):
    if kind == "f32":
        return torch.from_numpy(np.ascontiguousarray(s, dtype=np.float32)).cuda()
    b = np.where(np.isnan(s), 255, np.round(np.log2(np.where(np.isnan(s), 1.0, s))) + 127).astype(np.uint8)
    return torch.from_numpy(b).cuda().view(torch.float8_e8m0fnu)


def rel_rows(a, b):
    n = np.linalg.norm(b, axis=1)
    d = np.linalg.norm(a - b, axis=1)
    return float(np.max(np.where(n > 0, d / np.where(n > 0, n, 1.0), d))) if len(n) else 0.0


def padded(t, pad, offset=0):
    """The same rows in a wider buffer: row stride cols + pad, base moved by
    offset elements."""
    r, c = t.shape
    buf = torch.zeros(r * (c + pad) + offset + 64, dtype=t.dtype, device="cuda")
    v = buf[offset:].as_strided((r, c), (c + pad, 1))
    v.copy_(t)
    return v


def empty_padded(r, c, dtype, pad, offset=0):
    buf = torch.zeros((r * (c + pad) + offset + 64) * dtype.itemsize, dtype=torch.uint8, device="cuda")
    buf.fill_(0x55)
    return buf.view(dtype)[offset:].as_strided((r, c), (c + pad, 1)), buf


def heavy(rng, rows, cols):
    x = rng.standard_t(3, size=(rows, cols)).astype(np.float32)
    if cols > 40:
        x[:, rng.choice(cols, cols // 40, replace=False)] *= 50
    return x


def say(*a):
    print("\n[case]", *a, flush=True)


def check_codes(got, x, block_rows, kind):
    v, _ = Q.quotients(x, block_rows, kind)
    want = Q.encode(v)
    off = (got != want) & ~np.isnan(v)
    assert np.all(np.isnan(Q.decode(got[np.isnan(v)])))
    if off.any():
        assert np.all(np.abs(got[off].astype(int) - want[off].astype(int)) == 1)
        mid = (Q.decode(got[off]) + Q.decode(want[off])) / 2
        assert np.all(np.abs(v[off] - mid) <= 2.0 ** -23 * np.abs(mid)) and np.all(v[off] != mid)


# ------------------------------------------------------------------ coding
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (130, 129), (257, 640), (17, 2311), (64, 5120)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_is_exact(rows, cols, block_rows, io, kind):
    say("quantize", rows, cols, block_rows, io, kind)
    rng = np.random.default_rng(rows * 10007 + cols)
    x = torch.from_numpy(heavy(rng, rows, cols)).to(IO[io])
    x[rows // 2, :] = 0
    codes, scales = H.harp_quantize_q8(x.cuda(), block_rows, kind)
    torch.cuda.synchronize()
    assert np.array_equal(scales_np(scales), Q.quantize(x.float().numpy(), block_rows, kind)[1])
    check_codes(codes_np(codes), x.float().numpy(), block_rows, kind)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(block_rows, kind):
    say("quantize special", block_rows, kind)
    x = np.zeros((300, 520), dtype=np.float32)
    rng = np.random.default_rng(3)
    x[:, 128:256] = rng.standard_normal((300, 128)) * 1e-38      # below the smallest scale
    x[:, 256:384] = rng.standard_normal((300, 128)) * 1e38
    x[0, 256] = 3.4e38
    x[1, 384] = np.nan
    x[2, 519] = np.inf
    x[3, 518] = -np.inf
    x[7, 0:128] = 448.0 * 2.0 ** rng.integers(-8, 1, 128)        # maximum exactly 448 times a power of two
    codes, scales = H.harp_quantize_q8(torch.from_numpy(x).cuda(), block_rows, kind)
    torch.cuda.synchronize()
    want_s = Q.quantize(x, block_rows, kind)[1]
    got_s, got_c = scales_np(scales), codes_np(codes)
    assert np.array_equal(got_s, want_s, equal_nan=True)
    bad = np.isnan(Q.spread(want_s, block_rows, *x.shape))
    assert bad.any() and np.all(np.isnan(Q.decode(got_c[bad])))
    check_codes(got_c, x, block_rows, kind)


def test_quantize_ties_go_to_even():
    # values half way between two codes of a block with a maximum that is no power of two
    say("quantize ties")
    x = np.zeros((3, 128), dtype=np.float32)
    for r, top in enumerate((448.0, 3.0, 5.25)):
        mids = (Q.E4M3[0:126] + Q.E4M3[1:127]) / 2
        x[r, :126] = mids / 448.0 * top * np.where(np.arange(126) % 2, 1, -1)
        x[r, 127] = top
    keep = x.astype(np.float64) * 448.0 / np.array([[448.0], [3.0], [5.25]])
    codes, _ = H.harp_quantize_q8(torch.from_numpy(x).cuda())
    torch.cuda.synchronize()
    exact = np.isin(np.abs(keep), (Q.E4M3[0:126] + Q.E4M3[1:127]) / 2)
    assert exact.sum() > 126
    assert np.array_equal(codes_np(codes)[exact], Q.encode(keep)[exact])


def test_quantize_strides_and_guard_bytes():
    say("quantize strides")
    rng = np.random.default_rng(4)
    for io in ("f32", "bf16"):
        for pad, off in ((3, 1), (5, 0), (16, 8)):
            x = torch.from_numpy(heavy(rng, 37, 333)).to(IO[io])
            v = padded(x.cuda(), pad, off)
            codes, buf = empty_padded(37, 333, torch.float8_e4m3fn, pad, off)
            H.harp_quantize_q8(v, 1, "f32", codes=codes)
            torch.cuda.synchronize()
            check_codes(codes_np(codes), x.float().numpy(), 1, "f32")
            raw = buf.cpu().numpy().copy()
            inside = np.zeros(raw.size, dtype=bool)
            for r in range(37):
                inside[off + r * (333 + pad):off + r * (333 + pad) + 333] = True
            assert np.all(raw[~inside] == 0x55)                   # nothing written between the rows


# -------------------------------------------------------------------- norm
def check_coded(codes, scales, want, kind):
    """codes and scales are a coding of `want` up to its fp32 error."""
    c, s = codes_np(codes), scales_np(scales).astype(np.float64)
    amax = Q.block_max(want, 1)
    exact = np.maximum(amax / Q.TOP, Q.FLOOR)
    if kind == "f32":
        assert np.all(np.abs(s - exact) <= SLACK * exact)
    else:
        assert np.all(np.log2(s) == np.round(np.log2(s)))
        assert np.all(s >= exact * (1 - SLACK)) and np.all(s < 2 * exact * (1 + SLACK))
    v = want / Q.spread(s, 1, *want.shape)
    got = Q.decode(c)
    a = np.abs(v)
    step = np.where(a < 2.0 ** -6, 2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(a, 1e-30))) - 3))
    assert np.all(np.abs(got - v) <= step * 0.5 + SLACK * a * 2), np.max(np.abs(got - v) / step)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,gamma,residual,ckpt", [
    (1, 4096, False, True, False), (5, 1, True, True, True), (3, 130, True, False, True), (70, 4099, True, True, True),
    (33, 5120, False, True, True), (2, 20001, True, True, True), (1000, 64, True, True, True), (35, 128, True, False, True),
    (2, 9001, True, True, True), (2, 32768, False, False, True), (9, 512, True, True, False),
    (17001, 200, True, True, True), (9, 256, False, True, True), (3, 129, True, False, False)])
def test_rmsnorm(rows, d, gamma, residual, ckpt, io, kind):
    say("rmsnorm", rows, d, gamma, residual, ckpt, io, kind)
    rng = np.random.default_rng(rows + d)
    x = torch.from_numpy(heavy(rng, rows, d)).to(IO[io])
    res = torch.from_numpy(heavy(rng, rows, d)).to(IO[io]) if residual else None
    g = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(IO[io]) if gamma else None
    eps = 1e-5
    out = H.harp_rmsnorm_q8(x.cuda(), None if res is None else res.cuda(), None if g is None else g.cuda(), eps, kind,
                            checkpoint=ckpt)
    torch.cuda.synchronize()
    n, h, r, xn = Q.rmsnorm(np64(x), None if res is None else np64(res), None if g is None else np64(g), eps)
    check_coded(out.codes, out.scales, n, kind)
    if residual:
        assert torch.equal(out.h.cpu(), (x.float() + res.float()).to(IO[io]))
    else:
        assert out.h.shape == x.shape
    if ckpt:
        assert np.all(np.abs(np64(out.rstd) - r) <= SLACK * r)
        check_coded(out.ckpt_codes, out.ckpt_scales, xn, kind)
    else:
        assert out.rstd is None and out.ckpt_codes is None


def test_rmsnorm_in_place_and_strides():
    say("rmsnorm in place")
    rng = np.random.default_rng(8)
    for io in ("f32", "bf16"):
        x = torch.from_numpy(heavy(rng, 19, 1283)).to(IO[io])
        res = torch.from_numpy(heavy(rng, 19, 1283)).to(IO[io])
        want = H.harp_rmsnorm_q8(x.cuda(), res.cuda())
        xs, rs = padded(x.cuda(), 7, 3), padded(res.cuda(), 2, 1)
        codes, _ = empty_padded(19, 1283, torch.float8_e4m3fn, 5, 1)
        got = H.harp_rmsnorm_q8(xs, rs, h=rs, codes=codes)
        torch.cuda.synchronize()
        assert torch.equal(got.codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(got.scales, want.scales) and torch.equal(rs, want.h)
        assert torch.equal(xs.cpu(), x)


def test_rmsnorm_special_rows():
    say("rmsnorm special rows")
    x = np.random.default_rng(5).standard_normal((6, 300)).astype(np.float32)
    x[0] = 0
    x[1, 5] = np.nan
    x[2, 299] = np.inf
    x[3] *= 1e-30
    out = H.harp_rmsnorm_q8(torch.from_numpy(x).cuda(), None, None, 1e-6, "f32", checkpoint=True)
    torch.cuda.synchronize()
    v = Q.dequantize(codes_np(out.codes), scales_np(out.scales))
    assert np.all(v[0] == 0)
    assert np.all(np.isnan(v[1]))
    assert np.all(v[2, :256] == 0) and np.all(np.isnan(v[2, 256:]))   # the infinity's block; the rest is h * 0
    keep = [3, 4, 5]
    n = Q.rmsnorm(x.astype(np.float64)[keep], eps=1e-6)[0]
    check_coded(out.codes[keep], out.scales[keep], n, "f32")


# ----------------------------------------------------------- norm, backward
def coded(rng, x, kind):
    c, s = Q.quantize(x.astype(np.float32), 1, kind)
    return c, s


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,gamma,dres", [(1, 4096, True, True), (1, 1, True, False), (1500, 130, True, True),
                                               (37, 4099, False, True), (3, 20001, True, True), (40000, 64, True, True),
                                               (33, 128, True, False), (5, 9001, True, True), (2, 32768, True, False),
                                               (17001, 200, True, True), (9, 256, True, False), (3, 129, False, True)])
def test_rmsnorm_vjp(rows, d, gamma, dres, io, kind):
    say("rmsnorm_vjp", rows, d, gamma, dres, io, kind)
    rng = np.random.default_rng(rows + 3 * d)
    h = heavy(rng, rows, d)
    r = (1 / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1) + 1e-6)).astype(np.float32)
    c, s = coded(rng, h * r[:, None], kind)
    dn = torch.from_numpy(heavy(rng, rows, d)).to(IO[io])
    dr = torch.from_numpy(heavy(rng, rows, d)).to(IO[io]) if dres else None
    g = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(IO[io]) if gamma else None
    dh, dg = H.harp_rmsnorm_q8_vjp(to_codes(c), to_scales(s, kind), torch.from_numpy(r).cuda(), dn.cuda(),
                                   None if g is None else g.cuda(), None if dr is None else dr.cuda(),
                                   want_dgamma=True)
    torch.cuda.synchronize()
    want, wdg = Q.rmsnorm_vjp(Q.dequantize(c, s), r.astype(np.float64), np64(dn), None if g is None else np64(g),
                              None if dr is None else np64(dr))
    if d == 1 and not dres:       # u - n mean(u n) cancels: the bound is of the terms
        assert np.max(np.abs(np64(dh) - want)) <= 2 ** -7 * np.max(np.abs(np64(dn) * r[:, None])) * 2
    else:
        assert rel_rows(np64(dh), want) <= TOL[io]
    assert np.linalg.norm(np64(dg) - wdg) <= 1e-5 * np.linalg.norm(wdg)


def test_rmsnorm_vjp_against_differences():
    # h with values that E4M3 holds exactly, so that the checkpoint is the norm itself
    say("rmsnorm_vjp differences")
    rng = np.random.default_rng(11)
    rows, d, eps = 3, 150, 0.5
    h = Q.decode(rng.integers(0, 0x7f, (rows, d)).astype(np.uint8)) * rng.choice([-1.0, 1.0], (rows, d)) / 64
    h[:, [0, 40, 128]] = 7.0                                    # both blocks' maximum is 448 / 64
    g = 1 + 0.2 * rng.standard_normal(d).astype(np.float32)
    dn, dr = rng.standard_normal((rows, d)).astype(np.float32), rng.standard_normal((rows, d)).astype(np.float32)
    out = H.harp_rmsnorm_q8(torch.from_numpy(h.astype(np.float32)).cuda(), None, torch.from_numpy(g).cuda(), eps,
                            "f32", checkpoint=True)
    dh, dg = H.harp_rmsnorm_q8_vjp(out.ckpt_codes, out.ckpt_scales, out.rstd, torch.from_numpy(dn).cuda(),
                                   torch.from_numpy(g).cuda(), torch.from_numpy(dr).cuda())
    torch.cuda.synchronize()

    def loss(hh, gg):
        return np.sum(Q.rmsnorm(hh, None, gg, eps)[0] * dn) + np.sum(hh * dr)

    g64, e = g.astype(np.float64), 1e-4
    got, gotg = np64(dh), np64(dg)
    for i in range(rows):
        for j in range(0, d, 7):
            up, dw = h.copy(), h.copy()
            up[i, j] += e
            dw[i, j] -= e
            # central differences: error e^2 times the third derivative, far below 1e-5
            assert abs((loss(up, g64) - loss(dw, g64)) / (2 * e) - got[i, j]) <= 2e-5 * max(1.0, np.abs(got[i]).max())
    for j in range(0, d, 7):
        up, dw = g64.copy(), g64.copy()
        up[j] += e
        dw[j] -= e
        assert abs((loss(h, up) - loss(h, dw)) / (2 * e) - gotg[j]) <= 2e-5 * max(1.0, np.abs(gotg).max())


def test_rmsnorm_vjp_in_place_and_empty():
    say("rmsnorm_vjp in place, empty")
    rng = np.random.default_rng(12)
    rows, d = 41, 777
    c, s = coded(rng, rng.standard_normal((rows, d)), "f32")
    r = torch.rand(rows, device="cuda") + 0.5
    dn = torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32)).cuda()
    dr = torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32)).cuda()
    want, _ = H.harp_rmsnorm_q8_vjp(to_codes(c), to_scales(s, "f32"), r, dn, None, dr)
    a, b = padded(dn, 3, 1), padded(dr, 9, 2)
    H.harp_rmsnorm_q8_vjp(to_codes(c), to_scales(s, "f32"), r, a, None, dr, dh=a)
    H.harp_rmsnorm_q8_vjp(to_codes(c), to_scales(s, "f32"), r, dn, None, b, dh=b)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    dg = torch.full((d,), 7.0, device="cuda")
    z = torch.empty(0, d, device="cuda")
    H.harp_rmsnorm_q8_vjp(torch.empty(0, d, dtype=torch.float8_e4m3fn, device="cuda"),
                          torch.empty(0, Q.nblk(d), device="cuda"), torch.empty(0, device="cuda"), z, dgamma=dg)
    torch.cuda.synchronize()
    assert torch.all(dg == 0)


# ---------------------------------------------------------------- products
def operands(rng, rows, n, k, kind):
    a = rng.standard_normal((rows, k)) * np.exp(rng.standard_normal((rows, 1)))
    a[rows // 2] = 0
    w = rng.standard_normal((n, k)) * 0.02
    return Q.quantize(a, 1, kind), Q.quantize(w, 128, kind)


MATMUL = [(1, 1, 1), (1, 4096, 4096), (2, 130, 127), (5, 64, 129), (16, 300, 640), (17, 257, 1040), (33, 1000, 272),
          (64, 512, 2048), (65, 129, 128), (100, 700, 1000), (128, 128, 4096), (129, 385, 515), (200, 2100, 384),
          (300, 260, 5120), (513, 1030, 1296), (1030, 777, 400)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", MATMUL)
def test_matmul(rows, n, k, out, kind):
    say("matmul", rows, n, k, out, kind)
    rng = np.random.default_rng(rows + 7 * n + 13 * k)
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), out)
    torch.cuda.synchronize()
    assert rel_rows(np64(y), Q.matmul(ac, as_, wc, ws)) <= TOL[out]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", [(4200, 5130, 1168), (4353, 4100, 128), (8192, 2064, 272), (4096, 4096, 400)])
def test_matmul_large(rows, n, k, out, kind):
    # a round of the largest tiles on 256 compute units, ragged on every side; one, a few and many blocks of 128
    say("matmul", rows, n, k, out, kind)
    rng = np.random.default_rng(21)
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), out)
    torch.cuda.synchronize()
    assert rel_rows(np64(y), Q.matmul(ac, as_, wc, ws)) <= TOL[out]


@pytest.mark.parametrize("rows", [1, 50, 300])
def test_matmul_strides(rows):
    say("matmul strides", rows)
    rng = np.random.default_rng(22)
    n, k = 333, 528
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, "f32")
    want = Q.matmul(ac, as_, wc, ws)
    for pad, off in ((1, 3), (16, 0), (16, 16), (8, 4)):
        a, w = padded(to_codes(ac), pad, off), padded(to_codes(wc), pad, off)
        y, buf = empty_padded(rows, n, torch.float32, pad, off)
        H.harp_matmul_q8(a, to_scales(as_, "f32"), w, to_scales(ws, "f32"), "f32", y=y)
        torch.cuda.synchronize()
        assert rel_rows(np64(y), want) <= TOL["f32"]
        raw = buf.view(torch.int32).cpu().numpy()
        inside = np.zeros(raw.size, dtype=bool)
        for r in range(rows):
            inside[off + r * (n + pad):off + r * (n + pad) + n] = True
        assert np.all(raw[~inside] == 0x55555555)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("rows", [3, 40, 200])
def test_matmul_special_values(rows, kind):
    # a NaN code, a NaN scale and a zero block reach their own row or columns only
    say("matmul special", rows, kind)
    rng = np.random.default_rng(23)
    n, k = 300, 400
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    ac[1, 399] = 0x7f
    as_[2, 0] = np.nan
    ws[1, 2] = np.nan
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), "f32")
    torch.cuda.synchronize()
    want = Q.matmul(ac, as_, wc, ws)
    got = np64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = [r for r in range(rows) if r not in (1, 2)]
    cols = np.r_[0:128, 256:300]
    assert rel_rows(got[np.ix_(ok, cols)], want[np.ix_(ok, cols)]) <= TOL["f32"]


def test_matmul_extreme_scales():
    # E8M0 bytes at both ends and fp32 scales whose product leaves the normal range only together
    say("matmul extreme scales")
    rng = np.random.default_rng(24)
    (ac, as_), (wc, ws) = operands(rng, 20, 40, 300, "e8m0")
    as_[:, 1] = 2.0 ** -126
    ws[0, 1] = 2.0 ** 127
    as_[:, 0] = 2.0 ** 100
    ws[0, 0] = 2.0 ** -110
    for kind in ("f32", "e8m0"):
        y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), "f32")
        torch.cuda.synchronize()
        assert rel_rows(np64(y), Q.matmul(ac, as_, wc, ws)) <= TOL["f32"]


def test_matmul_far_offsets():
    # rows more than 2^31 bytes apart in a buffer of 4.3 GB
    say("matmul far offsets")
    rng = np.random.default_rng(25)
    (ac, as_), (wc, ws) = operands(rng, 3, 150, 256, "f32")
    ld = (1 << 31) + 4096
    big = torch.empty(2 * ld + 256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    a = big.as_strided((3, 256), (ld, 1))
    a.copy_(to_codes(ac))
    y = H.harp_matmul_q8(a, to_scales(as_, "f32"), to_codes(wc), to_scales(ws, "f32"), "f32")
    q, s = H.harp_quantize_q8(big.view(torch.bfloat16).as_strided((2, 64), (ld // 2, 1)))
    torch.cuda.synchronize()
    assert rel_rows(np64(y), Q.matmul(ac, as_, wc, ws)) <= TOL["f32"]
    x = big.view(torch.bfloat16).as_strided((2, 64), (ld // 2, 1)).float().cpu().numpy()
    keep = np.isfinite(x).all(axis=1)
    check_codes(codes_np(q)[keep], x[keep], 1, "f32")


@pytest.mark.parametrize("ldy", [1 << 21, 1 << 22])
def test_matmul_far_result_rows(ldy):
    # a 256-row tile of results over 1 and 2 GiB
    say("matmul far result rows", ldy)
    rng = np.random.default_rng(26)
    rows, n, k = 256, 160 * 256, 256
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, "f32")
    y = torch.empty((rows - 1) * ldy + n, dtype=torch.bfloat16, device="cuda").as_strided((rows, n), (ldy, 1))
    H.harp_matmul_q8(to_codes(ac), to_scales(as_, "f32"), to_codes(wc), to_scales(ws, "f32"), y=y)
    torch.cuda.synchronize()
    assert rel_rows(np64(y), Q.matmul(ac, as_, wc, ws)) <= TOL["bf16"]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_wgrad_far_rows(kind):
    # rows more than 2^22 values apart
    say("wgrad far rows", kind)
    rng = np.random.default_rng(32)
    rows, n, k, ld = 70, 144, 272, (1 << 22) + 16
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, kind)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16)
    fx = torch.empty((rows - 1) * ld + k, dtype=torch.float8_e4m3fn, device="cuda").as_strided((rows, k), (ld, 1))
    fd = torch.empty((rows - 1) * ld + n, dtype=torch.bfloat16, device="cuda").as_strided((rows, n), (ld, 1))
    fx.copy_(to_codes(xc))
    fd.copy_(dy.cuda())
    want = Q.wgrad(np64(dy), xc, xs)
    for a, b in ((fd, fx), (dy.cuda(), fx), (fd, to_codes(xc))):
        dw = H.harp_matmul_q8_wgrad(a, b, to_scales(xs, kind), "f32")
        torch.cuda.synchronize()
        assert rel_rows(np64(dw), want) <= TOL["f32"]


WGRAD = [(1, 1, 1), (1, 300, 130), (31, 128, 128), (32, 64, 640), (33, 129, 127), (100, 500, 272), (257, 260, 515),
         (1000, 384, 256), (1500, 1030, 400), (5000, 64, 80), (4097, 16, 130)]
# more than 256 tiles: the large tile for some formats, the small one for others
WGRAD_LARGE = [(100, 4096, 2048), (70, 2111, 4200), (65, 2048, 2304)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", WGRAD + WGRAD_LARGE)
def test_wgrad(rows, n, k, out, kind):
    say("wgrad", rows, n, k, out, kind)
    rng = np.random.default_rng(rows + 5 * n + 11 * k)
    xc, xs = Q.quantize(rng.standard_normal((rows, k)) * np.exp(rng.standard_normal((rows, 1))), 1, kind)
    dy = torch.from_numpy(heavy(rng, rows, n) * np.float32(1e-3)).to(torch.bfloat16)
    dw = H.harp_matmul_q8_wgrad(dy.cuda(), to_codes(xc), to_scales(xs, kind), out)
    torch.cuda.synchronize()
    want = Q.wgrad(np64(dy), xc, xs)
    # bf16 results of fp32 scales: x rounded (2^-9) and the result rounded (2^-9), independent
    tol = TOL[out] * (1.5 if out == "bf16" and kind == "f32" else 1.0)
    assert rel_rows(np64(dw), want) <= tol


def test_wgrad_strides_and_special_values():
    say("wgrad strides")
    rng = np.random.default_rng(31)
    rows, n, k = 200, 144, 272
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, "e8m0")
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16)
    want = Q.wgrad(np64(dy), xc, xs)
    for pad, off in ((1, 3), (16, 0), (16, 16), (8, 8)):
        dw, buf = empty_padded(n, k, torch.float32, pad, off)
        H.harp_matmul_q8_wgrad(padded(dy.cuda(), pad, off), padded(to_codes(xc), pad, off), to_scales(xs, "e8m0"),
                               "f32", dw=dw)
        torch.cuda.synchronize()
        assert rel_rows(np64(dw), want) <= TOL["f32"]
        raw = buf.view(torch.int32).cpu().numpy()
        inside = np.zeros(raw.size, dtype=bool)
        for r in range(n):
            inside[off + r * (k + pad):off + r * (k + pad) + k] = True
        assert np.all(raw[~inside] == 0x55555555)
    # a NaN gradient reaches its own output row, a NaN code its own column
    dy[5, 7] = float("nan")
    xc[9, 200] = 0x7f
    got = np64(H.harp_matmul_q8_wgrad(dy.cuda(), to_codes(xc), to_scales(xs, "e8m0"), "f32"))
    bad = np.zeros((n, k), dtype=bool)
    bad[7] = True
    bad[:, 200] = True
    assert np.array_equal(np.isnan(got), bad)


def test_wgrad_empty_writes_zeros():
    say("wgrad empty")
    dw = torch.full((70, 50), 3.0, device="cuda")
    H.harp_matmul_q8_wgrad(torch.empty(0, 70, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(0, 50, dtype=torch.float8_e4m3fn, device="cuda"),
                           torch.empty(0, 1, device="cuda"), "f32", dw=dw)
    torch.cuda.synchronize()
    assert torch.all(dw == 0)
    y = H.harp_matmul_q8(torch.empty(0, 50, dtype=torch.float8_e4m3fn, device="cuda"),
                         torch.empty(0, 1, device="cuda"), to_codes(np.zeros((4, 50), np.uint8)),
                         torch.ones(1, 1, device="cuda"))
    assert y.shape == (0, 4)


# -------------------------------------------------- streams, graphs, repeats
def _chain(x, res, g, wc, ws, dy):
    """Every operator once, feeding each other."""
    o = H.harp_rmsnorm_q8(x, res, g, 1e-6, "f32", checkpoint=True)
    y = H.harp_matmul_q8(o.codes, o.scales, wc, ws, "bf16")
    dw = H.harp_matmul_q8_wgrad(dy, o.codes, o.scales, "f32")
    dyc, dys = H.harp_quantize_q8(dy)
    dn = H.harp_matmul_q8(dyc, dys, wc.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn),
                          ws.t().contiguous(), "bf16")
    dh, dg = H.harp_rmsnorm_q8_vjp(o.ckpt_codes, o.ckpt_scales, o.rstd, dn, g, dy[:, :x.shape[1]].contiguous())
    return [o.codes.view(torch.uint8), o.scales, o.h, y, dw, dyc.view(torch.uint8), dn, dh, dg]


def _chain_inputs(rows=150, n=400, d=272):
    rng = np.random.default_rng(41)
    x = torch.from_numpy(heavy(rng, rows, d)).to(torch.bfloat16).cuda()
    res = torch.from_numpy(heavy(rng, rows, d)).to(torch.bfloat16).cuda()
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    wc, ws = H.harp_quantize_q8(torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda(), 128)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    return x, res, g, wc, ws, dy


def test_repeats_are_equal_and_streams_are_kept():
    say("repeats, streams")
    args = _chain_inputs()
    first = _chain(*args)
    second = _chain(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        third = _chain(*args)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays():
    say("graph")
    args = _chain_inputs()
    want = [t.clone() for t in _chain(*args)]
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _chain(*args)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        got = _chain(*args)
    for _ in range(4):
        for t in got:
            t.view(torch.uint8).zero_()
        _chain(*args)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
