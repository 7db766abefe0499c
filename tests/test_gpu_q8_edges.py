"""The 8-bit operators at special values: where a NaN, an infinity or a value
at the end of fp32's range may reach, in every form of the kernels.

Oracle and tolerances are those of tests/test_gpu_q8.py.
"""
import numpy as np
import pytest
import torch

import structured_rotations_amd as H
from oracle import q8_oracle as Q
from tests.test_gpu_q8 import (IO, SCALE, SLACK, TOL, check_coded, empty_padded, np64, operands, padded, rel_rows, say,
                               to_codes, to_scales)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- products
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_matmul_nan_stays_in_its_tile(kind):
    # 17 x 17 tiles of 256 x 256: 289, so that some of 256 workgroups compute a second one after the first.  Every
    # row of tiles has a NaN code in another row of the tile, in the last block of 128; one weight block is NaN
    say("matmul nan, two tiles per workgroup", kind)
    rng = np.random.default_rng(51)
    rows, n, k = 4352, 4352, 384
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    bad = [256 * t + 32 + (7 * t) % 32 for t in range(17)]
    ac[bad, 300] = 0x7f
    wc[1024:1152, 256:] = 0x7f
    ws[8, 2] = np.nan
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), "bf16")
    torch.cuda.synchronize()
    got = np64(y)
    mask = np.zeros((rows, n), dtype=bool)
    mask[bad] = True
    mask[:, 1024:1152] = True
    assert np.array_equal(np.isnan(got), mask)
    ok = np.setdiff1d(np.arange(rows), bad)
    cols = np.r_[0:1024, 1152:n]
    want = Q.matmul(ac[ok], as_[ok], wc, np.where(np.isnan(ws), 0, ws))
    assert rel_rows(got[np.ix_(ok, cols)], want[:, cols]) <= TOL["bf16"]


# where NaNs reach, per form of the product: rows, n, k that choose it (fp32 results never take the 256 x 256 form)
FORMS = [(3, 300, 400), (40, 300, 400), (200, 300, 400), (3, 300, 395), (40, 300, 395), (200, 300, 395),
         (40, 300, 2048), (1024, 2048, 400), (2304, 2304, 400), (4352, 2560, 400)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", FORMS)
def test_matmul_special_values_by_form(rows, n, k, out, kind):
    # a NaN code, NaN scales of both operands, zero blocks: own row or columns only
    say("matmul special by form", rows, n, k, out, kind)
    rng = np.random.default_rng(52)
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    ac[1, k - 1] = 0x7f
    as_[2, 0] = np.nan
    wc[n - 1, 130] = 0xff
    ws[1, 2] = np.nan
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, kind), to_codes(wc), to_scales(ws, kind), out)
    torch.cuda.synchronize()
    want = Q.matmul(ac, as_, wc, ws)
    got = np64(y)
    mask = np.zeros((rows, n), dtype=bool)
    mask[[1, 2]] = True
    mask[:, 128:256] = True
    mask[:, n - 1] = True
    assert np.array_equal(np.isnan(want), mask) and np.array_equal(np.isnan(got), mask)
    ok = [r for r in range(rows) if r not in (1, 2)]
    cols = np.r_[0:128, 256:n - 1]
    assert rel_rows(got[np.ix_(ok, cols)], want[np.ix_(ok, cols)]) <= TOL[out]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_matmul_strided_operands_of_large_tiles(kind):
    # the 256 x 256 form: operands and results with rows apart, whole 16-byte pieces or not
    say("matmul strides, large", kind)
    rng = np.random.default_rng(53)
    rows, n, k = 4100, 2576, 272
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, kind)
    want = Q.matmul(ac, as_, wc, ws)
    for pad, off in ((16, 16), (48, 0), (3, 5)):
        y, buf = empty_padded(rows, n, torch.bfloat16, pad, off)
        H.harp_matmul_q8(padded(to_codes(ac), pad, off), to_scales(as_, kind), padded(to_codes(wc), pad, off),
                         to_scales(ws, kind), y=y)
        torch.cuda.synchronize()
        assert rel_rows(np64(y), want) <= TOL["bf16"]
        outside = torch.ones(buf.numel() // 2, dtype=torch.bool, device="cuda")
        outside[off:].as_strided((rows, n), (n + pad, 1)).fill_(False)
        assert torch.all(buf.view(torch.int16)[outside] == 0x5555)


# --------------------------------------------------------- weight gradient
def same_specials(got, want, out):
    """NaNs and infinities where the formula in fp64, rounded to the result's type, has them."""
    want = np64(torch.from_numpy(want).float().to(IO[out]))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got == np.inf, want == np.inf) and np.array_equal(got == -np.inf, want == -np.inf)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", [(40, 144, 272), (200, 144, 272), (90, 77, 301), (70, 4096, 2304)])
def test_wgrad_infinite_gradients(rows, n, k, out, kind):
    say("wgrad infinities", rows, n, k, out, kind)
    rng = np.random.default_rng(61)
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, kind)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16)
    dy[5, 7], dy[6, 20], dy[38, 30], dy[39, 30] = float("inf"), float("-inf"), float("inf"), float("inf")
    xc[5, 3] = 0                                                  # inf * 0: a NaN by the formula, too
    with np.errstate(invalid="ignore"):
        want = Q.wgrad(np64(dy), xc, xs)
    got = np64(H.harp_matmul_q8_wgrad(dy.cuda(), to_codes(xc), to_scales(xs, kind), out))
    assert np.isnan(want).sum() >= 1 and np.isinf(want).sum() >= 2 * k - 2
    same_specials(got, want, out)
    ok = np.setdiff1d(np.arange(n), (7, 20, 30))
    assert rel_rows(got[ok], want[ok]) <= TOL[out] * (1.5 if out == "bf16" and kind == "f32" else 1.0)


@pytest.mark.parametrize("out,rows", [("f32", 40), ("f32", 200), ("bf16", 40)])
def test_wgrad_ends_of_the_range(out, rows):
    # values next to fp32's largest, infinite scales, and products that leave the range in the first part of a value
    say("wgrad range", out, rows)
    rng = np.random.default_rng(62)
    n, k = 48, 400
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, "f32")
    dy = np.zeros((rows, n), dtype=np.float32)
    dy[:, :16] = rng.standard_normal((rows, 16)) * 2.0 ** -30
    xs[:, 0] = 3.4e38 / 448
    xc[3, :128] = 0x7e                                            # 3.4e38
    dy[11, 20] = 2.0 ** 126
    xs[11, 1] = 0.3
    xc[11, 128:256] = rng.integers(0x58, 0x7f, 128)               # 16 .. 448, times 0.3: no bf16 values
    xs[12, 2] = np.inf
    xc[12, 256:384] = np.where(rng.random(128) < 0.5, 0x38, 0xb8)
    dy[12, 5], dy[12, 30] = 1.0, -1.0
    dyt = torch.from_numpy(dy).to(torch.bfloat16)
    with np.errstate(invalid="ignore"):
        want = Q.wgrad(np64(dyt), xc, xs)
    got = np64(H.harp_matmul_q8_wgrad(dyt.cuda(), to_codes(xc), to_scales(xs, "f32"), out))
    same_specials(got, want, out)
    keep = np.r_[0:5, 6:16]
    assert rel_rows(got[keep, :256], want[keep, :256]) <= TOL[out]
    assert (want[20, 128:256] > 3.41e38).all() and np.isfinite(want[:5, :256]).all()


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", [(40, 144, 272), (200, 144, 272), (200, 141, 275), (70, 4096, 2304),
                                      (70, 4099, 2305)])
def test_wgrad_nan_scales(rows, n, k, out, kind):
    # a NaN gradient reaches its result row, a NaN code its column, a NaN scale its block of 128 columns
    say("wgrad nan", rows, n, k, out, kind)
    rng = np.random.default_rng(63)
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, kind)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16)
    dy[5, 7] = float("nan")
    xc[9, 3] = 0xff
    xs[rows - 1, 1] = np.nan
    want = Q.wgrad(np64(dy), xc, xs)
    got = np64(H.harp_matmul_q8_wgrad(dy.cuda(), to_codes(xc), to_scales(xs, kind), out))
    mask = np.zeros((n, k), dtype=bool)
    mask[7] = True
    mask[:, 3] = True
    mask[:, 128:256] = True
    assert np.array_equal(np.isnan(got), mask)
    rest = np.ix_(np.setdiff1d(np.arange(n), 7), np.setdiff1d(np.arange(k), np.r_[3, 128:256]))
    assert rel_rows(got[rest], want[rest]) <= TOL[out] * (1.5 if out == "bf16" and kind == "f32" else 1.0)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k", [(50, 144, 272), (200, 144, 272), (70, 4096, 2304)])
def test_wgrad_strided_operands(rows, n, k, out, kind):
    say("wgrad strides", rows, n, k, out, kind)
    rng = np.random.default_rng(64)
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, kind)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).to(torch.bfloat16)
    want = Q.wgrad(np64(dy), xc, xs)
    for pad, off in ((1, 3), (16, 0), (16, 16), (8, 8)):
        dw, buf = empty_padded(n, k, IO[out], pad, off)
        H.harp_matmul_q8_wgrad(padded(dy.cuda(), pad, off), padded(to_codes(xc), pad, off), to_scales(xs, kind), out,
                               dw=dw)
        torch.cuda.synchronize()
        assert rel_rows(np64(dw), want) <= TOL[out] * (1.5 if out == "bf16" and kind == "f32" else 1.0)
        word = torch.int32 if out == "f32" else torch.int16
        outside = torch.ones(buf.numel() // word.itemsize, dtype=torch.bool, device="cuda")
        outside[off:].as_strided((n, k), (k + pad, 1)).fill_(False)
        assert torch.all(buf.view(word)[outside] == (0x55555555 if out == "f32" else 0x5555))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [40, 200])
def test_wgrad_ends_of_the_powers(rows, out):
    # E8M0 scales of either end, and dy that brings the products back
    say("wgrad e8m0 ends", rows, out)
    rng = np.random.default_rng(65)
    n, k = 48, 400
    xc, xs = Q.quantize(rng.standard_normal((rows, k)), 1, "e8m0")
    xs[:, 0] = 2.0 ** -110
    xs[:, 1] = 2.0 ** 110
    xs[:, 2] = 2.0 ** 118
    dy = torch.from_numpy((rng.standard_normal((rows, n)) * 2.0 ** -20).astype(np.float32)).to(torch.bfloat16)
    want = Q.wgrad(np64(dy), xc, xs)
    got = np64(H.harp_matmul_q8_wgrad(dy.cuda(), to_codes(xc), to_scales(xs, "e8m0"), out))
    for j in range(4):
        at = np.s_[:, 128 * j:128 * j + 128]
        assert rel_rows(got[at], want[at]) <= TOL[out]


# -------------------------------------------------------------------- norm
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 200, 300, 4099, 5120, 20001])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rmsnorm_far_from_one(d, io, kind, eps):
    # rows whose squares leave fp32's range at either end
    say("rmsnorm range", d, io, kind, eps)
    rng = np.random.default_rng(d)
    mult = np.array([1.0, 2e37, 1e25, 1e19, 1e18, 1.0] + ([1e-18, 1e-25, 1e-33] if eps == 0 else [1e-9]))
    x = rng.standard_normal((len(mult), d)) * mult[:, None]
    x = torch.from_numpy(x.astype(np.float32)).to(IO[io])
    g = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(IO[io])
    out = H.harp_rmsnorm_q8(x.cuda(), None, g.cuda(), eps, kind, checkpoint=True)
    torch.cuda.synchronize()
    n, _, r, xn = Q.rmsnorm(np64(x), None, np64(g), eps)
    assert np.all(np.abs(np64(out.rstd) - r) <= SLACK * r)
    check_coded(out.codes, out.scales, n, kind)
    check_coded(out.ckpt_codes, out.ckpt_scales, xn, kind)


# ----------------------------------------------------------------- streams
def test_memory_of_a_call_on_another_stream():
    # while the call's stream is busy, the current stream gets none of the call's memory, dropped or not
    say("memory of another stream")
    rng = np.random.default_rng(71)
    rows, n, k = 128, 128, 4096
    (ac, as_), (wc, ws) = operands(rng, rows, n, k, "f32")
    args = to_codes(ac), to_scales(as_, "f32"), to_codes(wc), to_scales(ws, "f32")
    need = H.harp_matmul_q8_workspace(rows, n, k)
    assert need > 0
    want = H.harp_matmul_q8(*args, "f32")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                         # about 10 ms
        y = H.harp_matmul_q8(*args, "f32", stream=side)
        dropped = H.harp_matmul_q8(*args, "f32", stream=side).data_ptr()
        others = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        others += [torch.full((rows, n), float("nan"), device="cuda") for _ in range(4)]
        assert dropped not in [t.data_ptr() for t in others]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, want)
        assert all(torch.all(t == 255) for t in others[:4]) and all(torch.isnan(t).all() for t in others[4:])


# ------------------------------------------------- arguments in one buffer
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_arguments_side_by_side_in_one_buffer(io):
    # columns of one buffer as input and output, and as two outputs: no common byte
    say("side by side", io)
    rng = np.random.default_rng(91)
    rows, d, n = 37, 272, 400
    x, res = (torch.from_numpy(rng.standard_normal((rows, d)).astype(np.float32)).to(IO[io]).cuda() for _ in range(2))
    g = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(IO[io]).cuda()
    want = H.harp_rmsnorm_q8(x, res, g, checkpoint=True)
    buf = torch.empty(rows, 3 * d + 5, dtype=IO[io], device="cuda")
    xb, rb, hb = buf[:, 5:5 + d], buf[:, 5 + d:5 + 2 * d], buf[:, 5 + 2 * d:]
    xb.copy_(x)
    rb.copy_(res)
    codes = torch.empty(rows, 2 * d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    got = H.harp_rmsnorm_q8(xb, rb, g, checkpoint=True, h=hb, codes=codes[:, d:], ckpt_codes=codes[:, :d])
    for a, b in ((got.codes, want.codes), (got.ckpt_codes, want.ckpt_codes)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(hb, want.h) and torch.equal(xb, x) and torch.equal(rb, res)
    dh, dg = H.harp_rmsnorm_q8_vjp(want.ckpt_codes, want.ckpt_scales, want.rstd, xb, g, rb, dh=hb)
    want_dh, want_dg = H.harp_rmsnorm_q8_vjp(want.ckpt_codes, want.ckpt_scales, want.rstd, x, g, res)
    assert torch.equal(dh, want_dh) and torch.equal(dg, want_dg) and torch.equal(xb, x)
    wc, ws = H.harp_quantize_q8(torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda(), 128)
    both = torch.empty(rows, d + 2 * n, dtype=torch.uint8, device="cuda")
    ab = both[:, 2 * n:].view(torch.float8_e4m3fn)
    ab.copy_(want.codes)
    yb = both.view(torch.bfloat16)[:, :n]
    H.harp_matmul_q8(ab, want.scales, wc, ws, y=yb)
    assert torch.equal(yb, H.harp_matmul_q8(want.codes, want.scales, wc, ws))
    assert torch.equal(ab.contiguous().view(torch.uint8), want.codes.view(torch.uint8))


# ---------------------------------------------------------- largest sizes
BIG = 1 << 30


def test_wgrad_of_the_most_rows():
    # dw has 2^30 rows of one value: dy times one power of two, exact
    say("wgrad n = 2^30")
    dy = (torch.arange(BIG, device="cuda", dtype=torch.int32) % 251 + 1).to(torch.bfloat16).view(1, BIG)
    x = torch.full((1, 1), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.full((1, 1), 0x7d, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    dw = H.harp_matmul_q8_wgrad(dy, x, scale, "f32")
    torch.cuda.synchronize()
    assert torch.equal(dw.view(-1), dy.view(-1).float() * 0.25)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_wgrad_of_the_longest_rows(kind):
    # one row of 2^30 values times 2: exact, fp32 scales with few bits
    say("wgrad k = 2^30", kind)
    codes = (torch.arange(BIG, device="cuda", dtype=torch.int32) % 119 + 8).to(torch.uint8).view(1, BIG)
    scale = torch.full((1, BIG // 128), 0.25, device="cuda")
    dw = H.harp_matmul_q8_wgrad(torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda"),
                                codes.view(torch.float8_e4m3fn), scale.to(SCALE[kind]), "f32")
    torch.cuda.synchronize()
    table = torch.from_numpy(Q.E4M3 * 0.5).float().cuda()
    for i in range(0, BIG, BIG // 8):
        want = table[codes[0, i:i + BIG // 8].int()]
        assert torch.all((dw[0, i:i + BIG // 8] - want).abs() <= 1e-6 * want)


@pytest.mark.parametrize("n,k", [(BIG, 16), ((1 << 28) + 4096, 17)])
def test_matmul_of_the_most_columns(n, k):
    # one row by n weight rows that repeat: results repeat, too
    say("matmul n", n, k)
    rng = np.random.default_rng(81)
    part = 1 << 12
    (ac, as_), (wc, _) = Q.quantize(rng.standard_normal((1, k))), Q.quantize(rng.standard_normal((part, k)), 128)
    ones = np.ones((part // 128, 1), np.float32)
    w = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    w.view(n // part, part, k).copy_(torch.from_numpy(wc).cuda())
    y = H.harp_matmul_q8(to_codes(ac), to_scales(as_, "f32"), w.view(torch.float8_e4m3fn),
                         torch.ones(n // 128, 1, device="cuda"), "bf16")
    torch.cuda.synchronize()
    y = y.view(n // part, part)
    assert rel_rows(np64(y[:1]), Q.matmul(ac, as_, wc, ones)) <= TOL["bf16"]
    assert torch.all(y == y[:1])
