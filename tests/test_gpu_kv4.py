"""Attention over a 4-bit cache on the GPU against the fp64 oracle.

Tolerances.  u = 2^-24 and h = 2^-8 are the largest relative errors of one
rounding to fp32 and to bf16.
- norm_rope, a head in l2: the sum of squares (d / 8 terms a lane, then 6
  exchanges) and its root 10 u, three products 3 u, cosine and sine 4 u each off
  (the angle's fraction of a turn is rounded to 2^-26 turns, 2^-23.3 radians) and
  two roundings, over a pair 9 u, 9 Hadamard stages and the normalisation 10 u:
  32 u = 2^-19; a bf16 result adds h.
- its reverse mode: the same for g and, relative to r |gamma g| of the head (the
  two parts of dx cancel), as much again for n and the mean: 2^-18; a bf16 result
  adds h of itself.  dgamma, relative to the sum of |g n|: 2^-18 and the sums in
  fp32, at most 100 terms one after the other in these tests: 2^-17.
- the cache is exact: codes, scales and values read back.
- attention: a score is d products summed in fp32, off by at most d u times the
  sum of their magnitudes (`score`), and by 3 u of itself by the scaling; call
  that dz.  A weight is off by dz, h for its rounding to bf16 and 2^-20 for the
  exponential and the sums: a result by 2 dz + h + 2^-19 of `size` (the weighted
  mean of |v|) and h of itself; lse by dz + 2^-20 + 2^-22 of itself.  Weights go
  by the largest, which is 1: one under 2^-126, which fp32 does not hold, is
  lost, and with it at most 2^-126 |v|, |v| < 2^6 here, for each of up to 2^13
  keys: 2^-107 in all.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as K
from structured_rotations_amd import kv4, rht_compose

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U, H = 2.0 ** -24, 2.0 ** -8
IO = {"f32": torch.float32, "bf16": BF}


def cpu(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def say(*a):
    print("\n[case]", *a, flush=True)


# ---------------------------------------------------- norm, position, rotation
QK = [  # d, pairs, interleaved, signs, gamma, io, tokens, q heads, k heads, positions up to
    (128, 64, False, True, True, "bf16", 5, 4, 2, 100),
    (128, 64, False, True, True, "f32", 37, 32, 8, 1 << 20),
    (128, 64, True, False, True, "f32", 1, 3, 1, 1 << 31),
    (128, 32, False, True, False, "f32", 9, 5, 0, 5000),
    (128, 16, True, True, True, "bf16", 300, 1, 1, 5000),
    (64, 32, False, True, True, "f32", 11, 7, 3, 300000),
    (64, 8, False, False, False, "bf16", 1000, 2, 2, 300000),
    (80, 24, True, False, True, "f32", 13, 12, 4, 2000000),
    (80, 40, False, False, True, "bf16", 13, 12, 4, 2000000),
    (96, 48, False, False, True, "f32", 21, 3, 3, 4096),
    (104, 8, False, False, True, "f32", 2, 17, 2, 4096),
    (192, 96, True, False, True, "bf16", 6, 6, 2, 4096),
    (256, 128, False, True, True, "f32", 7, 4, 1, 4096),
    (256, 64, True, True, True, "bf16", 33, 9, 3, 4096),
    (512, 256, False, True, True, "f32", 3, 2, 1, 4096),
    (512, 128, False, True, True, "bf16", 3, 5, 5, 4096),
    (8, 0, False, True, True, "f32", 50, 3, 2, 10),
    (16, 8, False, True, True, "f32", 50, 70, 2, 10),
    (32, 16, True, True, True, "bf16", 50, 3, 2, 10),
    (24, 8, False, False, True, "f32", 4, 1, 1, 10),
    (128, 64, False, True, True, "bf16", 5000, 3, 1, 10000),
]


def qk_case(d, pairs, inter, signs, gamma, io, tokens, hq, hk, far, seed=0):
    rng = np.random.default_rng(seed + d + tokens)
    dt = IO[io]
    # the projection's rows: queries, keys and something behind them, one odd element between tokens where alignment allows
    wide = (hq + hk + 1) * d + (1 if tokens % 2 else 0)
    buf = gpu(rng.standard_t(3, (tokens, wide)).astype(np.float32), dt)
    q = buf[:, :hq * d].unflatten(1, (hq, d))
    k = buf[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)) if hk else None
    w = {"gamma_q": gpu((1 + 0.3 * rng.standard_normal(d)).astype(np.float32), dt) if gamma else None,
         "gamma_k": gpu((1 + 0.3 * rng.standard_normal(d)).astype(np.float32), dt) if gamma and hk else None}
    pos = rng.integers(0, far, tokens)
    freqs = 10000.0 ** (-np.arange(pairs) / max(1, pairs))
    s = rng.choice([-1, 1], d).astype(np.int8) if signs else None
    position = gpu(pos.astype(np.int32)) if tokens % 3 == 0 and far < 1 << 31 else gpu(pos.astype(np.int64))
    return rng, q, k, w, pos, freqs, s, (position, gpu(freqs)), None if s is None else gpu(s)


def rel_rows(a, b):
    return np.linalg.norm(a - b, axis=-1) / np.maximum(np.linalg.norm(b, axis=-1), 1e-300)


@pytest.mark.parametrize("case", QK, ids=lambda c: "-".join(map(str, c)))
def test_qk_norm_rope(case):
    say("norm_rope", *case)
    d, pairs, inter, signs, gamma, io, *_ = case
    _, q, k, w, pos, freqs, s, at, sg = qk_case(*case)
    yq, yk = kv4.harp_qk_norm_rope(q, k, *at, **w, eps=1e-5, interleaved=inter, signs=sg)
    for y, x, g in ((yq, q, w["gamma_q"]), (yk, k, w["gamma_k"])):
        if x is None:
            assert y is None
            continue
        want = K.norm_rope(cpu(x), pos, freqs, None if g is None else cpu(g), 1e-5, inter, s)
        assert rel_rows(cpu(y), want).max() <= 2.0 ** -19 + (H if io == "bf16" else 0)
    # in place, and into another layout (heads outside)
    q2 = q.clone()
    k2 = None if k is None else torch.empty(k.shape[1], k.shape[0], d, dtype=k.dtype, device="cuda").transpose(0, 1)
    kv4.harp_qk_norm_rope(q2, k, *at, **w, eps=1e-5, interleaved=inter, signs=sg, q_out=q2, k_out=k2)
    assert torch.equal(q2, yq) and (k is None or torch.equal(k2, yk))


@pytest.mark.parametrize("case", QK, ids=lambda c: "-".join(map(str, c)))
def test_qk_norm_rope_vjp(case):
    say("norm_rope_vjp", *case)
    d, pairs, inter, signs, gamma, io, *_ = case
    rng, q, k, w, pos, freqs, s, at, sg = qk_case(*case, seed=1)
    dyq = gpu(rng.standard_t(3, q.shape).astype(np.float32), q.dtype)
    dyk = None if k is None else gpu(rng.standard_t(3, k.shape).astype(np.float32), k.dtype)
    r = kv4.harp_qk_norm_rope_vjp(q, k, *at, dyq, dyk, **w, eps=1e-5, interleaved=inter, signs=sg, want_dgamma=True)
    for x, g, dy, dx, dg in ((q, w["gamma_q"], dyq, r.dq, r.dgamma_q), (k, w["gamma_k"], dyk, r.dk, r.dgamma_k)):
        if x is None:
            assert dx is None and dg is None
            continue
        want, wg, size, gsize = K.norm_rope_vjp(cpu(x), pos, freqs, None if g is None else cpu(g), 1e-5, inter, s, cpu(dy))
        err = np.linalg.norm(cpu(dx) - want, axis=-1)
        assert (err <= 2.0 ** -18 * size + (H if io == "bf16" else 0) * np.linalg.norm(want, axis=-1)).all()
        assert (np.abs(cpu(dg) - wg) <= 2.0 ** -17 * gsize).all()
    # twice the same bits; in place over the upstream gradients; without dgamma
    r2 = kv4.harp_qk_norm_rope_vjp(q, k, *at, dyq, dyk, **w, eps=1e-5, interleaved=inter, signs=sg, want_dgamma=True)
    assert all(a is b or torch.equal(a, b) for a, b in zip(r, r2))
    r3 = kv4.harp_qk_norm_rope_vjp(q, k, *at, dyq, dyk, **w, eps=1e-5, interleaved=inter, signs=sg, want_dgamma=False, dq=dyq,
                                   dk=dyk)
    assert torch.equal(dyq, r.dq) and (k is None or torch.equal(dyk, r.dk)) and r3.dgamma_q is None


def test_qk_gradient_against_differences_of_the_kernel():
    # the forward kernel in fp32, central differences in fp64 of its outputs: steps of 2^-7 leave 2^-14 of curvature and
    # 2^-19 / 2^-7 of rounding, relative to |dy| |y| = 8; a directional derivative sums 128 of each: 1e-2 is ten times that
    say("differences")
    rng = np.random.default_rng(7)
    x, v, dy = (gpu(rng.standard_normal((1, 1, 128)).astype(np.float32)) for _ in range(3))
    g, s = gpu((1 + 0.1 * rng.standard_normal(128)).astype(np.float32)), gpu(rng.choice([-1, 1], 128).astype(np.int8))
    pos, f = torch.tensor([12], device="cuda"), gpu(10.0 ** (-np.arange(64) / 16.0))
    run = lambda a, w: kv4.harp_qk_norm_rope(a, None, pos, f, w, eps=1e-5, signs=s)[0].double()       # noqa: E731
    r = kv4.harp_qk_norm_rope_vjp(x, None, pos, f, dy, None, g, eps=1e-5, signs=s)
    e = 2.0 ** -7
    num = ((run(x + e * v, g) - run(x - e * v, g)) * dy.double()).sum() / (2 * e)
    assert abs(float(num) - float((r.dq.double() * v.double()).sum())) <= 1e-2
    gv = v[0, 0]
    num = ((run(x, g + e * gv) - run(x, g - e * gv)) * dy.double()).sum() / (2 * e)
    assert abs(float(num) - float((r.dgamma_q.double() * gv.double()).sum())) <= 1e-2


def test_qk_special_heads_stay_alone():
    say("special heads")
    x = torch.randn(4, 6, 128, device="cuda")
    f = gpu(10000.0 ** (-np.arange(64) / 64.0))
    pos = torch.arange(4, device="cuda")
    s = gpu(np.random.default_rng(0).choice([-1, 1], 128).astype(np.int8))
    good, _ = kv4.harp_qk_norm_rope(x, None, pos, f, signs=s)
    y = x.clone()
    y[1, 2, 5] = float("nan")
    y[2, 0, 7] = float("inf")
    y[3, 1] = 0.0
    y[3, 2] *= 1e30                                               # squares beyond fp32's range
    y[3, 3] *= 1e-30
    got, _ = kv4.harp_qk_norm_rope(y, None, pos, f, signs=s, eps=0.0)
    bad = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = bad[3, 1] = True                       # 0 / 0 without eps
    assert torch.isnan(got[bad]).all(-1).all() and torch.isfinite(got[~bad]).all()
    want = K.norm_rope(cpu(y)[3, 2:4][None].repeat(4, 0), np.arange(4), cpu(f), None, 0.0, False, cpu(s))[3]
    assert rel_rows(cpu(got[3, 2:4]), want).max() <= 2.0 ** -19
    other = ~bad
    other[3, 2:4] = False
    # eps is 1e-6 of a mean square near 1 in the first, 0 in the other
    assert ((got - good).abs()[other] <= 2e-6 * good.abs()[other] + 1e-6).all()


def test_qk_no_tokens():
    x = torch.randn(0, 4, 64, device="cuda")
    y, _ = kv4.harp_qk_norm_rope(x, None, torch.zeros(0, dtype=torch.int64, device="cuda"), gpu(np.ones(8)))
    assert y.shape == (0, 4, 64)
    dg = torch.full((64,), 3.0, device="cuda")
    r = kv4.harp_qk_norm_rope_vjp(x, None, None, None, x, None, torch.ones(64, device="cuda"), dgamma_q=dg)
    assert (dg == 0).all() and r.dgamma_q is dg


# ---------------------------------------------------------------------- plans
class Plan:
    """Sequences of `lengths` tokens, of which the call has the last `new`, over
    pages in random order; what is behind a sequence's end is garbage, scales of
    NaN and of the largest values among it."""

    def __init__(self, lengths, new, heads, d, page, seed=0, spare=2, extra_width=1):
        rng = np.random.default_rng(seed)
        self.rng, self.heads, self.d, self.page = rng, heads, d, page
        need = [-(-n // page) for n in lengths]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = rng.integers(-9, 10 ** 9, (len(lengths), max(1, max(need, default=0)) + extra_width))
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lengths = np.array(lengths)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.rows = int(self.starts[-1])

    def fill(self):
        shape = (self.pages, self.heads, self.page, self.d)
        cache = []
        for _ in range(2):
            x = self.rng.standard_normal(shape) * np.exp(0.5 * self.rng.standard_normal((*shape[:3], 1)))
            codes, scales = K.quantize(x)
            cache += [codes, scales]
        for b, n in enumerate(self.lengths):
            if n % self.page:
                last = self.table[b, n // self.page]
                for i in (0, 2):
                    cache[i][last, :, n % self.page:] = 0x77
                    cache[i + 1][last, :, n % self.page:] = self.rng.choice([253, 254, 255], cache[i + 1][last, :, n % self.page:].shape)
        self.cache = cache
        return self

    def on_gpu(self):
        return tuple(gpu(x.astype(np.int32)) for x in (self.starts, self.lengths, self.table))

    def cache_on_gpu(self, side_by_side=False):
        if not side_by_side:
            t = [gpu(c) for c in self.cache]
        else:
            both = torch.stack([gpu(self.cache[0]), gpu(self.cache[2])], 1)       # keys and values of a page in one buffer
            t = [both[:, 0], gpu(self.cache[1]), both[:, 1], gpu(self.cache[3])]
        return kv4.Cache4(t[0], t[1].view(kv4.SCALES), t[2], t[3].view(kv4.SCALES))


WRITE = [  # lengths, new, heads, d, page, io
    ([1], [1], 1, 32, 16, "f32"),
    ([16, 17, 40], [16, 1, 30], 2, 64, 16, "bf16"),
    ([5, 0, 33, 100], [5, 0, 1, 77], 3, 96, 32, "f32"),
    ([300, 7], [300, 7], 8, 128, 64, "bf16"),
    ([64] * 70, [1] * 70, 2, 128, 16, "bf16"),
    (list(range(1, 200)), [1 + i % 3 if i else 1 for i in range(199)], 1, 160, 16, "f32"),
    ([50, 3], [20, 3], 2, 192, 256, "bf16"),
    ([50, 3], [20, 9], 5, 224, 16, "f32"),                        # rows before the beginning
    ([90], [90], 4, 256, 16, "f32"),
]


@pytest.mark.parametrize("case", WRITE, ids=lambda c: f"{len(c[0])}x{c[2]}x{c[3]}-{c[4]}-{c[5]}")
def test_write_and_read(case):
    lengths, new, heads, d, page, io = case
    say("write", len(lengths), heads, d, page, io)
    p = Plan(lengths, new, heads, d, page).fill()
    tokens = p.rows + 3                                           # three rows behind the last sequence
    qkv = gpu((p.rng.standard_normal((tokens, 2 * heads + 1, d)) * np.exp(2 * p.rng.standard_normal((tokens, 2 * heads + 1, 1))))
              .astype(np.float32), IO[io])
    k, v = qkv[:, :heads], qkv[:, heads + 1:]
    cache = p.cache_on_gpu(side_by_side=heads == 2)
    plan = p.on_gpu()
    kv4.harp_kv4_write(k, v, cache, *plan)
    K.write(cpu(k), p.cache[0], p.cache[1], p.starts, p.lengths, p.table)
    K.write(cpu(v), p.cache[2], p.cache[3], p.starts, p.lengths, p.table)
    for got, want in zip(cache, p.cache):                         # the whole of it: nothing else has changed
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    for out in ("f32", "bf16"):
        ko, vo = (torch.full((tokens, heads, d), 7.0, dtype=IO[out], device="cuda") for _ in range(2))
        kv4.harp_kv4_read(cache, *plan, tokens, out, k=ko, v=vo)
        for got, c, s in ((ko, p.cache[0], p.cache[1]), (vo, p.cache[2], p.cache[3])):
            want = np.full((tokens, heads, d), 7.0)
            K.read(c, s, p.starts, p.lengths, p.table, want)
            assert np.array_equal(cpu(got), want, equal_nan=True)


def test_write_special_values():
    say("special values")
    p = Plan([40], [40], 1, 128, 16).fill()
    x = np.random.default_rng(3).standard_normal((40, 1, 128)).astype(np.float32)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 70] = np.nan, np.inf, -np.inf
    x[3] = 0.0
    x[4, 0, :32] = -0.0
    x[5, 0, :32] = np.linspace(-6, 6, 32)
    x[6, 0, :32] = np.arange(32) / 4.0 - 4                       # ties
    x[7] *= np.float32(1e-38)
    x[8] *= np.float32(1e-44)
    x[9, 0, :4] = [3.4e38, 1.0, -2e38, 0.0]
    x[10, 0, :4] = [2.9e38, 1.0, -2e38, 1e38]
    x[11, 0, :2] = [np.float32(1.75 * 2.0 ** 127), 1.0]
    x[12, 0, :2] = [np.nextafter(np.float32(1.75 * 2.0 ** 127), np.float32(0)), 1.0]
    for i in range(13, 40):
        x[i, 0, :8] = np.nextafter(np.float32(6.0 * 2.0 ** (i - 20)), np.float32((-1) ** i * 1e30))
        x[i, 0, 8:32] *= 2.0 ** (i - 20)
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    kv4.harp_kv4_write(gpu(x), gpu(-x), cache, *plan)
    K.write(x.astype(np.float64), p.cache[0], p.cache[1], p.starts, p.lengths, p.table)
    K.write(-x.astype(np.float64), p.cache[2], p.cache[3], p.starts, p.lengths, p.table)
    for got, want in zip(cache, p.cache):
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    ko, vo = kv4.harp_kv4_read(cache, *plan, 40, "f32")
    want = np.zeros((40, 1, 128))
    K.read(p.cache[0], p.cache[1], p.starts, p.lengths, p.table, want)
    assert np.array_equal(cpu(ko), want, equal_nan=True)
    assert np.isnan(want[0, 0, :32]).all() and np.isfinite(want[0, 0, 32:]).all() and np.isnan(want[9, 0, :32]).all()


def test_pages_that_are_not_there():
    say("bad pages")
    p = Plan([100, 60], [100, 60], 2, 64, 16, extra_width=0).fill()
    p.table[0, 2], p.table[0, 3], p.table[1, 0] = -1, p.pages, 1 << 30
    p.table = p.table[:, :5]                                      # tokens 80 to 99 of the first are beyond the table
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    x = gpu(p.rng.standard_normal((160, 2, 64)).astype(np.float32))
    kv4.harp_kv4_write(x, x, cache, *plan)
    K.write(cpu(x), p.cache[0], p.cache[1], p.starts, p.lengths, p.table)
    K.write(cpu(x), p.cache[2], p.cache[3], p.starts, p.lengths, p.table)
    for got, want in zip(cache, p.cache):
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    ko, _ = kv4.harp_kv4_read(cache, *plan, 160, "f32")
    want = np.zeros((160, 2, 64))
    K.read(p.cache[0], p.cache[1], p.starts, p.lengths, p.table, want)
    assert np.array_equal(cpu(ko), want, equal_nan=True) and np.isnan(want).any()
    # attention: rows that see such a place are NaN, the others are not
    q = gpu(p.rng.standard_normal((160, 4, 64)).astype(np.float32), BF)
    for window in (0, 10):
        out, lse = kv4.harp_kv4_attention(q, cache, *plan, window=window, lse=True)
        check_attention(p, q, out, lse, 1 / 8.0, True, window)


# ------------------------------------------------------------------ attention
def check_attention(p, q, out, lse, scale, causal, window):
    want, wl, size, score = K.attention(cpu(q), p.cache, p.starts, p.lengths, p.table, scale, causal, window)
    got, gl = cpu(out)[:p.rows], cpu(lse)[:p.rows]
    want, wl, size, score = want[:p.rows], wl[:p.rows], size[:p.rows], score[:p.rows]
    assert (np.isnan(got) == np.isnan(want)).all()
    dz = (p.d * U + 3 * U) * score
    tol = (2 * dz[..., None] + H + 2.0 ** -19) * size + H * np.abs(want) + 2.0 ** -107
    bad = np.abs(got - want) > tol
    assert not bad.sum(), (np.argwhere(bad)[:5], np.abs(got - want)[bad][:5], tol[bad][:5])
    none = wl == -np.inf
    assert ((gl == -np.inf) == none).all() and (got[none] == 0).all()
    fine = ~none & ~np.isnan(wl)
    assert (np.isnan(gl) == np.isnan(wl)).all()
    assert (np.abs(gl - wl)[fine] <= (dz + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl))[fine]).all()


ATTENTION = [  # lengths, new, q heads, heads, d, page, causal, window, scale
    ([1], [1], 1, 1, 32, 16, True, 0, None),
    ([33], [1], 4, 1, 64, 16, True, 0, None),
    ([100, 0, 257, 16], [1, 1, 1, 1], 8, 2, 128, 16, True, 0, None),
    ([4097], [1], 32, 8, 128, 64, True, 0, None),
    ([500, 31, 32, 33, 129], [3, 3, 3, 3, 3], 24, 4, 96, 32, True, 100, None),
    ([70, 200], [1, 1], 5, 1, 160, 16, True, 0, 0.2),
    ([70, 200, 1], [1, 2, 1], 6, 3, 192, 32, True, 0, None),
    ([130, 5], [2, 2], 8, 2, 224, 16, True, 0, None),
    ([300, 40], [1, 4], 16, 2, 256, 16, True, 0, None),
    ([90, 3, 64], [90, 3, 64], 6, 2, 128, 16, True, 0, None),
    ([400], [130], 4, 1, 128, 64, True, 0, None),
    ([400, 350], [130, 7], 8, 4, 64, 16, True, 50, None),
    ([150, 80], [100, 80], 4, 2, 96, 16, False, 0, None),
    ([150], [40], 4, 2, 32, 16, False, 60, None),
    ([20, 40], [33, 12], 4, 2, 128, 16, True, 0, None),            # rows before the beginning
    ([260], [200], 3, 3, 256, 16, True, 0, None),
    ([120, 500], [70, 90], 2, 1, 192, 64, True, 33, None),
    ([200, 90], [110, 90], 3, 1, 160, 16, True, 0, None),
    ([180], [100], 2, 2, 224, 32, True, 75, None),
    ([700, 20], [300, 20], 8, 2, 128, 16, True, 0, 0.5),
    ([64] * 130, [1] * 130, 2, 1, 64, 16, True, 0, None),
    ([1000], [1], 64, 1, 128, 16, True, 0, None),
    # many sequences, some without a token, of very different lengths
    ([(37 * i) % 190 for i in range(200)], [(1, 0, 2, 1)[i % 4] for i in range(200)], 2, 1, 64, 16, True, 0, None),
    ([2500, 0, 1900, 64, 3100], [1, 0, 1, 1, 2], 8, 8, 96, 16, True, 0, None),
    ([1500 if i == 70 else 5 for i in range(90)], [1] * 90, 4, 2, 128, 32, True, 0, None),
    # more tiles and heads than a chip has room for
    ([1 + (23 * i) % 37 for i in range(69)], [i % 3 for i in range(69)], 32, 32, 256, 16, True, 0, None),
    ([15 + (17 * i) % 30 for i in range(33)], [20] * 33, 32, 32, 192, 32, True, 19, None),
]


def run_attention(case, seed=0, side_by_side=False, **kw):
    lengths, new, hq, heads, d, page, causal, window, scale = case
    p = Plan(lengths, new, heads, d, page, seed).fill()
    tokens = p.rows + 2
    buf = gpu(p.rng.standard_normal((tokens, hq + 1, d)).astype(np.float32), BF)
    q = buf[:, :hq]
    out = torch.full((tokens, hq, d), 9.0, dtype=BF, device="cuda")
    lse = torch.full((tokens, hq), 9.0, device="cuda")
    cache = p.cache_on_gpu(side_by_side)
    plan = p.on_gpu()
    r = kv4.harp_kv4_attention(q, cache, *plan, scale=scale, causal=causal, window=window, out=out, lse=lse, **kw)
    assert r[0] is out and r[1] is lse
    return p, q, cache, plan, out, lse, scale or 1 / math.sqrt(d)


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: f"{len(c[0])}x{c[1][0]}-{c[0][0]}-{c[2]}/{c[3]}x{c[4]}-{c[5]}-{c[7]}")
def test_attention(case):
    say("attention", *case[2:], "sequences", len(case[0]), "first", case[0][0], case[1][0])
    p, q, cache, plan, out, lse, scale = run_attention(case, side_by_side=case[3] == 2)
    check_attention(p, q, out, lse, scale, case[6], case[7])
    assert (out[p.rows:] == 9).all() and (lse[p.rows:] == 9).all()
    # the same bits again, into another layout and without lse
    o2 = torch.empty(case[2], out.shape[0], case[4], dtype=BF, device="cuda").transpose(0, 1)
    kv4.harp_kv4_attention(q, cache, *plan, scale=scale, causal=case[6], window=case[7], out=o2)
    assert torch.equal(o2[:p.rows], out[:p.rows])


@pytest.mark.parametrize("hq,new", [(2, [1, 1]), (4, [60, 33]), (32, [1, 4])])
def test_nan_keys_and_values_reach_only_rows_that_see_them(hq, new):
    say("NaN", hq, new)
    p = Plan([200, 77], new, 2, 128, 16, seed=5).fill()
    for b, j, h, blk, side in ((0, 150, 0, 2, 1), (0, 190, 1, 0, 3), (0, 199, 0, 3, 3), (1, 50, 1, 1, 3), (1, 75, 0, 0, 1), (0, 3, 0, 1, 3)):
        p.cache[side][p.table[b, j // 16], h, j % 16, blk] = 255
    q = gpu(p.rng.standard_normal((p.rows, hq, 128)).astype(np.float32), BF)
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    for window in (0, 40):
        out, lse = kv4.harp_kv4_attention(q, cache, *plan, window=window, lse=True)
        check_attention(p, q, out, lse, 128 ** -0.5, True, window)


def test_special_queries_stay_alone():
    say("special queries")
    p = Plan([100], [20], 1, 64, 16, seed=6).fill()
    x = p.rng.standard_normal((20, 4, 64)).astype(np.float32)
    good = kv4.harp_kv4_attention(gpu(x, BF), p.cache_on_gpu(), *p.on_gpu())
    x[3, 1, 5], x[7, 2, 9] = np.nan, np.inf
    x[9, 0] = 0
    x[11, 3] *= 1000.0                                            # weights all but one hot
    q = gpu(x, BF)
    out, lse = kv4.harp_kv4_attention(q, p.cache_on_gpu(), *p.on_gpu(), lse=True)
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[7, 2]).all()
    same = torch.ones(20, 4, dtype=torch.bool, device="cuda")
    same[3, 1] = same[7, 2] = same[9, 0] = same[11, 3] = False
    assert torch.equal(out[same], good[same])
    x[3, 1], x[7, 2] = 0.5, -0.5
    out, lse = kv4.harp_kv4_attention(gpu(x, BF), p.cache_on_gpu(), *p.on_gpu(), lse=True)
    check_attention(p, gpu(x, BF), out, lse, 0.125, True, 0)


def test_plans_that_make_no_sense_stay_within_bounds():
    # the host's checks cannot see these; the kernels keep to the arrays (shown by their index checks), whatever comes out
    say("senseless plans")
    p = Plan([100, 60], [5, 5], 2, 64, 16).fill()
    cache = p.cache_on_gpu()
    q = torch.randn(10, 4, 64, device="cuda").to(BF)
    x = torch.randn(10, 2, 64, device="cuda")
    for starts, lengths in (([0, 9, 3], [100, 60]), ([-5, 4, 90], [100, 60]), ([3, 5, 10], [-7, 60]), ([0, 0, 0], [3, 3]),
                            ([0, 5, 10], [500, 400])):
        plan = (torch.tensor(starts, dtype=torch.int32, device="cuda"), torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                p.on_gpu()[2])
        out = kv4.harp_kv4_attention(q, cache, *plan)
        k, v = kv4.harp_kv4_read(cache, *plan, 10)
        kv4.harp_kv4_write(x, x, cache, *plan)
        torch.cuda.synchronize()
        assert out.shape == q.shape and k.shape == x.shape


def test_a_plan_that_gives_rows_to_many_sequences_ends():
    say("rows of many sequences")
    p = Plan([90] * 300, [1] * 300, 2, 64, 16).fill()
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    starts = torch.tensor([0, 300] * 150 + [250], dtype=torch.int32, device="cuda")
    buf = torch.full((302, 4, 64), 7.0, dtype=BF, device="cuda")
    q = torch.randn(300, 4, 64, device="cuda").to(BF)
    kv4.harp_kv4_attention(q, cache, starts, *plan[1:], out=buf[1:301])
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[301] == 7).all()


@pytest.mark.parametrize("lengths,new,heads,d", [([300, 40, 5], [1, 1, 1], 2, 128), ([300, 40, 5], [6, 6, 6], 2, 96),
                                                 ([400], [100], 1, 64)])
def test_a_workspace_is_used_up_to_its_size(lengths, new, heads, d):
    p = Plan(lengths, new, heads, d, 16).fill()
    q = gpu(p.rng.standard_normal((p.rows, 4, d)).astype(np.float32), BF)
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    need = kv4.harp_kv4_attention_workspace(p.rows, 4, heads, d, 16, len(lengths), plan[2].shape[1])
    assert need > 0
    buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    out, lse = kv4.harp_kv4_attention(q, cache, *plan, lse=True, workspace=buf[256:256 + need])
    assert (buf[:256] == 0x5a).all() and (buf[256 + need:] == 0x5a).all()
    check_attention(p, q, out, lse, 1 / math.sqrt(d), True, 0)
    with pytest.raises(Exception, match="workspace"):
        kv4.harp_kv4_attention(q, cache, *plan, workspace=buf[256:256 + need - 1])


def test_no_sequences_and_no_tokens():
    c = kv4.harp_kv4_cache(3, 2, 16, 64)
    none = (torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
            torch.zeros(0, 4, dtype=torch.int32, device="cuda"))
    out = torch.full((3, 4, 64), 5.0, dtype=BF, device="cuda")
    kv4.harp_kv4_attention(out.clone(), c, *none, out=out)
    assert (out == 5).all()
    p = Plan([20], [0], 2, 64, 16).fill()
    assert kv4.harp_kv4_attention(torch.zeros(0, 4, 64, dtype=BF, device="cuda"), p.cache_on_gpu(), *p.on_gpu()).shape == (0, 4, 64)
    assert kv4.harp_kv4_read(p.cache_on_gpu(), *p.on_gpu(), 0)[0].shape == (0, 2, 64)


# -------------------------------------------------------------- run together
def test_rotated_step_by_step_is_the_prompt_at_once():
    """A prompt's heads are normed, turned and rotated, written and attended; the
    same prompt token by token gives the same cache and the same rows within
    the results' rounding; and the rotation leaves scores as they are."""
    say("together")
    rng = np.random.default_rng(11)
    hq, hk, d, n, page = 8, 2, 128, 75, 16
    qkv = gpu(rng.standard_t(3, (n, hq + 2 * hk, d)).astype(np.float32), BF)
    g, s = gpu((1 + 0.2 * rng.standard_normal(d)).astype(np.float32), BF), gpu(rng.choice([-1, 1], d).astype(np.int8))
    f = gpu(10000.0 ** (-np.arange(64) / 64.0))
    table = torch.tensor([[3, 0, 4, 1, 2]], dtype=torch.int32, device="cuda")

    def step(cache, t0, t1):
        part = qkv[t0:t1]
        q, k = kv4.harp_qk_norm_rope(part[:, :hq], part[:, hq:hq + hk], torch.arange(t0, t1, device="cuda"), f, g, g, signs=s)
        v = rht_compose((8, 16), d, s[None], part[:, hq + hk:].reshape(-1, d)).view(t1 - t0, hk, d)
        plan = (torch.tensor([0, t1 - t0], dtype=torch.int32, device="cuda"), torch.tensor([t1], dtype=torch.int32, device="cuda"), table)
        kv4.harp_kv4_write(k, v, cache, *plan)
        return q, kv4.harp_kv4_attention(q, cache, *plan), plan

    once, bits = kv4.harp_kv4_cache(5, hk, page, d), kv4.harp_kv4_cache(5, hk, page, d)
    q, out, plan = step(once, 0, n)
    rows = [step(bits, t, t + 1)[1] for t in range(n)]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(once, bits))
    k, v = (cpu(x) for x in kv4.harp_kv4_read(once, *plan, n, "f32"))
    want, _, size, score = K.attention(cpu(q), [x.view(torch.uint8).cpu().numpy() for x in once], [0, n], [n], table.cpu().numpy(), d ** -0.5)
    tol = (2 * (d + 3) * U * score[..., None] + H + 2.0 ** -19) * size + H * np.abs(want)
    assert (np.abs(cpu(out) - want) <= tol).all() and (np.abs(cpu(torch.cat(rows)) - want) <= tol).all()
    # the rotation turned back: the heads as they were, within their rounding; the values within a code's, a quarter of
    # the value from the scale s on and s / 4 below
    plain = K.norm_rope(cpu(qkv[:, :hq]), np.arange(n), cpu(f), cpu(g), 1e-6, False, None)
    turned = cpu(q) @ K.hadamard(d) * cpu(s)
    assert rel_rows(turned, plain).max() <= 2.0 ** -18 + H
    values = cpu(qkv[:, hq + hk:])
    most = 2.0 ** (once.v_scales.view(torch.uint8).cpu().numpy().max() - 127.0)
    assert np.linalg.norm(v @ K.hadamard(d) * cpu(s) - values) <= \
        (0.25 + 2 * H) * np.linalg.norm(values) + 0.25 * most * math.sqrt(values.size)


def test_captured_and_replayed():
    """All operators in one graph; the plan's arrays, the queries and the cache
    change between replays, with eager work between them."""
    say("graph")
    p = Plan([300, 40], [1, 1], 2, 128, 16, seed=8, spare=8, extra_width=0).fill()
    cache, plan = p.cache_on_gpu(), p.on_gpu()
    rng = np.random.default_rng(9)
    qkv = gpu(rng.standard_normal((2, 12, 128)).astype(np.float32), BF)
    g = gpu((1 + 0.2 * rng.standard_normal(128)).astype(np.float32), BF)
    f, pos = gpu(10000.0 ** (-np.arange(64) / 64.0)), torch.tensor([299, 39], device="cuda")
    s = gpu(rng.choice([-1, 1], 128).astype(np.int8))
    ws = torch.empty(max(16, kv4.harp_kv4_attention_workspace(2, 8, 2, 128, 16, 2, plan[2].shape[1])), dtype=torch.uint8, device="cuda")

    def step(c):
        q, k = kv4.harp_qk_norm_rope(qkv[:, :8], qkv[:, 8:10], pos, f, g, g, signs=s)
        grads = kv4.harp_qk_norm_rope_vjp(qkv[:, :8], qkv[:, 8:10], pos, f, q, k, g, g, signs=s)
        kv4.harp_kv4_write(k, qkv[:, 10:], c, *plan)
        out, lse = kv4.harp_kv4_attention(q, c, *plan, lse=True, workspace=ws)
        return [q, k, *grads, out, lse, *kv4.harp_kv4_read(c, *plan, 2)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(kv4.Cache4(*(t.clone() for t in cache)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step(cache)
    for i in range(4):
        torch.cuda.synchronize()
        qkv.copy_(gpu(rng.standard_normal((2, 12, 128)).astype(np.float32), BF))
        plan[1].copy_(torch.tensor([300 - 20 * i, 40 - i], dtype=torch.int32))
        pos.copy_(torch.tensor([299 - 20 * i, 39 - i]))
        copy = kv4.Cache4(*(t.clone() for t in cache))
        want = step(copy)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
        for a, b in zip(cache, copy):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_another_stream_and_dropped_tensors():
    say("streams")
    case = ATTENTION[3]
    p, q, cache, plan, out, lse, scale = run_attention(case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kv4.harp_kv4_attention(q, cache, *plan, stream=side)
    del q, cache, plan
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[:p.rows], out[:p.rows]) and len(junk) == 8


def test_far_places_of_a_large_cache():
    """Pages beyond 2^31 bytes, and a sequence in them."""
    say("far pages")
    heads, d, page = 8, 256, 1024
    pages = (5 << 30) // (heads * page * d // 2)                  # 5 GiB of codes on each side
    c = kv4.harp_kv4_cache(pages, heads, page, d)
    n = page + 40
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    starts, lengths = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(10)
    x = gpu(rng.standard_normal((n, 2 * heads, d)).astype(np.float32), BF)
    kv4.harp_kv4_write(x[:, :heads], x[:, heads:], c, starts, lengths, table)
    k, v = kv4.harp_kv4_read(c, starts, lengths, table, n, "f32")
    for got, want in ((k, x[:, :heads]), (v, x[:, heads:])):
        rows = [0, 1, page - 1, page, n - 1]
        assert np.array_equal(cpu(got[rows]), K.dequantize(*K.quantize(cpu(want[rows]))))
    q = x[n - 1:, :heads].contiguous()
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out, lse = kv4.harp_kv4_attention(q, c, one, lengths, table, lse=True)
    kk, vv = cpu(k), cpu(v)
    for h in (0, heads - 1):
        want, wl, size, score = K.attend(cpu(q)[:, h], kk[:, h], vv[:, h], d ** -0.5, np.ones((1, n), bool))
        dz = (d + 3) * U * score[0]
        assert (np.abs(cpu(out)[0, h] - want[0]) <= (2 * dz + H + 2.0 ** -19) * size[0] + H * np.abs(want[0])).all()
        assert abs(float(lse[0, h]) - wl[0]) <= dz + 2.0 ** -20 + 2.0 ** -22 * abs(wl[0])
