"""What attention over a 4-bit cache and its heads compute, where a little less
would not be seen in ordinary values: weights of one dominant key, angles of far
positions, heads at the ends of fp32's range, gradients next to others that are not
numbers, and every code with every scale.

Tolerances.  u = 2^-24 and h = 2^-8 are the largest relative errors of one
rounding to fp32 and to bf16; half a step of bf16 at x is 2^(floor(log2 |x|) - 8).
Each test says how its own follows from them.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as K
from structured_rotations_amd import kv4

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U, H = 2.0 ** -24, 2.0 ** -8


def cpu(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def say(*a):
    print("\n[case]", *a, flush=True)


def half_step(x):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -120))) - 8)


# ------------------------------------------------------------------- weights
@pytest.mark.parametrize("tokens,heads", [(1, 16), (1, 48), (4, 64)], ids=["tiles of 16", "tiles of 32", "tiles of 128"])
def test_a_key_that_outweighs_the_others_and_comes_late(tokens, heads):
    """Two keys of score 0, then one a few units above: the reference that its
    weight goes by is theirs, and the result is its value to within the result's
    rounding.

    Scores here are exact: at most two products of few bits each.  A result is
    off by half its step; by 2^-19 of `size`, the weighted mean of |v|, for the
    exponentials, sums and divisions; in tiles of 16 rows by 2^-16 of `size`, the
    weights having 16 bits; in larger ones by h (1 + 2^-7) of `spread`, the
    weighted mean of |v - result|, the weights having 8 and their sum being that
    of the rounded ones."""
    say("late peak", tokens, heads)
    n, d = 1024, 64
    kc, vc = np.zeros((n, d // 2), np.uint8), np.zeros((n, d // 2), np.uint8)
    kc[:, 0] = 0x0f << 4                                     # all keys: 0, -6 in columns 0 and 1
    kc[[69, 133], 0], kc[199, 0] = 0x00, 0x02                # two early ones: 0, 0; the late one: 1, 0
    rng = np.random.default_rng(0)
    vc[:] = rng.integers(0, 256, (n, d // 2))
    vc[[69, 133]] = rng.integers(0, 2, (2, d // 2)) * 0x99   # 0 or -0.5
    vc[199] = rng.choice([0x33, 0x35, 0x57, 0x62], d // 2)   # 1.5, 3, 4, 6, 1
    pages = rng.permutation(n // 64)
    cache = []
    for c in (kc, vc):
        codes, scales = np.zeros((n // 64, 1, 64, d // 2), np.uint8), np.full((n // 64, 1, 64, d // 32), 127, np.uint8)
        codes[pages, 0] = c.reshape(-1, 64, d // 2)
        cache += [codes, scales]
    q = np.zeros((tokens, heads, d), np.float32)
    q[..., 0] = rng.uniform(0.5, 5.4, (tokens, heads))       # up to 7.8 powers of two above
    q[..., 1] = 6.0
    q = gpu(q, BF)
    plan = [np.array([0, tokens]), np.array([n]), pages[None]]
    out, lse = kv4.harp_kv4_attention(q, kv4.Cache4(*(gpu(c) if i % 2 == 0 else gpu(c).view(kv4.SCALES) for i, c in enumerate(cache))),
                                      *(gpu(x.astype(np.int32)) for x in plan), scale=1.0, lse=True)
    k, v = (K.sequence(cache[i], cache[i + 1], pages, n)[0] for i in (0, 2))
    z = cpu(q) @ k.T                                         # every key is in front of every row
    w = np.exp(z - z.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    want = w @ v
    size = w @ np.abs(v)
    if tokens * heads <= 16:
        tol = 2.0 ** -16 * size
    else:
        tol = np.stack([np.stack([w[i, j] @ np.abs(v - want[i, j]) for j in range(heads)]) for i in range(tokens)]) * (H * (1 + 2.0 ** -7))
    err = np.abs(cpu(out) - want)
    assert (err <= half_step(np.abs(want) + tol) + tol + 2.0 ** -19 * size).all(), (err / size).max()
    wl = np.log(np.exp(z).sum(-1))
    assert (np.abs(cpu(lse) - wl) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(wl)).all()


# -------------------------------------------------------------------- angles
def _turns_of_a_radian(bits=400):
    """1 / (2 pi) as a fraction, pi by Machin's formula."""
    one = 1 << bits

    def arctan(x):
        total, term, n = 0, one // x, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total
    return Fraction(one, 8 * (4 * arctan(5) - arctan(239)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_angles_of_far_positions(wide, interleaved):
    """Positions next to the ends of their range and frequencies up to 8, against
    angles reduced exactly.  A pair that is alone in its head: its square and root
    6 u, products 3 u, cosine and sine 4 u off each and rounded once more, over the
    pair 7 u: 2^-20 of the norm.  Whole heads 2^-19."""
    say("far angles", wide, interleaved)
    rng = np.random.default_rng(int(wide) + 2 * int(interleaved))
    d, n = 48, 64
    # three whose products with the rounded 1 / (2 pi) are far off, and others of all sizes
    freqs = np.concatenate([[float.fromhex(x) for x in ("0x1.c349b066fca73p+2", "0x1.f2a18f4e1c580p+2", "0x1.c75b84f6199a9p+2")],
                            rng.uniform(4, 8, 9), rng.uniform(1, 2, 6), 10.0 ** rng.uniform(-5, 0, 6)])
    far = 2 ** 31 if wide else 2 ** 31 - 1
    pos = np.concatenate([[far, -2 ** 31, far - 1, 0, 1], rng.integers(2 ** 31 - 5000, 2 ** 31, n - 25), -rng.integers(2 ** 30, 2 ** 31, 20)])
    x = rng.standard_normal((n, 2, d)).astype(np.float32)
    x[:, 1] = 0                                              # one pair alone in the second head
    x[np.arange(n), 1, np.arange(n) % 24 * (2 if interleaved else 1)] = 1.0
    y, _ = kv4.harp_qk_norm_rope(gpu(x), None, gpu(pos.astype(np.int64 if wide else np.int32)), gpu(freqs), eps=0.0,
                                 interleaved=interleaved)
    turn = _turns_of_a_radian()
    parts = [[Fraction(int(p)) * Fraction(float(f)) * turn for f in freqs] for p in pos]
    angle = np.array([[2 * math.pi * float(t - round(t)) for t in row] for row in parts])[:, None]
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 24), slice(24, 48))
    u = x.astype(np.float64)
    u /= np.sqrt((u * u).mean(-1, keepdims=True))
    want = np.zeros_like(u)
    want[..., a] = u[..., a] * np.cos(angle) - u[..., b] * np.sin(angle)
    want[..., b] = u[..., a] * np.sin(angle) + u[..., b] * np.cos(angle)
    err = np.linalg.norm(cpu(y) - want, axis=-1) / math.sqrt(d)
    assert err[:, 0].max() <= 2.0 ** -19 and err[:, 1].max() <= 2.0 ** -20, err.max(0)


# --------------------------------------------------------- the ends of a range
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256, 512, 80])
def test_heads_of_the_smallest_and_largest_values(d, io):
    """Norms do not depend on a head's size, without eps: 2^-19 of the norm as
    for any head, a bf16 result h more.  Gradients in the head's own size:
    2^-18 of r |g|, and of a bf16 result h of itself."""
    say("ends of the range", d, io)
    rng = np.random.default_rng(d)
    sizes = np.array([-148, -140, -133, -128, -126, -120, -100, -60, -39, 0, 40, 63, 64, 100, 120, 124], np.float64)
    x = np.clip(rng.standard_normal((len(sizes), 3, d)), -4, 4) * 2.0 ** sizes[:, None, None]
    x = gpu(x.astype(np.float32), {"f32": torch.float32, "bf16": BF}[io])
    x[:2, :, 0] = 2.0 ** -133                                # no head of zeros only: bf16 holds nothing smaller
    x[-1, 0, :] = 3.0e38
    signs = gpu(rng.choice([-1, 1], d).astype(np.int8)) if d != 80 else None
    s = None if signs is None else cpu(signs)
    y, _ = kv4.harp_qk_norm_rope(x, None, None, None, eps=0.0, signs=signs)
    # in units of the head's largest value, so that the oracle's squares stay finite
    top = np.abs(cpu(x)).max(-1, keepdims=True)
    zero, none = np.zeros(len(sizes)), np.zeros(0)
    want = K.norm_rope(cpu(x) / top, zero, none, None, 0.0, False, s)
    err = np.linalg.norm(cpu(y) - want, axis=-1) / math.sqrt(d)
    assert err.max() <= 2.0 ** -19 + (H if io == "bf16" else 0), err.max(-1)
    dy = rng.standard_normal(x.shape) * np.clip(top, 2.0 ** -60, 2.0 ** 60)
    dy = gpu(dy.astype(np.float32), x.dtype)
    r = kv4.harp_qk_norm_rope_vjp(x, None, None, None, dy, None, eps=0.0, signs=signs, want_dgamma=True)
    dx, dgamma, size, gsize = K.norm_rope_vjp(cpu(x) / top, zero, none, None, 0.0, False, s, cpu(dy))
    keep = (size / top[..., 0] < 2.0 ** 126) & (size / top[..., 0] > 2.0 ** -100)        # what fp32 and bf16 hold
    assert keep.sum() > keep.size / 2
    err = np.linalg.norm(cpu(r.dq) * top - dx, axis=-1)
    assert (err <= 2.0 ** -18 * size + (H * np.linalg.norm(dx, axis=-1) if io == "bf16" else 0))[keep].all()
    assert (np.abs(cpu(r.dgamma_q) - dgamma) <= 2.0 ** -17 * gsize).all()


# ----------------------------------------------------- gradients side by side
@pytest.mark.parametrize("hq,hk,d", [(3, 2, 128), (1, 1, 64), (5, 3, 80), (2, 1, 256)])
def test_gradients_that_are_not_numbers_stay_with_their_own_gamma(hq, hk, d):
    """Queries and keys share a wave, not a sum."""
    say("NaN gradients", hq, hk, d)
    rng = np.random.default_rng(d)
    n = 9
    q, k, dq, dk = (gpu(rng.standard_normal((n, h, d)).astype(np.float32)) for h in (hq, hk, hq, hk))
    pos, f = torch.arange(n, device="cuda"), gpu(10000.0 ** (-np.arange(8) / 8.0))
    g = torch.ones(d, device="cuda")
    good = kv4.harp_qk_norm_rope_vjp(q, k, pos, f, dq, dk, g, g)
    bad_q, bad_k = dq.clone(), dk.clone()
    bad_q[4, 0, 20], bad_k[2, hk - 1, 20], bad_k[3, 0, 30] = float("inf"), float("nan"), float("-inf")
    r = kv4.harp_qk_norm_rope_vjp(q, k, pos, f, dq, bad_k, g, g)
    assert torch.equal(r.dgamma_q, good.dgamma_q) and torch.equal(r.dq, good.dq)
    assert torch.isnan(r.dgamma_k[20]) and not torch.isfinite(r.dgamma_k[30])
    r = kv4.harp_qk_norm_rope_vjp(q, k, pos, f, bad_q, dk, g, g)
    assert torch.equal(r.dgamma_k, good.dgamma_k) and torch.equal(r.dk, good.dk) and not torch.isfinite(r.dgamma_q[20])


# ----------------------------------------------------------------- the format
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_code_and_scale_is_read_as_it_stands(out):
    """All pairs of codes with all scales, also those that a cache written here
    does not hold: exact where the type holds the value, infinite beyond it."""
    say("all codes", out)
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    codes = np.ascontiguousarray(np.broadcast_to(codes[None, :, None], (16, 16, 16, 16)))          # page, head, place, byte
    scales = np.arange(256, dtype=np.uint8).reshape(16, 1, 16, 1).repeat(16, 1)
    cache = kv4.Cache4(gpu(codes), gpu(scales).view(kv4.SCALES), gpu(codes), gpu(scales).view(kv4.SCALES))
    plan = ([0, 256], [256], [list(range(16))])
    k, v = kv4.harp_kv4_read(cache, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in plan), 256, out)
    want = K.sequence(codes, scales, np.arange(16), 256).transpose(1, 0, 2)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(cpu(k), want, equal_nan=True) and np.array_equal(cpu(v), want, equal_nan=True)
