"""fp64 numpy oracle of attention over a 4-bit cache: heads normed, turned and
rotated (with the gradients), 32-value blocks of E2M1 codes, a paged cache, and
softmax attention.  Written from the formulas, sequence by sequence and block
by block; it shares nothing with the kernels.
"""
from __future__ import annotations

import numpy as np

BLK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([E2M1, -E2M1])           # of the 16 codes
FLOOR = 7                                        # smallest scale byte, 2^-120
NAN = 255


# ------------------------------------------------------------------- blocks
def scale_byte(block) -> int:
    """The E8M0 byte of 32 values."""
    top = float(np.max(np.abs(block)))
    if not top < 1.75 * 2.0 ** 127:              # NaN and infinities too
        return NAN
    e = FLOOR
    while 6.0 * 2.0 ** (e - 127) < top:
        e += 1
    return e


def encode(v):
    """Codes of values that are at most 6 in magnitude: the nearest of the 8,
    ties to the even code; the sign is kept."""
    a = np.abs(v)[..., None]
    dist = np.abs(a - E2M1)
    best = dist == dist.min(-1, keepdims=True)
    even = best & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), best.argmax(-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantize(x):
    """x (..., d): packed codes (..., d / 2) and scale bytes (..., d / 32)."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    rows = x.reshape(-1, d)
    codes = np.zeros((len(rows), d), dtype=np.uint8)
    scales = np.zeros((len(rows), d // BLK), dtype=np.uint8)
    for i, row in enumerate(rows):
        for b in range(d // BLK):
            part = row[b * BLK:(b + 1) * BLK]
            scales[i, b] = e = scale_byte(part)
            if e != NAN:
                codes[i, b * BLK:(b + 1) * BLK] = encode(part / 2.0 ** (e - 127.0))
    packed = codes[:, 0::2] | codes[:, 1::2] << 4
    return packed.reshape(*x.shape[:-1], d // 2), scales.reshape(*x.shape[:-1], d // BLK)


def dequantize(codes, scales):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = np.where(scales == NAN, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return VALUES[c] * np.repeat(s, BLK, -1)


# -------------------------------------------------------------- paged cache
def places(starts, lengths, table, page_size, pages, tokens):
    """Of each of the call's rows: None (behind the last sequence), "before"
    (its sequence's beginning), "nowhere" (no page), or (page, place in it)."""
    out = [None] * tokens
    for b in range(len(lengths)):
        for r in range(starts[b], starts[b + 1]):
            pos = int(lengths[b]) - (int(starts[b + 1]) - r)
            if pos < 0:
                out[r] = "before"
                continue
            i = pos // page_size
            page = int(table[b][i]) if i < len(table[b]) else -1
            out[r] = (page, pos % page_size) if 0 <= page < pages else "nowhere"
    return out


def write(x, codes, scales, starts, lengths, table):
    """Puts x (tokens x heads x d) into codes and scales (pages x heads x
    page_size x ...), in place."""
    for r, at in enumerate(places(starts, lengths, table, codes.shape[2], codes.shape[0], len(x))):
        if isinstance(at, tuple):
            codes[at[0], :, at[1]], scales[at[0], :, at[1]] = quantize(x[r])


def read(codes, scales, starts, lengths, table, out):
    """Fills out (tokens x heads x d) from the cache, in place."""
    for r, at in enumerate(places(starts, lengths, table, codes.shape[2], codes.shape[0], len(out))):
        if at == "before":
            out[r] = 0.0
        elif at == "nowhere":
            out[r] = np.nan
        elif at is not None:
            out[r] = dequantize(codes[at[0], :, at[1]], scales[at[0], :, at[1]])


def sequence(codes, scales, table, length):
    """The first `length` tokens of a sequence (heads x length x d), NaN where
    there is no page."""
    pages, heads, ps = codes.shape[:3]
    d = codes.shape[3] * 2
    out = np.full((heads, length, d), np.nan)
    for i in range(0, length, ps):
        page = int(table[i // ps]) if i // ps < len(table) else -1
        n = min(ps, length - i)
        if 0 <= page < pages:
            out[:, i:i + n] = dequantize(codes[page, :, :n], scales[page, :, :n])
    return out


# ---------------------------------------------------------------- attention
def attend(q, k, v, scale, sees):
    """One head: q n x d, k and v m x d, sees n x m.  Returns the results, ln of
    the sums, the sums of weights times |v| over the sums of weights, and the
    largest sum of |q| |k| scale over the keys seen (what the errors of fp32
    arithmetic go by)."""
    n, d = q.shape
    out, lse = np.zeros((n, d)), np.full(n, -np.inf)
    size, score = np.zeros((n, d)), np.zeros(n)
    for i in range(n):
        j = np.nonzero(sees[i])[0]
        if len(j) == 0:
            continue
        with np.errstate(invalid="ignore"):
            z = scale * (k[j] @ q[i])
            top = z.max() if not np.isnan(z).any() else np.nan
            w = np.exp(z - top)
            out[i] = (w @ v[j]) / w.sum()
            lse[i] = top + np.log(w.sum())
            size[i] = (w @ np.abs(v[j])) / w.sum()
            score[i] = np.max(scale * (np.abs(k[j]) @ np.abs(q[i])))
    return out, lse, size, score


def attention(q, cache, starts, lengths, table, scale, causal=True, window=0, out=None):
    """q tokens x q_heads x d over cache (k codes, k scales, v codes, v scales).
    Rows behind the last sequence are NaN here.  Returns out, lse, size, score."""
    tokens, hq, d = q.shape
    heads = cache[0].shape[1]
    group = hq // heads
    res = [np.full((tokens, hq, d), np.nan), np.full((tokens, hq), np.nan), np.zeros((tokens, hq, d)),
           np.zeros((tokens, hq))]
    for b in range(len(lengths)):
        r0, r1, n = int(starts[b]), int(starts[b + 1]), max(0, int(lengths[b]))
        k = sequence(cache[0], cache[1], table[b], n)
        v = sequence(cache[2], cache[3], table[b], n)
        pos = n - (r1 - r0) + np.arange(r1 - r0)
        j = np.arange(n)
        sees = np.broadcast_to(pos[:, None] >= 0, (r1 - r0, n)).copy()
        if causal:
            sees &= j[None] <= pos[:, None]
        if window:
            sees &= j[None] > pos[:, None] - window
        for h in range(hq):
            for to, x in zip(res, attend(q[r0:r1, h], k[h // group], v[h // group], scale, sees)):
                to[r0:r1, h] = x
    return res


# ---------------------------------------------------- norm, position, rotation
def hadamard(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(d)


def turn(u, pos, freqs, interleaved, back=False):
    """u tokens x heads x d, its first 2 len(freqs) columns turned in pairs."""
    u = u.copy()
    n = len(freqs)
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freqs)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None] * (-1 if back else 1)
    first, second = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    x, y = u[..., first], u[..., second]
    u[..., first], u[..., second] = x * c - y * s, x * s + y * c
    return u


def norm_rope(x, pos, freqs, gamma, eps, interleaved, signs):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r if gamma is None else x * r * gamma
    u = turn(u, pos, freqs, interleaved)
    return u if signs is None else (u * signs) @ hadamard(x.shape[-1])


def norm_rope_vjp(x, pos, freqs, gamma, eps, interleaved, signs, dy):
    """dx, dgamma, and what their errors go by: r |gamma g| per head, sum |g n|."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    g = dy if signs is None else (dy @ hadamard(x.shape[-1])) * signs
    g = turn(g, pos, freqs, interleaved, back=True)
    v = g if gamma is None else g * gamma
    dx = r * (v - n * (v * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1)), np.linalg.norm(r * v, axis=-1), np.abs(g * n).sum((0, 1))
