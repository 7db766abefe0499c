"""Attention over a 4-bit cache in the forms that large calls take: heads and
cache rows beyond 32 MiB, which are streamed past the caches; the cache written
and read by waves that walk over many tokens; attention whose parts have more
steps than page numbers are held for; single tokens and prompts in one call.

Tolerances.  u = 2^-24 and h = 2^-8 are the largest relative errors of one
rounding to fp32 and to bf16.
- heads, in l2: 32 u = 2^-19 of the norm (sum of squares and root 10 u, products
  3 u, cosines and sines 9 u over a pair, 9 Hadamard stages and their factor 10 u),
  h more for a bf16 result; dx: 2^-18 of r |gamma g|, h of itself if bf16.
- dgamma: of the sum of |g n|, 2^-18 for g and n, and fp32 sums of fewer than 200
  terms one after the other (a lane's, 32 of a workgroup, 16 and 10 over them): in
  all 2^-16.
- the cache is exact.
- attention: a score is off by dz = (d + 3) u times the sum of its products'
  magnitudes, a weight by dz, by h for its rounding to bf16 (2^-16 in tiles of 16
  rows) and by 2^-20, a result by 2 dz + h + 2^-19 of the weighted mean of |v| and
  h of itself; lse by dz + 2^-20 + 2^-22 of itself.
"""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as K
from structured_rotations_amd import kv4

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U, H = 2.0 ** -24, 2.0 ** -8
IO = {"f32": torch.float32, "bf16": BF}
STREAMED = 32 << 20                                           # bytes


def cpu(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def say(*a):
    print("\n[case]", *a, flush=True)


# ---------------------------------------------------------------------- heads
def turn(u, pos, freqs, inter, back=False):
    """Heads in fp64 on the GPU, turned."""
    n = len(freqs)
    if n == 0:
        return u
    a = pos.double()[:, None, None] * freqs
    c, s = torch.cos(a), torch.sin(a) * (-1 if back else 1)
    x, y = (u[..., 0:2 * n:2], u[..., 1:2 * n:2]) if inter else (u[..., :n], u[..., n:2 * n])
    v, w = x * c - y * s, x * s + y * c
    first = torch.stack((v, w), -1).flatten(-2) if inter else torch.cat((v, w), -1)
    return torch.cat((first, u[..., 2 * n:]), -1)


HEADS = [  # d, pairs, interleaved, signs, io, tokens, q heads, k heads: every number of lanes, streamed and not
    (64, 32, False, True, "bf16", 33000, 6, 2),
    (128, 64, False, True, "bf16", 13200, 8, 2),
    (128, 64, False, True, "bf16", 4099, 8, 2),
    (128, 32, True, False, "f32", 16500, 3, 1),
    (80, 24, True, False, "f32", 17600, 5, 1),
    (96, 48, False, False, "bf16", 17500, 7, 3),
    (256, 128, False, True, "f32", 8300, 3, 1),
    (256, 128, False, True, "bf16", 8300, 6, 2),
    (512, 256, False, True, "bf16", 8300, 3, 1),
    (512, 128, True, True, "f32", 4200, 3, 1),
]


@pytest.mark.parametrize("case", HEADS, ids=lambda c: "-".join(map(str, c)))
def test_many_heads_and_their_gradients(case):
    d, pairs, inter, signs, io, tokens, hq, hk = case
    dt = IO[io]
    size = tokens * (hq + hk) * d * dt.itemsize
    say("many heads", *case, "streamed" if size >= STREAMED else "not streamed")
    assert (size >= STREAMED) == (case != HEADS[2])
    g = torch.Generator(device="cuda").manual_seed(d + tokens)
    odd = hk % 2                                              # rows an odd distance apart
    buf = torch.randn(tokens, (hq + 2 * hk) * d + odd, generator=g, device="cuda").to(dt)
    heads = [buf[:, :hq * d].unflatten(1, (hq, d)), buf[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))]
    up = [torch.randn(tokens, h, d, generator=g, device="cuda").to(dt) for h in (hq, hk)]
    gamma = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]
    pos = torch.randint(0, 1 << 17, (tokens,), generator=g, device="cuda")
    freqs = gpu(10000.0 ** (-np.arange(pairs) / pairs))
    sg = (torch.randint(0, 2, (d,), generator=g, device="cuda") * 2 - 1).to(torch.int8) if signs else None
    h = gpu(K.hadamard(d)) if signs else None
    y = kv4.harp_qk_norm_rope(*heads, pos, freqs, *gamma, eps=1e-5, interleaved=inter, signs=sg)
    kept = [x.clone() for x in heads]
    dx = [torch.full_like(x, 7.0) for x in kept]
    r = kv4.harp_qk_norm_rope_vjp(*heads, pos, freqs, *up, *gamma, eps=1e-5, interleaved=inter, signs=sg, dq=dx[0], dk=dx[1])
    h_ = H if io == "bf16" else 0
    for x, w, got, dy, dgot, dgamma in zip(heads, gamma, y, up, dx, (r.dgamma_q, r.dgamma_k)):
        x, w, dy = x.double(), w.double(), dy.double()
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
        n = x * rstd
        want = turn(n * w, pos, freqs, inter)
        if signs:
            want = torch.matmul(want * sg, h)
        err = (got.double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(err.max()) <= 2.0 ** -19 + h_
        gr = torch.matmul(dy, h) * sg if signs else dy
        gr = turn(gr, pos, freqs, inter, back=True)
        assert bool(((dgamma.double() - (gr * n).sum((0, 1))).abs() <= 2.0 ** -16 * (gr * n).abs().sum((0, 1))).all())
        v = gr * w
        want = rstd * (v - n * (v * n).mean(-1, keepdim=True))
        err = (dgot.double() - want).norm(dim=-1)
        assert bool((err <= 2.0 ** -18 * (rstd * v).norm(dim=-1) + h_ * want.norm(dim=-1)).all())
    # in place: results over the inputs, gradients over the inputs and over the upstream gradients
    kv4.harp_qk_norm_rope(*heads, pos, freqs, *gamma, eps=1e-5, interleaved=inter, signs=sg, q_out=heads[0], k_out=heads[1])
    assert torch.equal(heads[0], y[0]) and torch.equal(heads[1], y[1])
    for x, k in zip(heads, kept):
        x.copy_(k)
    tail = buf[:, (hq + hk) * d:].clone()
    r2 = kv4.harp_qk_norm_rope_vjp(*heads, pos, freqs, *up, *gamma, eps=1e-5, interleaved=inter, signs=sg, dq=heads[0], dk=heads[1])
    assert torch.equal(heads[0], dx[0]) and torch.equal(heads[1], dx[1]) and torch.equal(buf[:, (hq + hk) * d:], tail)
    assert torch.equal(r2.dgamma_q, r.dgamma_q) and torch.equal(r2.dgamma_k, r.dgamma_k)
    kv4.harp_qk_norm_rope_vjp(*kept, pos, freqs, *up, *gamma, eps=1e-5, interleaved=inter, signs=sg, dq=up[0], dk=up[1])
    assert torch.equal(up[0], dx[0]) and torch.equal(up[1], dx[1])


# ----------------------------------------------------------------- cache rows
def quantize(x):
    """The oracle's coding, all blocks at once; x (..., d) fp64."""
    b = x.reshape(*x.shape[:-1], -1, K.BLK)
    top = np.abs(b).max(-1)
    m, e = np.frexp(top)                                      # top = m 2^e, m from 1/2 on: at most 6 2^k for m 2^e <= 3/4 2^(k + 3)
    e = np.where(top == 0, -120, np.maximum(np.where(m <= 0.75, e - 3, e - 2), -120))
    codes = np.empty(b.shape, np.uint8)
    for i in range(0, len(b), 4096):
        codes[i:i + 4096] = K.encode(np.ldexp(b[i:i + 4096], -e[i:i + 4096, ..., None]))
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | codes[..., 1::2] << 4, (e + 127).astype(np.uint8)


ROWS = [  # sequences, tokens of each up to, heads, d, page, io: what a wave takes, and whether it is streamed
    (6000, 6, 3, 96, 16, "bf16"),                             # 2 tokens, of its 256 units 72 have a head
    (6000, 6, 3, 96, 16, "f32"),                              # the same, streamed
    (3100, 6, 5, 224, 32, "bf16"),                            # 2 tokens by two waves, of the second's 256 units 24; streamed
    (9000, 14, 1, 32, 16, "bf16"),                            # 7 tokens of 8 units
    (40, 900, 2, 64, 64, "f32"),                              # 2 tokens, pages that end within them
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_write_and_read_many_tokens(case):
    seqs, most, heads, d, page, io = case
    rng = np.random.default_rng(seqs + d)
    new = rng.integers(0, most + 1, seqs)                     # some have none
    before = rng.integers(-3, 2 * page, seqs) * (rng.random(seqs) < 0.7)
    lengths = np.maximum(new + before, 0)                     # in front of some, a few rows before their beginning
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1])
    tokens = rows + 37                                        # behind the last sequence
    rounds = -(-heads * d // 4 // 64)
    run = max(1, tokens * -(-rounds // 4) // 8192)
    size = 2 * tokens * heads * d * IO[io].itemsize
    say("many rows", *case, "rows", rows, "tokens of a wave", run, "streamed" if size >= STREAMED else "not streamed")
    assert tokens * rounds > 8192 and run >= 2
    need = -(-lengths // page)
    width, pages = int(need.max()) + 1, int(need.sum()) + 2
    table = rng.integers(-9, 10 ** 9, (seqs, width))
    order = rng.permutation(pages)
    first = np.concatenate([[0], np.cumsum(need)])
    for b in range(seqs):
        table[b, :need[b]] = order[first[b]:first[b + 1]]
    lost = rng.choice(np.nonzero(need)[0], 5)
    table[lost, need[lost] - 1] = [-1, pages, 1 << 30, -2 ** 31, pages + 1]
    c = [rng.integers(0, 256, (pages, heads, page, n), dtype=np.uint8) for n in (d // 2, d // 32)] * 2
    cache = kv4.Cache4(*(gpu(x) if i % 2 == 0 else gpu(x).view(kv4.SCALES) for i, x in enumerate(c)))
    c = [x.copy() for x in c]
    plan = tuple(gpu(x.astype(np.int32)) for x in (starts, lengths, table))
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(tokens, (2 * heads + 1) * d + 1, generator=g, device="cuda")
    qkv = (qkv * torch.exp(2 * torch.randn(tokens, 1, generator=g, device="cuda"))).to(IO[io])
    k, v = (qkv[:, i * d:(i + heads) * d].unflatten(1, (heads, d)) for i in (0, heads + 1))
    # every row's place, as the oracle has it (see test_the_places_are_the_oracles)
    kind, at, place = places(starts, lengths, table, page, pages, tokens)
    held = kind == 1
    kv4.harp_kv4_write(k, v, cache, *plan)
    for x, codes, scales in ((k, c[0], c[1]), (v, c[2], c[3])):
        x = cpu(x[gpu(np.nonzero(held)[0])])
        codes[at[held], :, place[held]], scales[at[held], :, place[held]] = quantize(x)
        some = rng.integers(0, len(x), 20)
        for a, b in zip(quantize(x[some]), K.quantize(x[some])):
            assert np.array_equal(a, b)
    for got, want in zip(cache, c):                           # the whole of it: nothing else has changed
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    out = torch.full((tokens, 2 * heads * d + 3), 7.0, dtype=IO[io], device="cuda")
    ko, vo = (out[:, i * heads * d:(i + 1) * heads * d].unflatten(1, (heads, d)) for i in (0, 1))
    kv4.harp_kv4_read(cache, *plan, tokens, io, k=ko, v=vo)
    for got, codes, scales in ((ko, c[0], c[1]), (vo, c[2], c[3])):
        want = np.full((tokens, heads, d), 7.0)
        want[kind == 0], want[kind == 2] = 0.0, np.nan
        want[held] = K.dequantize(codes[at[held], :, place[held]], scales[at[held], :, place[held]])
        assert np.array_equal(cpu(got), want, equal_nan=True)
    assert bool((out[:, 2 * heads * d:] == 7).all())


def places(starts, lengths, table, page, pages, tokens):
    """Of each row: 0 (before its sequence's beginning), 1 (in the cache), 2 (no
    page), 3 (of no sequence), its page and its place there."""
    row = np.arange(tokens)
    seq = np.minimum(np.searchsorted(starts[1:], row, side="right"), len(lengths) - 1)
    pos = lengths[seq] - (starts[seq + 1] - row)
    i = np.maximum(pos, 0) // page
    at = np.where(i < table.shape[1], table[seq, np.minimum(i, table.shape[1] - 1)], -1)
    kind = np.where(row >= starts[-1], 3, np.where(pos < 0, 0, np.where((at >= 0) & (at < pages), 1, 2)))
    return kind, at, np.maximum(pos, 0) % page


# ------------------------------------------------------------------ attention
class Long:
    """Sequences over a cache of random codes, of which they may share pages."""

    def __init__(self, lengths, new, heads, d, page, pages, seed=0):
        rng = np.random.default_rng(seed)
        self.rng, self.lengths, self.heads, self.d, self.page = rng, np.array(lengths), heads, d, page
        self.starts = np.concatenate([[0], np.cumsum(new)])
        self.rows = int(self.starts[-1])
        need = -(-self.lengths // page)
        self.table = np.full((len(lengths), int(need.max())), -1)
        for b, n in enumerate(need):
            self.table[b, :n] = np.concatenate([rng.permutation(pages) for _ in range(1 + n // pages)])[:n]
        self.cache = []
        for _ in range(2):
            self.cache += [rng.integers(0, 256, (pages, heads, page, d // 2), dtype=np.uint8),
                           rng.integers(124, 129, (pages, heads, page, d // 32), dtype=np.uint8)]

    def on_gpu(self):
        return (kv4.Cache4(*(gpu(x) if i % 2 == 0 else gpu(x).view(kv4.SCALES) for i, x in enumerate(self.cache))),
                tuple(gpu(x.astype(np.int32)) for x in (self.starts, self.lengths, self.table)))

    def one(self, b, h, side):
        """A sequence's keys (side 0) or values (2) of one head, NaN where it has no page."""
        codes, scales = (x[:, h:h + 1] for x in self.cache[side:side + 2])
        return K.sequence(codes, scales, self.table[b], int(self.lengths[b]))[0]

    def check(self, q, out, lse, some, window=0):
        """Some rows: (sequence, token of the call, head)."""
        group = q.shape[1] // self.heads
        got, gl, q = cpu(out), cpu(lse), cpu(q)
        held = {}
        for b, i, h in some:
            key = b, h // group
            if key not in held:
                held = {key: (self.one(*key, 0), self.one(*key, 2))}
            k, v = held[key]
            row, n = int(self.starts[b]) + i, int(self.lengths[b])
            pos = n - int(self.starts[b + 1] - self.starts[b]) + i
            j = np.arange(n)
            sees = (j <= pos) & (j > pos - window if window else True) & (pos >= 0)
            want, wl, size, score = K.attend(q[row:row + 1, h], k, v, self.d ** -0.5, sees[None])
            dz = (self.d + 3) * U * score[0]
            if np.isnan(want).any():
                assert np.array_equal(np.isnan(got[row, h]), np.isnan(want[0])), (b, i, h)
                continue
            tol = (2 * dz + H + 2.0 ** -19) * size[0] + H * np.abs(want[0]) + 2.0 ** -107
            assert (np.abs(got[row, h] - want[0]) <= tol).all(), (b, i, h)
            assert gl[row, h] == wl[0] or abs(gl[row, h] - wl[0]) <= dz + 2.0 ** -20 + 2.0 ** -22 * abs(wl[0]), (b, i, h)


RENEWED = [  # sequences, their lengths up to, tokens, q heads, heads, d, page, window
    (1, 2500, 2100, 32, 32, 32, 16, 0),                       # 128 rows a tile, up to 40 steps of 64 keys, 16 held
    (1, 2500, 2100, 32, 32, 32, 32, 1500),
    (1, 5200, 2050, 16, 16, 128, 64, 0),                      # in two parts of up to 41 steps
    (1, 3300, 2050, 8, 4, 96, 16, 0),                         # in parts of few steps, beginning behind the first pages
    (80, 8192, 1, 8, 8, 32, 16, 0),                           # 16 rows, parts of 140 and more steps of 32 keys, 128 held
    (75, 8192, 1, 32, 8, 128, 32, 0),
    (70, 8192, 2, 16, 8, 96, 16, 6000),
    (70, 8192, 5, 32, 8, 64, 16, 0),                          # 32 rows
    (512, 5000, 1, 8, 8, 32, 16, 0),                          # an item to a workgroup, up to 157 steps
    (400, 4800, 1, 32, 8, 128, 64, 0),
]


@pytest.mark.parametrize("case", RENEWED, ids=lambda c: "-".join(map(str, c)))
def test_page_numbers_are_renewed(case):
    seqs, longest, new, hq, heads, d, page, window = case
    say("renewed page numbers", *case)
    rng = np.random.default_rng(seqs + d)
    lengths = [longest] + [int(n) for n in rng.integers(longest * 3 // 4, longest + 1, seqs - 1)]
    lengths[-1] = lengths[min(3, seqs - 1)] = longest
    p = Long(lengths, [new] * seqs, heads, d, page, longest // page // 2 + 3)
    # a page that is missing behind the first that are held; the rows in front of it do not see it
    bad = 0 if seqs == 1 else 3
    missing = longest * 3 // 4 // page if seqs == 1 else 4400 // page
    p.table[bad, missing] = -1
    q = gpu(p.rng.standard_normal((p.rows, hq, d)).astype(np.float32), BF)
    cache, plan = p.on_gpu()
    out, lse = kv4.harp_kv4_attention(q, cache, *plan, window=window, lse=True)
    if seqs == 1:
        edge = missing * page - (longest - new)               # the first row that sees it
        some = [(0, i, h) for h in (0, hq // 2 + 1, hq - 1) for i in (0, 1, edge - 1, edge, new // 3, new // 2, new - 2, new - 1)]
        assert torch.isnan(out[edge:min(new, edge + (window or new))]).all() and torch.isfinite(out[:edge]).all()
    else:
        some = sorted((int(b), int(rng.integers(0, new)), int(h))
                      for b, h in zip(rng.integers(0, seqs, 14), rng.integers(0, hq, 14)))
        some += [(0, new - 1, 0), (bad, new - 1, hq - 1), (seqs - 1, 0, hq - 1)]
        nan = torch.isnan(out).any(-1).any(-1).view(seqs, new).any(1)
        assert nan.nonzero().flatten().tolist() == [bad]
    p.check(q, out, lse, some, window)


@pytest.mark.parametrize("singles,chunk,hq,heads,d", [(40, 90, 8, 2, 64), (20, 300, 8, 2, 128), (5, 700, 8, 2, 64), (63, 513, 8, 8, 96),
                                                      (7, 400, 4, 1, 256)])
@pytest.mark.parametrize("window", [0, 100])
def test_single_tokens_and_a_prompt_in_one_call(singles, chunk, hq, heads, d, window):
    """Whichever of the two the form suits, at the beginning, in the middle and
    at the end of the call; some sequences have nothing to ask."""
    say("mixed", singles, chunk, hq, heads, d, window)
    rng = np.random.default_rng(singles)
    new = [1] * singles
    lengths = [int(n) for n in rng.integers(1, 1200, singles)]
    for at, n, extra in ((0, chunk, 37), (singles // 2, chunk // 2 + 1, 300), (len(new), chunk // 3, 0)):
        new.insert(at, n)
        lengths.insert(at, n + extra)
    new[3], lengths[4] = 0, 0                                 # no token; a token in front of its sequence's beginning
    p = Long(lengths, new, heads, d, 16, 40, seed=singles)
    q = gpu(p.rng.standard_normal((p.rows + 2, hq, d)).astype(np.float32), BF)
    cache, plan = p.on_gpu()
    out = torch.full_like(q, 9.0)
    lse = torch.full((p.rows + 2, hq), 9.0, device="cuda")
    kv4.harp_kv4_attention(q, cache, *plan, window=window, out=out, lse=lse)
    some = [(b, i, h) for b, n in enumerate(new) for h in (0, hq - 1) for i in ([0] if n == 1 else sorted({0, 1, n // 2, n - 2, n - 1}) if n else [])]
    p.check(q, out, lse, some, window)
    assert bool((out[p.rows:] == 9).all()) and bool((lse[p.rows:] == 9).all())
