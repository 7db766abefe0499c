"""The operators of attention over a cache in 4 bits, as cases that can be measured.

A cache holds the keys and values of each head in blocks of 32 values: E2M1
codes (0 .5 1 1.5 2 3 4 6 and a sign, two to a byte, the lower half first) and
one scale, a power of two (E8M0): the smallest with max|v| <= 6 scale, at least
2^-120.  It is made of pages of `page` tokens, [pages][heads][page][...]; the
pages of a sequence stand in its row of a table.  The tokens of a call are the
last ones of their sequences.

  norm_rope       root-mean-square norm of every query and key head, then the
                  position rotation, then (signs) the signed Hadamard rotation
  norm_rope_grad  its gradients
  write           new tokens' keys and values into the cache, and what the
                  cache then holds of them
  read            a sequence's keys and values out of the cache
  attention       queries over the cache

`own` chooses between the plain form (torch, fp32) and the library's calls.
"""
import math

import torch

own = False

BLK = 32
EPS = 1e-6
_IO = {"f32": torch.float32, "bf16": torch.bfloat16}
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of decoding: latency
        {"name": "norm_rope 1 token 32+8x128", "op": "norm_rope", "tokens": 1, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "interleaved": False, "gamma": True, "signs": True, "io": "bf16", "far": 100000},
        # a batch of prompts, rotated heads for the 4-bit cache
        {"name": "norm_rope 16384 tokens 32+8x128", "op": "norm_rope", "tokens": 16384, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "interleaved": False, "gamma": True, "signs": True, "io": "bf16", "far": 16384},
        # the backward pass of a training batch of that size
        {"name": "norm_rope_grad 16384x32+8x128", "op": "norm_rope_grad", "tokens": 16384, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "interleaved": False, "gamma": True, "signs": True, "io": "bf16", "far": 16384},
        # a ragged batch of fp32 heads of 80, of which 48 are rotated, in neighbouring pairs
        {"name": "norm_rope_grad 1021x12+4x80 f32", "op": "norm_rope_grad", "tokens": 1021, "hq": 12, "hk": 4, "d": 80,
         "rot": 48, "interleaved": True, "gamma": True, "signs": False, "io": "f32", "far": 2000000},
        # one new token for each of 64 requests
        {"name": "write 64x1 8x128", "op": "write", "seqs": 64, "new": 1, "shortest": 100, "longest": 4096, "hk": 8,
         "d": 128, "page": 16, "io": "bf16"},
        # chunks of 7 prompts
        {"name": "write 7x4000 8x128", "op": "write", "seqs": 7, "new": 4000, "shortest": 1000, "longest": 12000, "hk": 8,
         "d": 128, "page": 64, "io": "bf16"},
        # whole sequences back, for a program without 4-bit attention
        {"name": "read 8x8192 8x128", "op": "read", "seqs": 8, "new": 8192, "shortest": 777, "longest": 8192, "hk": 8,
         "d": 128, "page": 64, "io": "bf16"},
        # one token of one request: latency
        {"name": "attention 1x1 4096 32/8x128", "op": "attention", "seqs": 1, "new": 1, "shortest": 4096, "longest": 4096,
         "hq": 32, "hk": 8, "d": 128, "page": 16, "window": 0, "causal": True},
        # one token for each of 64 requests of all ages
        {"name": "attention 64x1 8192 32/8x128", "op": "attention", "seqs": 64, "new": 1, "shortest": 50, "longest": 8192,
         "hq": 32, "hk": 8, "d": 128, "page": 16, "window": 0, "causal": True},
        # one token behind a very long text
        {"name": "attention 1x1 131072 64/8x128", "op": "attention", "seqs": 1, "new": 1, "shortest": 131072,
         "longest": 131072, "hq": 64, "hk": 8, "d": 128, "page": 64, "window": 0, "causal": True},
        # three drafted tokens each, heads of 96, a sliding window, one sequence that has nothing yet
        {"name": "attention 9x3 1500 24/4x96", "op": "attention", "seqs": 9, "new": 3, "shortest": 0, "longest": 1500,
         "hq": 24, "hk": 4, "d": 96, "page": 32, "window": 500, "causal": True},
        # chunks of four prompts behind what the cache already holds
        {"name": "attention 4x2048 8192 32/8x128", "op": "attention", "seqs": 4, "new": 2048, "shortest": 2048,
         "longest": 8192, "hq": 32, "hk": 8, "d": 128, "page": 64, "window": 0, "causal": True},
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of lo..hi."""
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "write", "read", "attention", "attention", "attention"])
    c = {"op": op}
    if op.startswith("norm_rope"):
        c["hk"] = rng.choice([1, 2, 4, 8])
        c["hq"] = c["hk"] * rng.choice([1, 3, 4])
        c["d"] = rng.choice([64, 80, 96, 128, 192, 256])
        c["io"] = rng.choice(["bf16", "f32"])
        c["tokens"] = _spread(rng, 1, 16384 * (128 if c["io"] == "bf16" else 64) // c["d"])
        c["rot"] = c["d"] if rng.random() < 0.6 else 16 * rng.randint(1, c["d"] // 16)
        c |= {"interleaved": rng.random() < 0.4, "gamma": rng.random() < 0.7,
              "signs": c["d"] in (64, 128, 256) and rng.random() < 0.6, "far": _spread(rng, 1000, 2000000)}
        return c
    c["page"] = rng.choice([16, 32, 64, 256])
    c["hk"] = rng.choice([1, 2, 3, 4, 8])
    c["d"] = rng.choice([64, 96, 128, 128, 192, 256])
    if op != "attention":
        c["io"] = rng.choice(["bf16", "f32"])
        c["seqs"] = _spread(rng, 1, 64)
        c["longest"] = _spread(rng, 16, 32768 * (128 if c["io"] == "bf16" else 64) // c["d"] // c["seqs"])
        c["shortest"] = rng.randint(0, c["longest"])
        c["new"] = 1 if op == "write" and rng.random() < 0.3 else _spread(rng, 1, c["longest"])
        return c
    kind = rng.choice(["tokens", "drafts", "prompts"])
    wide = 128 / max(128, c["d"])
    if kind == "prompts":
        c["hq"] = c["hk"] * rng.choice([1, 2, 4])
        c["seqs"] = rng.randint(1, 4)
        c["new"] = _spread(rng, 16, int(2048 * wide))
        c["longest"] = _spread(rng, c["new"], 4500)
    else:
        c["hq"] = c["hk"] * rng.choice([1, 2, 4, 5, 8])
        c["seqs"] = _spread(rng, 1, 64)
        c["new"] = 1 if kind == "tokens" else rng.randint(2, 8)
        c["longest"] = _spread(rng, 16, int(131072 * wide) // c["seqs"])
    c["shortest"] = rng.randint(0, c["longest"])
    c["window"] = _spread(rng, 16, 4096) if rng.random() < 0.25 else 0
    c["causal"] = rng.random() < 0.9 or c["window"] > 0
    return c


def _lengths(case):
    """The sequences' lengths, ragged, the first the longest, and how many of each one's tokens are the call's."""
    lo, hi = case["shortest"], case["longest"]
    lengths = [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(case["seqs"])]
    if lo == 0 and len(lengths) > 1:
        lengths[-1] = 0
    return lengths, [min(case["new"], n) if case["op"] != "attention" else case["new"] for n in lengths]


# ----------------------------------------------------------------- inputs
def _heavy(g, *shape):
    """Student-t values of 3 degrees of freedom."""
    chi = torch.zeros(*shape, device="cuda")
    for _ in range(3):
        chi += torch.randn(*shape, generator=g, device="cuda") ** 2
    return torch.randn(*shape, generator=g, device="cuda") * torch.sqrt(3.0 / chi.clamp_(min=1e-6))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    d, hk = case["d"], case["hk"]
    if case["op"].startswith("norm_rope"):
        io, n, hq, grad = _IO[case["io"]], case["tokens"], case["hq"], case["op"] == "norm_rope_grad"
        # the projection's output: queries, keys and values of a token side by side
        qkv = _heavy(g, n, hq + 2 * hk, d).to(io)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["gq"], s["gk"] = ((1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(io) for _ in range(2)) \
            if case["gamma"] else (None, None)
        far = case["far"]
        s["pos"] = (torch.randint(0, far, (1,), generator=g, device="cuda") + torch.arange(n, device="cuda")) % far
        s["freqs"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        s["sg"] = (torch.randint(0, 2, (d,), generator=g, device="cuda") * 2 - 1).to(torch.int8) if case["signs"] else None
        if grad:
            s["dyq"], s["dyk"] = (_heavy(g, n, h, d).mul_(1e-3).to(io) for h in (hq, hk))
        s["yq"], s["yk"] = (torch.empty(n, h, d, dtype=io, device="cuda") for h in (hq, hk))
        return s
    lengths, new = _lengths(case)
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    width, pages = max(1, max(need)), sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")[None]
    held = col < torch.tensor(need, device="cuda")[:, None]
    table[held] = order[(at[:-1, None] + col)[held]]
    s["table"] = table
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["rows"], s["most"] = sum(new), max(new)
    if case["op"] == "write":
        io = _IO[case["io"]]
        qkv = torch.randn(s["rows"], 2 * hk, d, generator=g, device="cuda")
        s["k"], s["v"] = (qkv * torch.exp(0.5 * torch.randn(s["rows"], 2 * hk, 1, generator=g, device="cuda"))) \
            .to(io).split(hk, 1)
        s["cache"] = [torch.zeros(pages, hk, page, d // n, dtype=torch.uint8, device="cuda") for n in (2, BLK, 2, BLK)]
    else:
        # what earlier tokens left: keys and values close to normal, their sizes spread; unwritten places hold anything
        s["cache"] = []
        for _ in range(2):
            x = torch.randn(pages, hk, page, d, generator=g, device="cuda")
            x *= torch.exp(0.5 * torch.randn(pages, hk, page, 1, generator=g, device="cuda"))
            s["cache"] += _plain_quantise(x)
        ends = [(b, n % page) for b, n in enumerate(lengths) if n % page]
        if ends:
            used = table[[b for b, _ in ends], [need[b] - 1 for b, _ in ends]].long()
            behind = torch.arange(page, device="cuda") >= torch.tensor([n for _, n in ends], device="cuda")[:, None]
            for scales in (s["cache"][1], s["cache"][3]):
                scales[used] = torch.where(behind[:, None, :, None], 255, scales[used])
        if case["op"] == "attention":
            s["q"] = torch.randn(s["rows"], case["hq"], d, generator=g, device="cuda").to(torch.bfloat16)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["rows"], case["hq"], device="cuda")
    s["cache"] = tuple(t if i % 2 == 0 else t.view(torch.float8_e8m0fnu) for i, t in enumerate(s["cache"]))
    if case["op"] != "attention":
        s["ko"], s["vo"] = (torch.empty(s["rows"], hk, d, dtype=_IO[case["io"]], device="cuda") for _ in range(2))
    return s


# -------------------------------------------------------------- one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import structured_rotations_amd as lib
    op = s["op"]
    if op == "norm_rope":
        return lib.harp_qk_norm_rope(s["q"], s["k"], s["pos"], s["freqs"], s["gq"], s["gk"], EPS, s["interleaved"],
                                     s["sg"], q_out=s["yq"], k_out=s["yk"])
    if op == "norm_rope_grad":
        return lib.harp_qk_norm_rope_vjp(s["q"], s["k"], s["pos"], s["freqs"], s["dyq"], s["dyk"], s["gq"], s["gk"], EPS,
                                         s["interleaved"], s["sg"], dq=s["yq"], dk=s["yk"])
    cache = lib.Cache4(*s["cache"])
    plan = (s["starts"], s["lengths"], s["table"])
    if op == "attention":
        return lib.harp_kv4_attention(s["q"], cache, *plan, causal=s["causal"], window=s["window"], out=s["out"],
                                      lse=s["lse"])
    if op == "write":
        lib.harp_kv4_write(s["k"], s["v"], cache, *plan)
    return lib.harp_kv4_read(cache, *plan, s["rows"], s["io"], k=s["ko"], v=s["vo"])


def _plain(s):
    op = s["op"]
    if op == "norm_rope":
        turn = _plain_turn(s)
        return tuple(_plain_hadamard(_plain_rope(_plain_norm(x.float(), w)[0], *turn, s["interleaved"]), s["sg"]).to(x.dtype)
                     for x, w in ((s["q"], s["gq"]), (s["k"], s["gk"])))
    if op == "norm_rope_grad":
        (dq, dgq), (dk, dgk) = (_plain_grad(s, *a) for a in ((s["q"], s["gq"], s["dyq"]), (s["k"], s["gk"], s["dyk"])))
        return dq, dk, dgq, dgk
    if op == "attention":
        return _plain_attention(s)
    page = s["page"]
    seq, at = _plain_places(s)
    slot = (s["table"][seq, (at // page).long()].long(), (at % page).long())
    if op == "write":
        for x, codes, scales in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
            c, e = _plain_quantise(x.float())
            codes[slot[0], :, slot[1]] = c
            scales.view(torch.uint8)[slot[0], :, slot[1]] = e
    return tuple(_plain_values(codes[slot[0], :, slot[1]], scales.view(torch.uint8)[slot[0], :, slot[1]]).to(_IO[s["io"]])
                 for codes, scales in (s["cache"][:2], s["cache"][2:]))


def _plain_norm(x, w):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    return (n if w is None else n * w.float()), n, r


def _plain_turn(s):
    a = s["pos"].double()[:, None] * s["freqs"]          # far positions: the angle in 64 bits
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _plain_rope(x, cos, sin, interleaved):
    n = cos.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _plain_hadamard_matrix(d, device):
    i = torch.arange(d, device=device)
    ones = ((i[:, None] & i)[..., None] >> torch.arange(10, device=device) & 1).sum(-1)
    return (1 - 2 * (ones & 1)).float() / math.sqrt(d)


def _plain_hadamard(x, signs):
    return x if signs is None else torch.matmul(x * signs.float(), _plain_hadamard_matrix(x.shape[-1], x.device))


def _plain_grad(s, x, w, dy):
    cos, sin = _plain_turn(s)
    _, n, r = _plain_norm(x.float(), None)
    g = dy.float()
    if s["sg"] is not None:
        g = torch.matmul(g, _plain_hadamard_matrix(g.shape[-1], g.device)) * s["sg"].float()
    g = _plain_rope(g, cos, -sin, s["interleaved"])
    v = g if w is None else g * w.float()
    dx = r * (v - n * (v * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (None if w is None else (g * n).sum((0, 1)))


def _plain_quantise(x):
    """Packed codes and scale bytes of the last dimension's blocks of 32."""
    b = x.unflatten(-1, (-1, BLK))
    m, e = torch.frexp(b.abs().amax(-1))                  # max = m 2^e, 1/2 <= m < 1; 6 2^k = 3/4 2^(k + 3)
    e = torch.where(m == 0, -120, torch.where(m <= 0.75, e - 3, e - 2)).clamp(min=-120)
    a = torch.ldexp(b, -e[..., None])
    v = a.abs()
    code = (v > 0.25).byte() + (v >= 0.75).byte() + (v > 1.25).byte() + (v >= 1.75).byte() + (v > 2.5).byte() \
        + (v >= 3.5).byte() + (v > 5.0).byte() + 8 * torch.signbit(a).byte()
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).byte()


def _plain_values(codes, scales):
    levels = torch.tensor(_LEVELS, device=codes.device)
    levels = torch.cat((levels, -levels))
    v = levels[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return v * torch.exp2(scales.float() - 127.0).repeat_interleave(BLK, -1)


def _plain_places(s):
    """Of every row: its sequence, and its position there."""
    row = torch.arange(s["rows"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["starts"][1:], row, right=True)
    return seq, s["lengths"][seq] - s["starts"][1:][seq] + row


def _plain_attention(s):
    q, hk, d, most = s["q"], s["hk"], s["d"], s["most"]
    seqs, width = s["table"].shape
    keys = width * s["page"]
    table = s["table"].clamp(min=0).long()
    j = torch.arange(keys, device=q.device)
    held = (j < s["lengths"][:, None])[:, None, :, None]
    k, v = (torch.where(held, _plain_values(codes[table].transpose(1, 2).flatten(2, 3),
                                            scales.view(torch.uint8)[table].transpose(1, 2).flatten(2, 3)), 0.0)
            for codes, scales in (s["cache"][:2], s["cache"][2:]))                 # seqs x hk x keys x d
    i = torch.arange(most, device=q.device)
    count = s["starts"][1:] - s["starts"][:-1]
    row = (s["starts"][:-1, None] + i).clamp(max=max(0, s["rows"] - 1)).long()     # a row beyond a sequence's: any
    at = (s["lengths"] - count)[:, None] + i                                       # seqs x most
    sees = (j < s["lengths"][:, None])[:, None] & (at >= 0)[..., None]
    if s["causal"]:
        sees = sees & (j <= at[..., None])
    if s["window"]:
        sees = sees & (j > at[..., None] - s["window"])
    qp = q[row].float().view(seqs, most, hk, -1, d).permute(0, 2, 3, 1, 4)         # seqs x hk x group x most x d
    z = torch.matmul(qp.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (-1, most)) / math.sqrt(d)
    z = z.masked_fill_(~sees[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, most)) / torch.where(l == 0, 1.0, l)
    seq, _ = _plain_places(s)
    back = (torch.arange(s["rows"], device=q.device) - s["starts"][seq]).long()
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, back]
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[seq, back]
    return o.to(q.dtype), lse


# ------------------------------------------------------------------- work
def work(case):
    d, hk = case["d"], case["hk"]
    if case["op"].startswith("norm_rope"):
        n, eb = case["tokens"] * (case["hq"] + hk) * d, 4 if case["io"] == "f32" else 2
        small = 8 * case["tokens"] + 4 * case["rot"] + (2 * d * eb if case["gamma"] else 0) + (d if case["signs"] else 0)
        turn = 10 + (2 * math.log2(d) if case["signs"] else 0)
        if case["op"] == "norm_rope":
            return {"bytes": 2 * n * eb + small, "flops": n * turn}
        return {"bytes": 3 * n * eb + small + (8 * d if case["gamma"] else 0), "flops": n * (turn + 8)}
    lengths, new = _lengths(case)
    pages = 4 * sum(-(-n // case["page"]) for n in lengths)
    if case["op"] != "attention":
        n, eb = 2 * sum(new) * hk * d, 4 if case["io"] == "f32" else 2
        both = case["op"] == "write"
        return {"bytes": n * eb * (1 + both) + n * 17 // 32 + pages, "flops": n * (4 + 4 * both)}
    pairs = touched = 0
    for n, t in zip(lengths, new):
        at = range(n - t, n)
        hi = [min(n, p + 1) if case["causal"] else n for p in at]
        lo = [max(0, p + 1 - case["window"]) if case["window"] else 0 for p in at]
        seen = [max(0, h - l) if p >= 0 else 0 for p, h, l in zip(at, hi, lo)]
        pairs += sum(seen)
        if any(seen):
            touched += max(h for h, c in zip(hi, seen) if c) - min(l for l, c in zip(lo, seen) if c)
    rows = sum(new) * case["hq"]
    return {"bytes": 2 * touched * hk * d * 17 // 32 + pages + rows * (4 * d + 4), "flops": 4 * d * case["hq"] * pairs}


# ------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_forward(case, s, x, w) for x, w in ((s["q"], s["gq"]), (s["k"], s["gk"])))
    if case["op"] == "norm_rope_grad":
        (dq, dgq), (dk, dgk) = (_exact_grad(case, s, *a)
                                for a in ((s["q"], s["gq"], s["dyq"]), (s["k"], s["gk"], s["dyk"])))
        return dq, dk, dgq, dgk
    lengths, new = _lengths(case)
    if case["op"] == "write":
        return tuple(_exact_round(s[x].double()) for x in ("k", "v"))
    k, v = (_exact_decode(s["cache"][i], s["cache"][i + 1]) for i in (0, 2)) if case["op"] == "read" else (None, None)
    if case["op"] == "read":
        outs = []
        for x in (k, v):
            rows = [_exact_rows(x, s["table"][b], n, case["page"])[n - t:] for b, (n, t) in enumerate(zip(lengths, new))]
            outs.append(torch.cat(rows))
        return tuple(outs)
    group = case["hq"] // case["hk"]
    out = torch.zeros(s["rows"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, t) in enumerate(zip(lengths, new)):
        used = s["table"][b, :-(-n // case["page"])].long()
        kb, vb = (_exact_decode(s["cache"][i][used], s["cache"][i + 1][used]).transpose(1, 2).flatten(0, 1)[:n] for i in (0, 2))
        at = torch.arange(n - t, n, device="cuda")
        j = torch.arange(n, device="cuda")
        hidden = (at < 0)[:, None] | (j[None] < 0)
        if case["causal"]:
            hidden |= j[None] > at[:, None]
        if case["window"]:
            hidden |= j[None] <= at[:, None] - case["window"]
        some = ~hidden.all(1)
        for h in range(case["hq"] if n else 0):
            z = torch.mm(s["q"][first:first + t, h].double(), kb[:, h // group].t().contiguous()) * case["d"] ** -0.5
            z[hidden] = -math.inf
            e = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(some, e, 0.0)[:, None])
            out[first:first + t, h] = torch.mm(p, vb[:, h // group].contiguous())
            lse[first:first + t, h] = e
        first += t
    return out, lse


def _exact_decode(codes, scales):
    """sign, then mantissa and exponent bits of each E2M1 code, times the block's power of two."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    man, ex = c % 2, c // 2 % 4
    mag = torch.where(ex == 0, man * 0.5, (1 + 0.5 * man) * torch.exp2(ex.double() - 1))
    two = torch.exp2(scales.view(torch.uint8).double() - 127)
    return (torch.where(c >= 8, -mag, mag).unflatten(-1, (-1, BLK)) * two[..., None]).flatten(-2)


def _exact_rows(x, table, n, page):
    """The first n tokens of a sequence, tokens x heads x d."""
    return x[table[:-(-n // page)].long()].transpose(1, 2).flatten(0, 1)[:n]


def _exact_round(x):
    """x as a cache holds it."""
    b = x.unflatten(-1, (-1, BLK))
    top = b.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    scale = torch.exp2(torch.ceil(torch.log2(top / 6.0)).clamp(min=-120.0))
    scale = torch.where(6.0 * scale < top, 2.0 * scale, scale)
    scale = torch.where((3.0 * scale >= top) & (scale > 2.0 ** -120), 0.5 * scale, scale)
    a = b / scale
    # two significant bits from 1 on, steps of 1/2 below; round to even
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=1.0))) - 1.0)
    return (torch.round(a / step) * step * scale).flatten(-2)


def _exact_turn(case, s, x, back):
    """Pairs as complex numbers, turned; two positions in 2^31 turns apart still differ."""
    half = case["rot"] // 2
    unit = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), (-1 if back else 1) * torch.outer(s["pos"].double(), s["freqs"]))
    x = x.clone()
    first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
    second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_hadamard(x):
    """The Kronecker power of [[1, 1], [1, -1]] / sqrt 2, one factor at a time."""
    d, step = x.shape[-1], 1
    while step < d:
        y = x.unflatten(-1, (-1, 2, step))
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2).flatten(-3) * 0.5 ** 0.5
        step *= 2
    return x


def _exact_forward(case, s, x, w):
    x = x.double()
    y = x * (x.square().sum(-1, keepdim=True) / case["d"] + EPS) ** -0.5
    if w is not None:
        y = y * w.double()
    y = _exact_turn(case, s, y, False)
    return y if s["sg"] is None else _exact_hadamard(y * s["sg"].double())


def _exact_grad(case, s, x, w, dy):
    x, g = x.double(), dy.double()
    if s["sg"] is not None:
        g = _exact_hadamard(g) * s["sg"].double()
    g = _exact_turn(case, s, g, True)
    ms = x.square().sum(-1, keepdim=True) / case["d"] + EPS
    dgamma = None if w is None else (g * x * ms ** -0.5).sum(0).sum(0)
    if w is not None:
        g = g * w.double()
    # d/dx of x ms^-1/2
    return g * ms ** -0.5 - x * ((g * x).sum(-1, keepdim=True) / case["d"]) * ms ** -1.5, dgamma
