"""Python binding of include/harp.h's operators of attention over a cache in
4 bits, one function per entry point.

Arrays of heads are tensors of tokens x heads x d, torch.float32 or
torch.bfloat16, each head contiguous; tokens and heads may lie any distance
apart (the queries, keys and values of one projection's output are used as they
are).  A cache is four tensors (Cache4), pages of which belong to sequences by
a plan: starts, lengths and table, torch.int32 on the GPU.  The tokens of a call
are the last ones of their sequences: rows starts[b] .. starts[b + 1] - 1 are the
last of the lengths[b] tokens of sequence b, and table[b, i] is the page that
holds its tokens i page_size and on.

Argument marshalling only, with the rules of q8.py: every check runs first, the
GPU check last, then one library call.  stream: as in q8.py.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import lib
from ._streams import launch, new
from .q8 import _IO, _IO_NAME, _named, _on_gpu as _on_one_gpu, _p, _vec, _work

BLOCK = 32
SCALES = torch.float8_e8m0fnu
_WIDE = {torch.int32: 0, torch.int64: 1}


class Cache4(NamedTuple):
    """Keys and values in 4 bits: codes pages x kv_heads x page_size x d / 2
    (torch.uint8, two E2M1 codes a byte, the even column in the lower half) and
    scales pages x kv_heads x page_size x d / 32 (torch.float8_e8m0fnu).  Pages
    may lie any distance apart, everything within a page is contiguous."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def harp_kv4_cache(pages: int, kv_heads: int, page_size: int, d: int, device="cuda") -> Cache4:
    """An empty cache (zeros)."""
    if pages < 1 or kv_heads < 1 or not 16 <= page_size <= 1 << 20 or page_size & (page_size - 1):
        raise ValueError(f"pages and kv_heads must be at least 1, page_size a power of two from 16 to 2^20, "
                         f"got {pages}, {kv_heads}, {page_size}")
    if not BLOCK <= d <= 256 or d % BLOCK:
        raise ValueError(f"d must be a multiple of {BLOCK} up to 256, got {d}")

    def zeros(n):
        return torch.zeros(pages, kv_heads, page_size, n, dtype=torch.uint8, device=device)
    return Cache4(zeros(d // 2), zeros(d // BLOCK).view(SCALES), zeros(d // 2), zeros(d // BLOCK).view(SCALES))


def _heads(t, name, dtypes, tokens=None, heads=None, d=None):
    """A tokens x heads x d tensor: the distances of its tokens and heads."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(x) for x in dtypes)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be tokens x heads x d, got {tuple(shape)}")
    n, h, c = shape
    if tokens is not None and (n != tokens or c != d or (heads is not None and h != heads)):
        raise ValueError(f"{name} must be {tokens} x {'heads' if heads is None else heads} x {d}, got {n} x {h} x {c}")
    if h < 1 or c < 1:
        raise ValueError(f"{name} has no heads")
    st, sh, sd = t.stride()
    if sd != 1 and c > 1 and n > 0:
        raise ValueError(f"{name}: a head's values must be contiguous")
    return st, sh


def _out_heads(t, name, dtype, shape, like, stream):
    """The caller's result, checked, or a new one: it and its distances."""
    if t is None:
        t = new(shape, dtype, like, stream)
        return t, shape[1] * shape[2], shape[2]
    st, sh = _heads(t, name, (dtype,), *shape)
    return t, st, sh


def _cache(cache, kv_heads=None, d=None):
    """What the library takes of a cache (its pointers and distances), and its
    sizes.  The usual one, whole and contiguous, by few comparisons (a decoding
    step is a few calls of 10 us each); _cache_slowly has the others and the words."""
    try:
        kc, ks, vc, vs = cache
        shape = kc.shape
        pages, h, ps, c = shape
        scales = (pages, h, ps, c >> 4)
        if (c & 15 == 0 and pages > 0 and h > 0 and ps > 0 and c > 0 and kc.dtype is torch.uint8 and
                vc.dtype is torch.uint8 and ks.dtype is SCALES and vs.dtype is SCALES and vc.shape == shape and
                ks.shape == scales and vs.shape == scales and kc.is_contiguous() and ks.is_contiguous() and
                vc.is_contiguous() and vs.is_contiguous() and (d is None or 2 * c == d) and
                (kv_heads is None or h == kv_heads)):
            n = h * ps * c
            e = n >> 4
            return (kc.data_ptr(), n, ks.data_ptr(), e, vc.data_ptr(), n, vs.data_ptr(), e), (pages, h, ps, 2 * c)
    except (AttributeError, TypeError, ValueError):
        pass
    return _cache_slowly(cache, kv_heads, d)


def _cache_slowly(cache, kv_heads, d):
    kc, ks, vc, vs = cache
    args = []
    shape = None
    for t, name, dtype, per in ((kc, "k_codes", torch.uint8, 2), (ks, "k_scales", SCALES, BLOCK),
                                (vc, "v_codes", torch.uint8, 2), (vs, "v_scales", SCALES, BLOCK)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be pages x kv_heads x page_size x d / {per}, got {tuple(t.shape)}")
        pages, h, ps, c = t.shape
        if shape is None:
            shape = pages, h, ps, c * per
            if (kv_heads is not None and h != kv_heads) or (d is not None and c * per != d):
                raise ValueError(f"the cache holds {h} heads of {c * per} values, the call has "
                                 f"{'heads' if kv_heads is None else f'{kv_heads} heads'} of {d}")
            if pages < 1 or h < 1 or ps < 1 or c < 1:
                raise ValueError("the cache is empty")
        elif (pages, h, ps, c * per) != shape:
            raise ValueError(f"{name} must be {shape[0]} x {shape[1]} x {shape[2]} x {shape[3] // per}, got {tuple(t.shape)}")
        if t.is_contiguous():
            page = h * ps * c
        elif t[0].is_contiguous():
            page = t.stride(0)
        else:
            raise ValueError(f"{name} must be contiguous within a page")
        args += [t.data_ptr(), page]
    return args, shape


def _on_gpu(*tensors):
    """As that of q8.py, which has the words."""
    dev = tensors[0].get_device()
    if dev >= 0:
        for t in tensors:
            if t is not None and t.get_device() != dev:
                break
        else:
            return dev
    return _on_one_gpu(*tensors)


def _plan(starts, lengths, table):
    """What the library takes of a plan; as _cache."""
    try:
        n, width = table.shape
        if (starts.dtype is torch.int32 and lengths.dtype is torch.int32 and table.dtype is torch.int32 and width > 0 and
                starts.shape == (n + 1,) and lengths.shape == (n,) and starts.is_contiguous() and
                lengths.is_contiguous() and table.is_contiguous()):
            return starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), width, n, width
    except (AttributeError, TypeError, ValueError):
        pass
    return _plan_slowly(starts, lengths, table)


def _plan_slowly(starts, lengths, table):
    for t, name, dims in ((starts, "starts", 1), (lengths, "lengths", 1), (table, "table", 2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimension{'s' if dims > 1 else ''}, got {tuple(t.shape)}")
    n = lengths.shape[0]
    if starts.shape[0] != n + 1 or table.shape[0] != n:
        raise ValueError(f"for {n} lengths, starts must have {n + 1} entries and table {n} rows, "
                         f"got {starts.shape[0]} and {table.shape[0]}")
    width = table.shape[1]
    if width < 1:
        raise ValueError("table has no columns")
    if not starts.is_contiguous() or not lengths.is_contiguous() or (n > 0 and width > 1 and table.stride(1) != 1):
        raise ValueError("starts, lengths and the rows of table must be contiguous")
    ld = table.stride(0) if n > 1 else width
    return starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), ld, n, width


# ---------------------------------------------------- norm, position, rotation
class _Turn:
    """The arguments that harp_qk_norm_rope and its reverse mode share."""

    def __init__(self, q, k, positions, freqs, gamma_q, gamma_k, signs):
        self.q_at = _heads(q, "q", _IO)
        self.io = io = q.dtype
        self.tokens, self.hq, self.d = tokens, _, d = q.shape
        self.hk = 0
        self.k_at = (0, 0)
        if k is not None:
            self.k_at = _heads(k, "k", (io,), tokens, None, d)
            self.hk = k.shape[1]
        elif gamma_k is not None:
            raise ValueError("gamma_k goes with k only")
        self.pairs = 0
        self.wide = 0
        if freqs is not None:
            if not isinstance(freqs, torch.Tensor):
                raise TypeError("freqs must be a tensor")
            self.pairs = freqs.shape[0] if freqs.dim() == 1 else -1
            if self.pairs < 0 or 2 * self.pairs > d:
                raise ValueError(f"freqs must have at most {d // 2} entries, one for each pair, got {tuple(freqs.shape)}")
            _vec(freqs, "freqs", torch.float64, self.pairs)
        if self.pairs:
            if not isinstance(positions, torch.Tensor) or positions.dtype not in _WIDE:
                raise TypeError("positions must be a torch.int32 or torch.int64 tensor")
            _vec(positions, "positions", positions.dtype, tokens)
            self.wide = _WIDE[positions.dtype]
        if gamma_q is not None:
            _vec(gamma_q, "gamma_q", io, d)
        if gamma_k is not None:
            _vec(gamma_k, "gamma_k", io, d)
        if signs is not None:
            _vec(signs, "signs", torch.int8, d)


def harp_qk_norm_rope(q, k, positions, freqs, gamma_q=None, gamma_k=None, eps: float = 1e-6, interleaved: bool = False,
                      signs=None, q_out=None, k_out=None, stream=None):
    """Of every head of q and k (tokens x heads x d; k may be None): root-mean-
    square norm times gamma, then the turn of pair j by positions * freqs[j]
    radians (pairs are columns j and j + len(freqs), interleaved: 2j and 2j + 1),
    then, with signs, the signed Hadamard rotation of the head.  freqs: fp64, a
    multiple of 8 of them; None: no turn.  Returns (q_out, k_out); q_out may be
    q and k_out k."""
    a = _Turn(q, k, positions, freqs, gamma_q, gamma_k, signs)
    q_out, qt, qh = _out_heads(q_out, "q_out", a.io, (a.tokens, a.hq, a.d), q, stream)
    kt = kh = 0
    if k is not None:
        k_out, kt, kh = _out_heads(k_out, "k_out", a.io, (a.tokens, a.hk, a.d), q, stream)
    elif k_out is not None:
        raise ValueError("k_out goes with k only")
    if not a.pairs:
        positions = freqs = None
    tensors = (q, k, positions, freqs, gamma_q, gamma_k, signs, q_out, k_out)
    dev = _on_gpu(*tensors)
    launch(lib().harp_qk_norm_rope, stream, dev, tensors, _p(q), *a.q_at, a.hq, _p(k), *a.k_at, a.hk, a.tokens, a.d,
           _IO[a.io], _p(positions), a.wide, _p(freqs), a.pairs, bool(interleaved), _p(gamma_q), _p(gamma_k), eps,
           _p(signs), _p(q_out), qt, qh, _p(k_out), kt, kh)
    return q_out, k_out


def harp_qk_norm_rope_vjp_workspace(tokens: int, q_heads: int, k_heads: int, d: int) -> int:
    """Workspace bytes harp_qk_norm_rope_vjp needs for the gammas' gradients
    (-1: out of range)."""
    return int(lib().harp_qk_norm_rope_vjp_workspace(tokens, q_heads, k_heads, d))


class QkGrads(NamedTuple):
    """Gradients of q, k and (fp32, None unless wanted) of the two gammas."""
    dq: torch.Tensor
    dk: Optional[torch.Tensor]
    dgamma_q: Optional[torch.Tensor]
    dgamma_k: Optional[torch.Tensor]


def harp_qk_norm_rope_vjp(q, k, positions, freqs, dq_out, dk_out, gamma_q=None, gamma_k=None, eps: float = 1e-6,
                          interleaved: bool = False, signs=None, dq=None, dk=None, want_dgamma=None, dgamma_q=None,
                          dgamma_k=None, workspace=None, stream=None) -> QkGrads:
    """Reverse mode of harp_qk_norm_rope, from its inputs and the gradients of
    its results.  want_dgamma: by default those of the gammas that are given."""
    a = _Turn(q, k, positions, freqs, gamma_q, gamma_k, signs)
    gq = _heads(dq_out, "dq_out", (a.io,), a.tokens, a.hq, a.d)
    gk = (0, 0)
    if k is not None:
        gk = _heads(dk_out, "dk_out", (a.io,), a.tokens, a.hk, a.d)
    elif dk_out is not None or dk is not None or dgamma_k is not None:
        raise ValueError("dk_out, dk and dgamma_k go with k only")
    dq, qt, qh = _out_heads(dq, "dq", a.io, (a.tokens, a.hq, a.d), q, stream)
    kt = kh = 0
    if k is not None:
        dk, kt, kh = _out_heads(dk, "dk", a.io, (a.tokens, a.hk, a.d), q, stream)
    if want_dgamma is False and (dgamma_q is not None or dgamma_k is not None):
        raise ValueError("dgamma_q and dgamma_k go with want_dgamma")
    sums = []
    for t, name, wanted in ((dgamma_q, "dgamma_q", gamma_q is not None or want_dgamma),
                            (dgamma_k, "dgamma_k", k is not None and (gamma_k is not None or want_dgamma))):
        if t is not None:
            _vec(t, name, torch.float32, a.d)
        elif wanted and want_dgamma is not False:
            t = new(a.d, torch.float32, q, stream)
        sums.append(t)
    need = 0
    if sums[0] is not None or sums[1] is not None:
        need = lib().harp_qk_norm_rope_vjp_workspace(a.tokens, a.hq, a.hk, a.d)
    workspace, ws_bytes = _work(workspace, need, q, stream)
    if not a.pairs:
        positions = freqs = None
    tensors = (q, k, positions, freqs, gamma_q, gamma_k, signs, dq_out, dk_out, dq, dk, *sums, workspace)
    dev = _on_gpu(*tensors)
    launch(lib().harp_qk_norm_rope_vjp, stream, dev, tensors, _p(q), *a.q_at, a.hq, _p(k), *a.k_at, a.hk, a.tokens, a.d,
           _IO[a.io], _p(positions), a.wide, _p(freqs), a.pairs, bool(interleaved), _p(gamma_q), _p(gamma_k), eps,
           _p(signs), _p(dq_out), *gq, _p(dk_out), *gk, _p(dq), qt, qh, _p(dk), kt, kh, _p(sums[0]), _p(sums[1]),
           _p(workspace), ws_bytes)
    return QkGrads(dq, dk, *sums)


# ---------------------------------------------------------------------- cache
def harp_kv4_write(k, v, cache: Cache4, starts, lengths, table, stream=None) -> None:
    """Puts the keys and values (tokens x kv_heads x d) of the plan's tokens
    into the cache, in 4 bits.  Two sequences must not write the same place."""
    kt, kh = _heads(k, "k", _IO)
    tokens, heads, d = k.shape
    vt, vh = _heads(v, "v", (k.dtype,), tokens, heads, d)
    c, (pages, _, ps, _) = _cache(cache, heads, d)
    plan = _plan(starts, lengths, table)
    tensors = (k, v, *cache, starts, lengths, table)
    dev = _on_gpu(*tensors)
    launch(lib().harp_kv4_write, stream, dev, tensors, _p(k), kt, kh, _p(v), vt, vh, tokens, _IO[k.dtype], *c, pages,
           heads, ps, d, *plan)


def harp_kv4_read(cache: Cache4, starts, lengths, table, tokens: int, out: str = "bf16", k=None, v=None, stream=None):
    """The keys and values (tokens x kv_heads x d, "bf16" or "f32", both exact)
    that the cache holds of the plan's tokens.  Rows from starts[-1] on are left
    as they are.  Returns (k, v)."""
    c, (pages, heads, ps, d) = _cache(cache)
    plan = _plan(starts, lengths, table)
    if tokens < 0:
        raise ValueError(f"tokens must be at least 0, got {tokens}")
    odt = _named(_IO_NAME, out, "out")
    k, kt, kh = _out_heads(k, "k", odt, (tokens, heads, d), cache[0], stream)
    v, vt, vh = _out_heads(v, "v", odt, (tokens, heads, d), cache[0], stream)
    tensors = (*cache, starts, lengths, table, k, v)
    dev = _on_gpu(*tensors)
    launch(lib().harp_kv4_read, stream, dev, tensors, *c, pages, heads, ps, d, *plan, _p(k), kt, kh, _p(v), vt, vh, tokens,
           _IO[odt])
    return k, v


# ------------------------------------------------------------------ attention
def harp_kv4_attention_workspace(tokens: int, q_heads: int, kv_heads: int, d: int, page_size: int, sequences: int,
                                 width: int) -> int:
    """Workspace bytes harp_kv4_attention needs (0: none, -1: out of range);
    width: the table's columns."""
    return int(lib().harp_kv4_attention_workspace(tokens, q_heads, kv_heads, d, page_size, sequences, width))


def harp_kv4_attention(q, cache: Cache4, starts, lengths, table, scale: Optional[float] = None, causal: bool = True,
                       window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of q (tokens x q_heads x d, bf16) over the cache: a token sees
    its sequence's keys up to its own place (causal) and, with a window, only the
    last `window` of them.  scale: d^-1/2 by default.  lse: None, an fp32 tensor
    of tokens x q_heads, or True for a new one, to receive ln of the sums of
    weights.  Returns out (bf16), with lse (out, lse).  Rows from starts[-1] on
    are left as they are; a row that sees no key is 0, its lse -infinity."""
    qt, qh = _heads(q, "q", (torch.bfloat16,))
    tokens, hq, d = q.shape
    c, (pages, heads, ps, _) = _cache(cache, None, d)
    if hq % heads:
        raise ValueError(f"{hq} heads of queries for {heads} of keys: must be a multiple")
    plan = _plan(starts, lengths, table)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, ot, oh = _out_heads(out, "out", torch.bfloat16, (tokens, hq, d), q, stream)
    if lse is True:
        lse = new((tokens, hq), torch.float32, q, stream)
    elif lse is not None:
        if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32:
            raise TypeError("lse must be True or a torch.float32 tensor")
        if lse.shape != (tokens, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous, {tokens} x {hq}, got {tuple(lse.shape)}")
    need = lib().harp_kv4_attention_workspace(tokens, hq, heads, d, ps, plan[4], plan[5])
    workspace, ws_bytes = _work(workspace, need, q, stream)
    tensors = (q, *cache, starts, lengths, table, out, lse, workspace)
    dev = _on_gpu(*tensors)
    launch(lib().harp_kv4_attention, stream, dev, tensors, _p(q), qt, qh, tokens, hq, *c, pages, heads, ps, d, *plan,
           scale, bool(causal), window, _p(out), ot, oh, _p(lse), _p(workspace), ws_bytes)
    return out if lse is None else (out, lse)
