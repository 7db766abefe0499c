"""Host-side tests of attention over a 4-bit cache (no GPU needed): the oracle
against other routes, the C ABI's refusals before any HIP call, the checks of
the Python binding before the library is reached, and what an explicit stream
does with memory.
"""
import contextlib
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as K
from structured_rotations_amd import _lib, _streams, kv4

F32, BF16, I8, F64 = _lib.HARP_F32, _lib.HARP_BF16, _lib.HARP_I8, _lib.HARP_F64
OK, BAD, UNSUP = _lib.HARP_OK, _lib.HARP_ERR_INVALID_ARG, _lib.HARP_ERR_UNSUPPORTED


# ------------------------------------------------------------------ oracle
def test_codes_by_hand():
    v = np.array([0.0, -0.0, 0.25, 0.26, 0.75, 1.25, 1.3, 1.75, 2.5, 2.6, 3.5, 5.0, 5.1, 6.0, -0.25, -0.75, -5.0])
    want = [0, 8, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 8, 10, 14]
    assert K.encode(v).tolist() == want


def test_scales_by_hand():
    block = np.zeros(32)
    assert K.scale_byte(block) == 7
    for top, byte in ((6.0, 127), (np.nextafter(6.0, 7), 128), (3.0, 126), (3.0001, 127), (2.0 ** -119, 7), (1.0, 125),
                      (np.inf, 255), (np.nan, 255), (1.75 * 2.0 ** 127, 255), (1.74 * 2.0 ** 127, 253)):
        block[5] = -top
        assert K.scale_byte(block) == byte, top
    x = np.zeros(64)
    x[0], x[1], x[63] = 6.0, -1.0, 24.0
    codes, scales = K.quantize(x)
    assert scales.tolist() == [127, 129] and codes[0] == 7 | 10 << 4 and codes[31] == 7 << 4
    assert np.array_equal(K.dequantize(codes, scales), x)


def test_rounding_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(3 * rng.standard_normal((50, 1)))
    codes, scales = K.quantize(x)
    y = K.dequantize(codes, scales)
    s = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)
    a = np.abs(x) / s
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(x) <= 6 * s).all() and (np.abs(x).reshape(50, 3, 32).max(-1) > 3 * s[:, ::32]).all()
    assert (np.abs(y - x) <= step / 2 * s).all()


def test_attention_against_a_dense_softmax():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((n, 8)) for n in (3, 11, 11))
    sees = rng.random((3, 11)) < 0.6
    sees[1] = False
    out, lse, _, _ = K.attend(q, k, v, 0.3, sees)
    z = torch.from_numpy(0.3 * q @ k.T).masked_fill(~torch.from_numpy(sees), -torch.inf)
    p = torch.softmax(z[[0, 2]], -1).numpy()
    assert np.allclose(out[[0, 2]], p @ v, atol=1e-13) and np.allclose(lse, torch.logsumexp(z, -1).numpy(), atol=1e-13)
    assert (out[1] == 0).all() and lse[1] == -np.inf


def test_cache_by_hand():
    # two sequences over pages of 16: 20 and 3 tokens, the call has 5 and 3 of them, and one row behind
    codes, scales = np.zeros((4, 1, 16, 16), np.uint8), np.zeros((4, 1, 16, 1), np.uint8)
    starts, lengths, table = [0, 5, 8], [20, 3], [[2, 0], [3, -7]]
    at = K.places(starts, lengths, table, 16, 4, 9)
    assert at == [(2, 15), (0, 0), (0, 1), (0, 2), (0, 3), (3, 0), (3, 1), (3, 2), None]
    assert K.places([0, 2], [1], [[9]], 16, 4, 2) == ["before", "nowhere"]
    x = np.random.default_rng(2).standard_normal((9, 1, 32))
    K.write(x, codes, scales, starts, lengths, table)
    seq = K.sequence(codes, scales, table[0], 20)
    for r in range(5):
        assert np.array_equal(seq[0, 15 + r], K.dequantize(*K.quantize(x[r, 0])))
    out = np.full((9, 1, 32), 5.0)
    K.read(codes, scales, starts, lengths, table, out)
    assert np.array_equal(out[:5, 0], seq[0, 15:]) and (out[8] == 5).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_keeps_products_and_goes_by_distance(interleaved):
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((2, 1, 1, 16))
    f = 1.0 / 7.0 ** np.arange(6)
    t = lambda u, p: K.turn(u, [p], f, interleaved)[0, 0]            # noqa: E731
    assert np.isclose(t(x, 5) @ t(y, 9), t(x, 105) @ t(y, 109), atol=1e-12)
    assert np.allclose(K.turn(K.turn(x, [3], f, interleaved), [3], f, interleaved, back=True), x)
    j = (0, 1) if interleaved else (0, 6)
    assert np.isclose(t(x, 2)[j[0]], x[0, 0, j[0]] * np.cos(2) - x[0, 0, j[1]] * np.sin(2))
    assert np.array_equal(t(x, 2)[12:], x[0, 0, 12:])


@pytest.mark.parametrize("interleaved,signs", [(False, False), (True, True)])
def test_norm_rope_gradient_against_differences(interleaved, signs):
    rng = np.random.default_rng(4)
    x, dy, g = rng.standard_normal((2, 3, 16)), rng.standard_normal((2, 3, 16)), rng.standard_normal(16)
    pos, f = [3, 11], 1.0 / 5.0 ** np.arange(8 if signs else 5)
    s = np.sign(rng.standard_normal(16)) if signs else None
    dx, dg, _, _ = K.norm_rope_vjp(x, pos, f, g, 0.1, interleaved, s, dy)
    loss = lambda a, b: np.sum(K.norm_rope(a, pos, f, b, 0.1, interleaved, s) * dy)       # noqa: E731
    for idx in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[idx] = 1e-6
        assert abs((loss(x + e, g) - loss(x - e, g)) / 2e-6 - dx[idx]) < 1e-7
    for j in range(16):
        e = np.zeros(16)
        e[j] = 1e-6
        assert abs((loss(x, g + e) - loss(x, g - e)) / 2e-6 - dg[j]) < 1e-7


def test_hadamard_keeps_products():
    rng = np.random.default_rng(5)
    q, k, s = rng.standard_normal((4, 1, 64)), rng.standard_normal((4, 1, 64)), np.sign(rng.standard_normal(64))
    a, b = (K.norm_rope(x, [1, 2, 3, 4], [], None, 0.0, False, s)[:, 0] for x in (q, k))
    c, d = (K.norm_rope(x, [1, 2, 3, 4], [], None, 0.0, False, None)[:, 0] for x in (q, k))
    assert np.allclose(a @ b.T, c @ d.T)


# --------------------------------------------------------------------- ABI
@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def P(i):
    return ctypes.c_void_p(0x1000000 * (i + 1))                   # never dereferenced


def off(i, by):
    return ctypes.c_void_p(0x1000000 * (i + 1) + by)


def qk(lib, q=P(0), qt=512, qh=128, hq=4, k=P(1), kt=256, kh=128, hk=2, tokens=7, d=128, io=BF16, pos=P(2), wide=1,
       freqs=P(3), pairs=64, inter=0, gq=P(4), gk=P(5), eps=1e-6, signs=P(6), qo=P(7), qot=512, qoh=128, ko=P(8), kot=256,
       koh=128):
    return lib.harp_qk_norm_rope(q, qt, qh, hq, k, kt, kh, hk, tokens, d, io, pos, wide, freqs, pairs, inter, gq, gk, eps,
                                 signs, qo, qot, qoh, ko, kot, koh, None)


QK_BAD = [
    (dict(io=I8), UNSUP), (dict(io=F64), UNSUP), (dict(tokens=-1), BAD), (dict(tokens=(1 << 30) + 1), BAD),
    (dict(d=0), BAD), (dict(d=520, signs=None), BAD), (dict(d=100, signs=None, pairs=48), UNSUP), (dict(d=96, pairs=48), UNSUP),
    (dict(hq=0), BAD), (dict(hk=-1), BAD), (dict(hq=65536), BAD), (dict(pairs=65), BAD), (dict(pairs=-8), BAD),
    (dict(pairs=60), UNSUP), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(pos=None), BAD), (dict(freqs=None), BAD), (dict(qt=500), BAD), (dict(qh=127), BAD), (dict(qt=-512), BAD),
    (dict(qt=300, qh=200), BAD), (dict(q=off(0, 1)), BAD), (dict(pos=off(2, 4)), BAD), (dict(freqs=off(3, 4)), BAD),
    (dict(gq=off(4, 1)), BAD), (dict(hk=0), BAD), (dict(hk=0, k=None), BAD), (dict(qot=511), BAD)]
QK_APART = [
    (dict(qo=None), BAD), (dict(ko=None), BAD), (dict(qo=P(1)), BAD), (dict(ko=P(0)), BAD), (dict(ko=P(7)), BAD),
    (dict(qo=P(0), qot=1024), BAD), (dict(qo=off(0, 256)), BAD), (dict(qo=P(4)), BAD), (dict(qo=P(2)), BAD),
    (dict(ko=P(6)), BAD), (dict(qo=P(0), qt=1024, qh=256, qot=1024, qoh=128), BAD)]


@pytest.mark.parametrize("kw,status", QK_BAD + QK_APART)
def test_qk_norm_rope_rejects_on_host(lib, kw, status):
    assert qk(lib, **kw) == status
    assert lib.harp_last_error().decode()


def qk_vjp(lib, q=P(0), qt=512, qh=128, hq=4, k=P(1), kt=256, kh=128, hk=2, tokens=7, d=128, io=BF16, pos=P(2), wide=1,
           freqs=P(3), pairs=64, inter=0, gq=P(4), gk=P(5), eps=1e-6, signs=P(6), dyq=P(7), dyqt=512, dyqh=128, dyk=P(8),
           dykt=256, dykh=128, dq=P(9), dqt=512, dqh=128, dk=P(10), dkt=256, dkh=128, dgq=P(11), dgk=P(12), ws=P(13),
           wsb=1 << 22):
    return lib.harp_qk_norm_rope_vjp(q, qt, qh, hq, k, kt, kh, hk, tokens, d, io, pos, wide, freqs, pairs, inter, gq, gk,
                                     eps, signs, dyq, dyqt, dyqh, dyk, dykt, dykh, dq, dqt, dqh, dk, dkt, dkh, dgq, dgk, ws,
                                     wsb, None)


@pytest.mark.parametrize("kw,status", [x for x in QK_BAD if "qot" not in x[0]] + [
    (dict(dyq=None), BAD), (dict(dyk=None), BAD), (dict(dq=None), BAD), (dict(dk=None), BAD), (dict(dyqt=511), BAD),
    (dict(dqh=100), BAD), (dict(dq=P(8)), BAD), (dict(dk=P(9)), BAD), (dict(dq=P(1)), BAD), (dict(dq=off(7, 16)), BAD),
    (dict(dgq=P(12)), BAD), (dict(dgq=P(0)), BAD), (dict(dgk=P(9)), BAD), (dict(dgq=off(11, 2)), BAD), (dict(dgq=P(4)), BAD),
    (dict(ws=None), BAD), (dict(wsb=100), BAD), (dict(ws=off(13, 2)), BAD), (dict(ws=P(9)), BAD), (dict(ws=P(11)), BAD),
    (dict(ws=P(2)), BAD), (dict(hk=0, k=None, gk=None), BAD)])
def test_qk_norm_rope_vjp_rejects_on_host(lib, kw, status):
    assert qk_vjp(lib, **kw) == status
    assert lib.harp_last_error().decode()


CACHE = dict(kc=P(2), kcp=2 * 16 * 64, ks=P(3), ksp=2 * 16 * 4, vc=P(4), vcp=2 * 16 * 64, vs=P(5), vsp=2 * 16 * 4, pages=9,
             heads=2, ps=16, d=128)
PLAN = dict(starts=P(6), lengths=P(7), table=P(8), ldt=5, seqs=3, width=5)


def cache_args(kw):
    a = {**CACHE, **{k: v for k, v in kw.items() if k in CACHE}}
    return [a[k] for k in CACHE]


def plan_args(kw):
    a = {**PLAN, **{k: v for k, v in kw.items() if k in PLAN}}
    return [a[k] for k in PLAN]


def write(lib, k=P(0), kt=256, kh=128, v=P(1), vt=256, vh=128, tokens=7, io=BF16, **kw):
    return lib.harp_kv4_write(k, kt, kh, v, vt, vh, tokens, io, *cache_args(kw), *plan_args(kw), None)


def read(lib, k=P(0), kt=256, kh=128, v=P(1), vt=256, vh=128, tokens=7, io=BF16, **kw):
    return lib.harp_kv4_read(*cache_args(kw), *plan_args(kw), k, kt, kh, v, vt, vh, tokens, io, None)


def attention(lib, q=P(0), qt=512, qh=128, tokens=7, hq=4, scale=0.1, causal=1, window=0, out=P(1), ot=512, oh=128, lse=P(9),
              ws=P(10), wsb=1 << 23, **kw):
    return lib.harp_kv4_attention(q, qt, qh, tokens, hq, *cache_args(kw), *plan_args(kw), scale, causal, window, out, ot, oh,
                                  lse, ws, wsb, None)


CACHE_BAD = [
    (dict(kc=None), BAD), (dict(ks=None), BAD), (dict(vc=None), BAD), (dict(vs=None), BAD), (dict(kc=off(2, 8)), BAD),
    (dict(vs=off(5, 4)), BAD), (dict(kcp=2 * 16 * 64 - 16), BAD), (dict(vsp=2 * 16 * 4 + 8), BAD), (dict(pages=0), BAD),
    (dict(pages=(1 << 30) + 1), BAD), (dict(heads=0), BAD), (dict(heads=65536), BAD), (dict(ps=8), BAD), (dict(ps=24), UNSUP),
    (dict(ps=1 << 21), BAD), (dict(d=48), UNSUP), (dict(d=288), BAD), (dict(d=0), BAD), (dict(seqs=-1), BAD),
    (dict(seqs=(1 << 24) + 1), BAD), (dict(width=0), BAD), (dict(width=(1 << 24) + 1), BAD), (dict(ldt=4), BAD),
    (dict(starts=None), BAD), (dict(lengths=None), BAD), (dict(table=None), BAD), (dict(starts=off(6, 2)), BAD),
    (dict(seqs=1 << 24, heads=128, kcp=1 << 40, ksp=1 << 40, vcp=1 << 40, vsp=1 << 40), BAD), (dict(kcp=1 << 62), BAD)]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(io=I8), UNSUP), (dict(tokens=-1), BAD), (dict(tokens=(1 << 30) + 1), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(kt=255), BAD), (dict(vh=64), BAD), (dict(v=off(1, 1)), BAD), (dict(k=P(2)), BAD), (dict(kc=P(3)), BAD),
    (dict(kc=P(6)), BAD), (dict(vs=P(8)), BAD), (dict(vc=P(2)), BAD)])
def test_kv4_write_rejects_on_host(lib, kw, status):
    assert write(lib, **kw) == status
    assert lib.harp_last_error().decode()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(io=F64), UNSUP), (dict(tokens=-1), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(kt=255), BAD),
    (dict(vh=64), BAD), (dict(v=P(0)), BAD), (dict(k=P(2)), BAD), (dict(v=P(8)), BAD)])
def test_kv4_read_rejects_on_host(lib, kw, status):
    assert read(lib, **kw) == status
    assert lib.harp_last_error().decode()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(tokens=-1), BAD), (dict(tokens=1 << 29), BAD), (dict(hq=3), BAD), (dict(hq=0), BAD), (dict(scale=0.0), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(window=-1), BAD),
    (dict(window=1 << 31), BAD), (dict(q=None), BAD), (dict(out=None), BAD), (dict(qt=511), BAD), (dict(oh=127), BAD),
    (dict(out=P(0)), BAD), (dict(out=P(3)), BAD), (dict(out=P(7)), BAD), (dict(lse=P(1)), BAD), (dict(lse=P(0)), BAD),
    (dict(lse=off(9, 2)), BAD)])
def test_kv4_attention_rejects_on_host(lib, kw, status):
    assert attention(lib, **kw) == status
    assert lib.harp_last_error().decode()


def test_attention_rejects_short_workspaces(lib):
    kw = dict(width=4096, ldt=4096)
    need = lib.harp_kv4_attention_workspace(7, 4, 2, 128, 16, 3, 4096)
    assert need > 0
    for more in (dict(ws=None), dict(wsb=need - 1), dict(ws=off(10, 8)), dict(ws=P(9)), dict(ws=P(2)), dict(ws=P(1))):
        assert attention(lib, **{**kw, "wsb": need, **more}) == BAD
        assert lib.harp_last_error().decode()


def test_sizes_out_of_range(lib):
    fn = lib.harp_kv4_attention_workspace
    good = (7, 8, 2, 128, 16, 3, 5)
    assert fn(*good) >= 0
    for i, bad in ((0, -1), (0, 1 << 30), (1, 7), (1, 0), (2, 0), (3, 48), (3, 288), (4, 8), (4, 24), (5, -1), (5, 1 << 30),
                   (6, 0)):
        args = list(good)
        args[i] = bad
        assert fn(*args) == -1, (i, bad)
    fn = lib.harp_qk_norm_rope_vjp_workspace
    assert fn(0, 1, 0, 8) == 0 and fn(5, 4, 2, 128) > 0
    for args in ((-1, 1, 1, 64), (1, 0, 1, 64), (1, 1, -1, 64), (1, 1, 1, 60), (1, 1, 1, 520), (1 << 31, 1, 1, 64)):
        assert fn(*args) == -1


def test_nothing_to_do_is_a_noop(lib):
    assert qk(lib, tokens=0, q=None, k=None, qo=None, ko=None) == OK
    assert qk_vjp(lib, tokens=0, dgq=None, dgk=None, q=None, k=None, dyq=None, dyk=None, dq=None, dk=None, ws=None) == OK
    for call in (write, read):
        assert call(lib, tokens=0, k=None, v=None, kc=None) == OK
        assert call(lib, seqs=0) == OK
    assert attention(lib, tokens=0, q=None, out=None) == OK and attention(lib, seqs=0) == OK


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
    real = kv4.lib()
    monkeypatch.setattr(kv4, "lib", lambda: _Guard(real))


BF = torch.bfloat16


def heads(t, h, d=128, dtype=BF):
    return torch.zeros(t, h, d, dtype=dtype)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def plan(n=3, width=5, tokens=7):
    return torch.linspace(0, tokens, n + 1).int(), torch.full((n,), 40, dtype=torch.int32), torch.zeros(n, width, dtype=torch.int32)


def cache(**kw):
    return kv4.harp_kv4_cache(**{**dict(pages=9, kv_heads=2, page_size=16, d=128, device="cpu"), **kw})


def gpu_only(fn):
    with pytest.raises(TypeError, match="GPU tensor"):
        fn()


def refuses(exc, match, fn):
    with pytest.raises(exc, match=match):
        fn()


def test_cache_sizes():
    c = cache()
    assert c.k_codes.shape == c.v_codes.shape == (9, 2, 16, 64) and c.k_codes.dtype == torch.uint8
    assert c.k_scales.shape == c.v_scales.shape == (9, 2, 16, 4) and c.v_scales.dtype == torch.float8_e8m0fnu
    for kw in (dict(pages=0), dict(kv_heads=0), dict(page_size=24), dict(page_size=8), dict(d=48), dict(d=288), dict(d=0)):
        refuses(ValueError, "must be", lambda kw=kw: cache(**kw))


def test_qk_norm_rope_checks(guard):
    g, s, f, p = torch.ones(128, dtype=BF), torch.ones(128, dtype=torch.int8), torch.zeros(64, dtype=torch.float64), torch.arange(7)

    def call(q=heads(7, 4), k=heads(7, 2), p=p, f=f, gq=g, gk=g, signs=s, **kw):
        return kv4.harp_qk_norm_rope(q, k, p, f, gq, gk, signs=signs, **kw)

    gpu_only(call)
    gpu_only(lambda: call(k=None, gk=None))
    gpu_only(lambda: call(f=None, p=None))
    gpu_only(lambda: call(q=heads(7, 8)[:, 2:6], p=p.int()))
    refuses(TypeError, "q must be", lambda: call(q=heads(7, 4, dtype=torch.float16)))
    refuses(TypeError, "k must be", lambda: call(k=heads(7, 2, dtype=torch.float32)))
    refuses(TypeError, "tensor", lambda: call(q=[1.0]))
    refuses(ValueError, "tokens x heads x d", lambda: call(q=heads(7, 4)[0]))
    refuses(ValueError, "k must be", lambda: call(k=heads(6, 2)))
    refuses(ValueError, "k must be", lambda: call(k=heads(7, 2, 64)))
    refuses(ValueError, "contiguous", lambda: call(q=heads(7, 128, 128).transpose(1, 2)))
    refuses(ValueError, "no heads", lambda: call(q=heads(7, 0)))
    refuses(TypeError, "positions", lambda: call(p=torch.zeros(7)))
    refuses(TypeError, "positions", lambda: call(p=None))
    refuses(ValueError, "positions", lambda: call(p=torch.arange(6)))
    refuses(TypeError, "freqs", lambda: call(f=f.float()))
    refuses(ValueError, "freqs", lambda: call(f=torch.zeros(65, dtype=torch.float64)))
    refuses(ValueError, "freqs", lambda: call(f=f.view(8, 8)))
    refuses(ValueError, "gamma_q", lambda: call(gq=g[:64]))
    refuses(TypeError, "gamma_k", lambda: call(gk=g.float()))
    refuses(ValueError, "gamma_k", lambda: call(k=None))
    refuses(TypeError, "signs", lambda: call(signs=g))
    refuses(ValueError, "signs", lambda: call(signs=s[:64]))
    refuses(ValueError, "q_out", lambda: call(q_out=heads(7, 3)))
    refuses(TypeError, "k_out", lambda: call(k_out=heads(7, 2, dtype=torch.float32)))
    refuses(ValueError, "k_out", lambda: call(k=None, gk=None, k_out=heads(7, 2)))


def test_qk_norm_rope_vjp_checks(guard):
    g, f, p = torch.ones(128, dtype=BF), torch.zeros(64, dtype=torch.float64), torch.arange(7)

    def call(dyq=heads(7, 4), dyk=heads(7, 2), k=heads(7, 2), gk=g, **kw):
        return kv4.harp_qk_norm_rope_vjp(heads(7, 4), k, p, f, dyq, dyk, g, gk, **kw)

    gpu_only(call)
    gpu_only(lambda: call(dyk=None, k=None, gk=None))
    refuses(ValueError, "dq_out", lambda: call(dyq=heads(7, 3)))
    refuses(TypeError, "tensor", lambda: call(dyk=None))
    refuses(TypeError, "dk_out", lambda: call(dyk=heads(7, 2, dtype=torch.float32)))
    refuses(ValueError, "with k only", lambda: call(k=None, gk=None))
    refuses(ValueError, "dq must be", lambda: call(dq=heads(6, 4)))
    refuses(ValueError, "dgamma_q", lambda: call(dgamma_q=torch.zeros(64)))
    refuses(TypeError, "dgamma_k", lambda: call(dgamma_k=torch.zeros(128, dtype=BF)))
    refuses(ValueError, "want_dgamma", lambda: call(want_dgamma=False, dgamma_q=torch.zeros(128)))


def test_cache_checks(guard):
    def call(c=cache(), k=heads(7, 2), v=heads(7, 2), pl=plan()):
        return kv4.harp_kv4_write(k, v, c, *pl)

    gpu_only(call)
    both = torch.zeros(9, 2, 2, 16, 64, dtype=torch.uint8)                        # keys and values of a page side by side
    gpu_only(lambda: call(cache()._replace(k_codes=both[:, 0], v_codes=both[:, 1])))
    refuses(TypeError, "k_codes", lambda: call(cache()._replace(k_codes=both[:, 0].to(torch.int8))))
    refuses(TypeError, "v_scales", lambda: call(cache()._replace(v_scales=cache().v_scales.view(torch.uint8))))
    refuses(ValueError, "v_codes", lambda: call(cache()._replace(v_codes=both[:8, 0])))
    refuses(ValueError, "k_scales", lambda: call(cache()._replace(k_scales=cache(d=64).k_scales)))
    refuses(ValueError, "k_codes", lambda: call(cache()._replace(k_codes=both)))
    refuses(ValueError, "contiguous", lambda: call(cache()._replace(v_codes=both.transpose(2, 3)[:, 0].contiguous().transpose(1, 2))))
    refuses(ValueError, "cache holds", lambda: call(k=heads(7, 4), v=heads(7, 4)))
    refuses(ValueError, "cache holds", lambda: call(k=heads(7, 2, 64), v=heads(7, 2, 64)))
    refuses(ValueError, "v must be", lambda: call(v=heads(6, 2)))
    refuses(TypeError, "v must be", lambda: call(v=heads(7, 2, dtype=torch.float32)))
    refuses(TypeError, "starts", lambda: call(pl=(plan()[0].long(), *plan()[1:])))
    refuses(ValueError, "starts must have 4", lambda: call(pl=(plan()[0][:3], *plan()[1:])))
    refuses(ValueError, "table", lambda: call(pl=(*plan()[:2], plan()[2][:2])))
    refuses(ValueError, "dimension", lambda: call(pl=(*plan()[:2], plan()[2][0])))
    refuses(ValueError, "no columns", lambda: call(pl=(*plan()[:2], plan()[2][:, :0])))
    refuses(ValueError, "contiguous", lambda: call(pl=(*plan()[:2], plan(5, 3)[2].t())))
    gpu_only(lambda: call(pl=(*plan()[:2], plan(3, 9)[2][:, :5])))


def test_read_and_attention_checks(guard):
    def rd(tokens=7, out="bf16", **kw):
        return kv4.harp_kv4_read(cache(), *plan(), tokens, out, **kw)

    gpu_only(rd)
    refuses(ValueError, "out must be", lambda: rd(out="f16"))
    refuses(ValueError, "tokens", lambda: rd(-1))
    refuses(ValueError, "k must be", lambda: rd(k=heads(6, 2)))
    refuses(TypeError, "v must be", lambda: rd(out="f32", v=heads(7, 2)))

    def at(q=heads(7, 4), **kw):
        return kv4.harp_kv4_attention(q, cache(), *plan(), **kw)

    gpu_only(at)
    gpu_only(lambda: at(lse=True, window=3, causal=False))
    refuses(TypeError, "q must be", lambda: at(heads(7, 4, dtype=torch.float32)))
    refuses(ValueError, "multiple", lambda: at(heads(7, 3)))
    refuses(ValueError, "cache holds", lambda: at(heads(7, 4, 64)))
    refuses(ValueError, "out must be", lambda: at(out=heads(7, 3)))
    refuses(TypeError, "lse", lambda: at(lse=torch.zeros(7, 4, dtype=BF)))
    refuses(ValueError, "lse", lambda: at(lse=torch.zeros(4, 7).t()))
    refuses(ValueError, "lse", lambda: at(lse=torch.zeros(7, 3)))


# ------------------------------------------------- streams, devices and memory
_empty = torch.empty


def meta(*shape, dtype=torch.float32):
    return _empty(shape, dtype=dtype, device="meta")


def fake_stream(handle, gpu=0):
    return SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", gpu))


class _Lib:
    def __init__(self, real, log):
        self._real, self._log = real, log

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return getattr(self._real, name)

        def entry(*a):
            self._log.launched.append((self._log.gpu, a[-1]))
            return 0
        return entry


@pytest.fixture
def calls(monkeypatch):
    log = SimpleNamespace(active=None, made=[], recorded=[], launched=[], gpu=0, tensors_on=0)

    @contextlib.contextmanager
    def on(stream):
        before, log.active = log.active, stream
        yield
        log.active = before

    @contextlib.contextmanager
    def device(gpu):
        before, log.gpu = log.gpu, gpu
        yield
        log.gpu = before

    def logged(*a, **k):
        t = _empty(*a, **k)
        log.made.append((t, log.active))
        return t

    real = kv4.lib()
    here = fake_stream(7)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: here)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_streams, "_current_device", lambda: log.gpu, raising=False)
    monkeypatch.setattr(_streams, "_current_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch, "empty", logged)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.recorded.append((t, s)))
    monkeypatch.setattr(kv4, "lib", lambda: _Lib(real, log))
    monkeypatch.setattr(kv4, "_on_gpu", lambda *t: log.tensors_on)
    log.here = here
    return log


def _meta_cache():
    e8 = torch.float8_e8m0fnu
    return kv4.Cache4(meta(9, 2, 16, 64, dtype=torch.uint8), meta(9, 2, 16, 4, dtype=e8), meta(9, 2, 16, 64, dtype=torch.uint8),
                      meta(9, 2, 16, 4, dtype=e8))


def _meta_plan():
    return meta(4, dtype=torch.int32), meta(3, dtype=torch.int32), meta(3, 4096, dtype=torch.int32)


def norm_call(stream):
    q, k, p, f = meta(7, 4, 128), meta(7, 2, 128), meta(7, dtype=torch.int64), meta(64, dtype=torch.float64)
    return (q, k, p, f), kv4.harp_qk_norm_rope(q, k, p, f, stream=stream), 2


def norm_vjp_call(stream):
    q, k, p, f, g = meta(7, 4, 128), meta(7, 2, 128), meta(7, dtype=torch.int64), meta(64, dtype=torch.float64), meta(128)
    return (q, k, p, f, g), kv4.harp_qk_norm_rope_vjp(q, k, p, f, q, k, g, g, stream=stream), 5


def write_call(stream):
    k, c, pl = meta(7, 2, 128), _meta_cache(), _meta_plan()
    kv4.harp_kv4_write(k, k, c, *pl, stream=stream)
    return (k, *c, *pl), (), 0


def read_call(stream):
    c, pl = _meta_cache(), _meta_plan()
    return (*c, *pl), kv4.harp_kv4_read(c, *pl, 7, stream=stream), 2


def attention_call(stream):
    q, c, pl = meta(7, 4, 128, dtype=BF), _meta_cache(), _meta_plan()
    return (q, *c, *pl), kv4.harp_kv4_attention(q, c, *pl, lse=True, stream=stream), 3


CALLS = [norm_call, norm_vjp_call, write_call, read_call, attention_call]


@pytest.mark.parametrize("call", CALLS)
def test_an_explicit_stream_allocates_and_is_recorded(calls, call):
    s = fake_stream(99)
    inputs, outputs, made = call(s)
    assert len(calls.made) == made and all(active is s for _, active in calls.made)
    told = {(id(t), st.cuda_stream) for t, st in calls.recorded}
    for t in [*inputs, *outputs, *(t for t, _ in calls.made)]:
        assert (id(t), 99) in told and (id(t), 7) in told


@pytest.mark.parametrize("call", CALLS)
def test_a_call_goes_to_its_tensors_gpu(calls, call):
    calls.tensors_on = 1                                          # while GPU 0 is the current one
    call(None)
    call(fake_stream(99, 1))
    with pytest.raises(ValueError, match="stream is on GPU 0"):
        call(fake_stream(99, 0))
    assert list(dict.fromkeys(calls.launched)) == [(1, 101), (1, 99)] and calls.gpu == 0
