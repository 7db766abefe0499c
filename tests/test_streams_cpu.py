"""Host-side tests (no GPU needed) of what a call with an explicit stream does
with memory: everything it makes is allocated on that stream, and the allocator
is told that the stream and the current one use the call's tensors; and of the
GPU that a call goes to.

Meta tensors take the GPU ones' place, and recorders the library's and torch's.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from structured_rotations_amd import _streams, api, q8

E4 = torch.float8_e4m3fn


_empty = torch.empty


def meta(*shape, dtype=torch.float32):
    return _empty(shape, dtype=dtype, device="meta")


def fake_stream(handle, gpu=0):
    return SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", gpu))


class _Lib:
    """The real library's size helpers; every entry point succeeds."""

    def __init__(self, real, log):
        self._real, self._log = real, log

    def __getattr__(self, name):
        if name.endswith(("_workspace", "_count")):
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

    def logged(*a, **k):
        t = _empty(*a, **k)
        log.made.append((t, log.active))
        return t

    def like(t):
        return logged(t.shape, dtype=t.dtype, device=t.device)

    @contextlib.contextmanager
    def device(gpu):
        before, log.gpu = log.gpu, gpu
        yield
        log.gpu = before

    real = q8.lib()
    here = fake_stream(7)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: here)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_streams, "_current_device", lambda: log.gpu, raising=False)
    monkeypatch.setattr(_streams, "_current_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch, "empty", logged)
    monkeypatch.setattr(torch, "empty_like", like)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.recorded.append((t, s)))
    for binding in (q8, api):
        monkeypatch.setattr(binding, "lib", lambda: _Lib(real, log))
    monkeypatch.setattr(q8, "_on_gpu", lambda *t: log.tensors_on)
    monkeypatch.setattr(api, "_on_gpu", lambda **t: ([v for v in t.values() if v is not None], log.tensors_on),
                        raising=False)
    log.here = here
    return log


def quantize(stream):
    x = meta(200, 300)
    return (x,), q8.harp_quantize_q8(x, stream=stream), 2


def norm(stream):
    x, g = meta(200, 300), meta(300)
    return (x, g), q8.harp_rmsnorm_q8(x, x, g, checkpoint=True, stream=stream), 6


def norm_vjp(stream):
    dn, c, s, r = meta(200, 300), meta(200, 300, dtype=E4), meta(200, 3), meta(200)
    return (dn, c, s, r), q8.harp_rmsnorm_q8_vjp(c, s, r, dn, want_dgamma=True, stream=stream), 3


def matmul(stream):
    a, sa, w, sw = meta(128, 4096, dtype=E4), meta(128, 32), meta(128, 4096, dtype=E4), meta(1, 32)
    return (a, sa, w, sw), (q8.harp_matmul_q8(a, sa, w, sw, stream=stream),), 2


def wgrad(stream):
    dy, x, s = meta(4096, 128, dtype=torch.bfloat16), meta(4096, 128, dtype=E4), meta(4096, 1)
    return (dy, x, s), (q8.harp_matmul_q8_wgrad(dy, x, s, stream=stream),), 2


SCH, D = (8, 8, 8), 512


def blocks():
    return meta(api.harp_block_count(SCH, D))


def materialize(stream):
    th = meta(api.harp_theta_count(SCH, D), dtype=torch.float64)
    out = api.harp_materialize_blocks(SCH, D, th, None, "i8", stream=stream)
    codes = api.harp_quantize_theta(SCH, D, th, stream=stream)
    more = api.harp_materialize_blocks_q8(SCH, D, *codes, None, "i8", stream=stream)
    return (th,), (*out, *codes, *more), 6


def apply(stream):
    b, x = blocks(), meta(5, D)
    return (b, x), (api.harp_apply(SCH, D, b, None, None, x, stream=stream),
                    api.harp_apply_inverse(SCH, D, b, None, None, x, stream=stream),
                    api.harp_apply_decode(SCH, D, b, None, None, x, stream=stream)), None


def apply_vjp(stream):
    b, x, dy = blocks(), meta(5, D), meta(5, D)
    return (b, x, dy), api.harp_apply_vjp(SCH, D, b, None, None, x, dy, stream=stream), 3


def theta_vjp(stream):
    th, db = meta(api.harp_theta_count(SCH, D), dtype=torch.float64), blocks()
    return (th, db), (api.harp_theta_vjp(SCH, D, th, None, db, stream=stream),), 1


def rotate(stream):
    b, w = blocks(), meta(D, D)
    return (b, w), (api.harp_rotate_weight(SCH, b, None, None, SCH, b, None, None, w, stream=stream),), 2


def rht(stream):
    signs, x = meta(2, D, dtype=torch.int8), meta(5, D)
    return (signs, x), (api.rht_compose(SCH, D, signs, x, stream=stream),), 1


CALLS = [quantize, norm, norm_vjp, matmul, wgrad, materialize, apply, apply_vjp, theta_vjp, rotate, rht]


@pytest.mark.parametrize("call", CALLS)
def test_an_explicit_stream_allocates_and_is_recorded(calls, call):
    s = fake_stream(99)
    inputs, outputs, made = call(s)
    assert made is None or len(calls.made) == made                # results, and a workspace where one is needed
    assert all(active is s for _, active in calls.made)
    told = {(id(t), st.cuda_stream) for t, st in calls.recorded}
    for t in [*inputs, *outputs, *(t for t, _ in calls.made)]:
        assert (id(t), 99) in told and (id(t), 7) in told


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_needs_no_record(calls, call):
    call(calls.here)
    assert not calls.recorded
    assert all(active is calls.here for _, active in calls.made)


@pytest.mark.parametrize("call", CALLS)
def test_a_call_goes_to_its_tensors_gpu(calls, call):
    calls.tensors_on = 1                                          # while GPU 0 is the current one
    call(None)
    call(fake_stream(99, 1))
    calls.tensors_on = 0
    call(None)
    assert list(dict.fromkeys(calls.launched)) == [(1, 101), (1, 99), (0, 100)] and calls.gpu == 0


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_gpu_is_refused(calls, call):
    calls.tensors_on = 1
    with pytest.raises(ValueError, match="stream is on GPU 0"):
        call(fake_stream(99, 0))
    assert not calls.launched


def test_arguments_on_two_gpus_are_refused():
    a, b = (SimpleNamespace(get_device=lambda i=i: i) for i in (0, 1))
    with pytest.MonkeyPatch.context() as m:
        m.setattr(api, "_dev", lambda t, name: None)
        assert api._on_gpu(x=a, y=None, z=a) == ([a, a], 0)
        with pytest.raises(ValueError, match="different GPUs"):
            api._on_gpu(x=a, y=b)
    with pytest.raises(ValueError, match="different GPUs"):
        q8._on_gpu(a, None, b)
