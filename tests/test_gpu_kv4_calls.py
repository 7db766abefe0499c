"""Attention over a 4-bit cache as programs call it: arrays at any place, all of
a cache in one buffer, calls on two streams at once, graphs that share a
workspace.  What is compared is the same work called another way: the same bits.
"""
import numpy as np
import pytest
import torch

from structured_rotations_amd import kv4

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def say(*a):
    print("\n[case]", *a, flush=True)


def case(lengths, new, hq, heads, d, page, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = kv4.harp_kv4_cache(pages, heads, page, d)
    for t, lo, hi in zip(cache, (0, 124, 0, 124), (256, 129, 256, 129)):
        t.view(torch.uint8).copy_(torch.randint(lo, hi, t.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8))
    starts = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").to(BF)
    return q, cache, (starts, torch.tensor(lengths, dtype=torch.int32, device="cuda"), table)


SHAPES = [([700, 33, 250], [1, 1, 1], 8, 2, 128, 16), ([700, 33, 250], [5, 6, 7], 8, 2, 96, 32), ([700, 40], [200, 37], 8, 4, 64, 16),
          ([300, 40], [100, 37], 4, 1, 160, 16)]


@pytest.mark.parametrize("shape", SHAPES, ids=["1", "6", "100", "100x160"])
def test_arrays_at_any_place(shape):
    say("odd places", *shape)
    q, cache, plan = case(*shape)
    want, lse = kv4.harp_kv4_attention(q, cache, *plan, lse=True)
    n, h, d = q.shape
    buf = torch.full((n * (h * (d + 1) + 3) + 1,), 7.0, dtype=BF, device="cuda")
    odd = buf[1:].view(n, -1)[:, :h * (d + 1)].unflatten(1, (h, d + 1))[..., :d]      # one element off, odd distances
    odd.copy_(q)
    to = torch.full_like(buf, 7.0)
    out = to[1:].view(n, -1)[:, :h * (d + 1)].unflatten(1, (h, d + 1))[..., :d]
    lbuf = torch.full((n * h + 3,), 7.0, device="cuda")
    kv4.harp_kv4_attention(odd, cache, *plan, out=out, lse=lbuf[1:-2].view(n, h))
    assert torch.equal(out, want) and torch.equal(lbuf[1:-2].view(n, h), lse)
    out.fill_(7.0)                                            # nothing between heads and tokens has changed
    assert bool((to == 7).all()) and bool((lbuf[[0, -2, -1]] == 7).all())
    # a plan whose table is a part of a wider one, and longer
    wide = torch.full((plan[2].shape[0] + 2, plan[2].shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide[1:-1, 2:-3] = plan[2]
    again = kv4.harp_kv4_attention(q, cache, plan[0], plan[1], wide[1:-1, 2:-3])
    assert torch.equal(again, want)


@pytest.mark.parametrize("shape", SHAPES[:3], ids=["1", "6", "100"])
def test_a_cache_in_one_buffer(shape):
    """Pages of several layers, each with its keys' codes and scales and its
    values' one behind the other."""
    say("one buffer", *shape)
    q, cache, plan = case(*shape)
    pages, heads, page, half = cache.k_codes.shape
    sizes = [heads * page * half, heads * page * half // 16] * 2
    layers = 3
    buf = torch.full((pages, layers, sum(sizes)), 255, dtype=torch.uint8, device="cuda")
    ends = np.cumsum([0] + sizes)
    one = kv4.Cache4(*(buf[:, 1, a:b].unflatten(1, (heads, page, t.shape[3])).view(t.dtype) for a, b, t in zip(ends, ends[1:], cache)))
    for t, x in zip(one, cache):
        t.view(torch.uint8).copy_(x.view(torch.uint8))
    assert torch.equal(kv4.harp_kv4_attention(q, one, *plan), kv4.harp_kv4_attention(q, cache, *plan))
    k, v = (torch.randn(q.shape[0], heads, q.shape[2], device="cuda") for _ in range(2))
    kv4.harp_kv4_write(k, v, one, *plan)
    kv4.harp_kv4_write(k, v, cache, *plan)
    for t, x in zip(one, cache):
        assert torch.equal(t.view(torch.uint8), x.view(torch.uint8))
    for a, b in zip(kv4.harp_kv4_read(one, *plan, len(k)), kv4.harp_kv4_read(cache, *plan, len(k))):
        assert torch.equal(a, b)
    assert bool((buf[:, [0, 2]] == 255).all())                # the other layers


def test_calls_on_two_streams_at_once():
    say("two streams")
    cases = [case(*s, seed=i) for i, s in enumerate(SHAPES)]
    want = [kv4.harp_kv4_attention(q, c, *p, lse=True) for q, c, p in cases]
    read = [kv4.harp_kv4_read(c, *p, len(q)) for q, c, p in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for turn in range(6):
        for i, (q, c, p) in enumerate(cases):
            s = streams[(i + turn) % 2]
            got.append((i, kv4.harp_kv4_attention(q, c, *p, lse=True, stream=s), kv4.harp_kv4_read(c, *p, len(q), stream=s)))
    torch.cuda.synchronize()
    for i, a, k in got:
        assert torch.equal(a[0], want[i][0]) and torch.equal(a[1], want[i][1])
        assert torch.equal(k[0], read[i][0]) and torch.equal(k[1], read[i][1])


def test_two_graphs_that_share_a_workspace():
    """Replayed one after the other, in any order, with other work between them;
    what the workspace held does not matter."""
    say("two graphs")
    cases = [case(*s, seed=i) for i, s in enumerate(SHAPES)]
    need = [kv4.harp_kv4_attention_workspace(len(q), q.shape[1], c.k_codes.shape[1], q.shape[2], c.k_codes.shape[2], *p[2].shape)
            for q, c, p in cases]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graphs, held = [], []
    for q, c, p in cases:
        kv4.harp_kv4_attention(q, c, *p, lse=True, workspace=ws, stream=side)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            held.append(kv4.harp_kv4_attention(q, c, *p, lse=True, workspace=ws))
    rng = np.random.default_rng(0)
    for turn in range(12):
        i = int(rng.integers(0, len(cases)))
        q, c, p = cases[i]
        q.copy_(torch.randn_like(q.float()).to(BF))
        want = kv4.harp_kv4_attention(q, c, *p, lse=True)
        ws.fill_(int(rng.integers(0, 256)))
        graphs[i].replay()
        if turn % 3 == 0:
            torch.cuda.synchronize()
        assert torch.equal(held[i][0], want[0]) and torch.equal(held[i][1], want[1])
