"""The 8-bit layer (structured_rotations_amd/linear8.py): its operators
together, forward and backward, for a batch and for one token.

Two comparisons.  Against fp64 from the same stored codes and checkpoints only
the roundings between the operators differ: bf16 rows between them (2^-8 each
at most, three in a row) and, backward, the coding of the gradient rows.
Against the layer without any rounding the coded operands count: an E4M3 code
is off by at most 2^-4 of its value (rms below 2^-5), two operands add in
squares, so 2 * 2^-5 bounds the relative l2 error of a product.
"""
import numpy as np
import pytest
import torch

from oracle import harp_oracle as O
from oracle import q8_oracle as Q
from structured_rotations_amd import linear8 as L

pytestmark = pytest.mark.gpu


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes_np(t):
    return t.view(torch.uint8).cpu().numpy()


def scales_np(t):
    return t.cpu().numpy() if t.dtype == torch.float32 else Q.e8m0(t.view(torch.uint8).cpu().numpy())


def dense(p):
    """A processor's matrix in fp64: rows of the transform of the identity."""
    eye = torch.eye(p.d, device="cuda")
    return np64(L.api.harp_apply(p.schedule, p.d, p.blocks, p.scales, p.signs, eye)).T


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("rows", [1, 300])
def test_layer(rows, kind):
    print("\n[case] linear8", rows, kind, flush=True)
    n, k, eps = 640, 512, 1e-6
    u, v = L.random_processor((8, 8, 5, 2), n, 1), L.random_processor((8, 8, 8), k, 2)
    rng = np.random.default_rng(3)
    w = torch.from_numpy((rng.standard_normal((n, k)) * 0.02).astype(np.float32)).cuda()
    gamma = torch.from_numpy((1 + 0.2 * rng.standard_normal(k)).astype(np.float32)).cuda()
    x = rng.standard_normal((rows, k)).astype(np.float32)
    res = rng.standard_normal((rows, k)).astype(np.float32)
    x[:, ::97] *= 50
    bf = torch.bfloat16
    layer = L.Linear8(w, u, v, gamma, eps, kind, backward=True)
    xr, rr = v.apply(torch.from_numpy(x).cuda()).to(bf), v.apply(torch.from_numpy(res).cuda()).to(bf)
    y, h, ckpt = layer.forward(xr, rr, checkpoint=True)
    dy = torch.from_numpy(rng.standard_normal((rows, n)).astype(np.float32)).cuda().to(bf)
    dh = torch.from_numpy((rng.standard_normal((rows, k)) * 0.1).astype(np.float32)).cuda().to(bf)
    dx, dw = layer.backward(dy, ckpt, dh)
    torch.cuda.synchronize()
    mu, mv = dense(u), dense(v)

    # from what is stored
    xc, xs, rstd = codes_np(ckpt[0]), scales_np(ckpt[1]), np64(ckpt[2])
    wt = Q.dequantize(codes_np(layer.codes), scales_np(layer.scales), 128)
    xn = Q.dequantize(xc, xs)
    assert rel(np64(y), xn @ wt.T @ mu) <= 3 * 2.0 ** -8
    dyr = np64(dy) @ mu.T
    assert rel(np64(dw), dyr.T @ xn) <= 2.0 ** -8
    want_dx, _ = Q.rmsnorm_vjp(xn, rstd, dyr @ wt, None, np64(dh))
    assert rel(np64(dx), want_dx) <= 2.0 ** -5 + 3 * 2.0 ** -8

    # from the layer itself
    hh = x.astype(np.float64) + res
    hn = hh / np.sqrt(np.mean(hh * hh, axis=1, keepdims=True) + eps)
    assert rel(np64(y), (hn * np64(gamma)) @ np64(w).T) <= 2 * 2.0 ** -5
    assert rel(np64(h), hh @ mv.T) <= 2 * 2.0 ** -8


def test_demo_runs(capsys):
    print("\n[case] linear8 demo", flush=True)
    assert L.main() == 0
    assert "rotated" in capsys.readouterr().out


def test_dense_helper_matches_the_oracle():
    p = L.random_processor((8, 8, 5, 2), 640, 1)
    blocks = [b for b in np.split(np64(p.blocks), np.cumsum([640 * r for r in p.schedule])[:-1])]
    blocks = [b.reshape(640 // r, r, r) for b, r in zip(blocks, p.schedule)]
    x = np.random.default_rng(5).standard_normal((3, 640))
    want = O.apply(x, p.schedule, blocks, p.signs.cpu().numpy().astype(float))
    assert rel(x @ dense(p).T, want) <= 1e-5
