"""A linear layer kept in rotated coordinates and 8 bits.

W (n x k) is used behind a root-mean-square norm with weight gamma:
y = W diag(gamma) norm(h), h = x + residual.  With the input processor M_V
(harp_apply) and the output processor M_U,

    W~ = M_U W diag(gamma) M_V^T,    y = M_U^T W~ norm(M_V h),

since a norm without weight commutes with an orthogonal M_V.  A stream of
hidden states that is kept rotated (M_V h) therefore goes from the norm's
8-bit output straight into the 8-bit product, and its blocks of 128 hold no
outlier channels.  The norm's 8-bit rows are also all that the backward pass
needs of the forward pass, with one number per row.

    python -m structured_rotations_amd.linear8      # a small layer against fp32
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import api, q8


@dataclass
class Processor:
    """A rotation of rows of length d (harp_materialize_blocks' output)."""
    schedule: tuple
    d: int
    blocks: torch.Tensor
    scales: Optional[torch.Tensor]
    signs: Optional[torch.Tensor]

    def apply(self, x, inverse: bool = False):
        fn = api.harp_apply_decode if x.shape[0] <= 128 else (api.harp_apply_inverse if inverse else api.harp_apply)
        kw = {"inverse": inverse} if fn is api.harp_apply_decode else {}
        return fn(self.schedule, self.d, self.blocks, self.scales, self.signs, x, **kw)


class Linear8:
    """The layer's stored form: coded W~ and, for the backward pass, its
    transpose (the same codes and scales, transposed)."""

    def __init__(self, weight, out_proc: Processor, in_proc: Processor, gamma=None, eps: float = 1e-6,
                 scale_dtype: str = "e8m0", backward: bool = False):
        self.out_proc, self.in_proc, self.eps, self.scale_dtype = out_proc, in_proc, eps, scale_dtype
        w = weight if gamma is None else (weight.float() * gamma.float()).to(weight.dtype)
        u, v = out_proc, in_proc
        w = api.harp_rotate_weight(u.schedule, u.blocks, u.scales, u.signs, v.schedule, v.blocks, v.scales, v.signs, w)
        self.codes, self.scales = q8.harp_quantize_q8(w, q8.BLOCK, scale_dtype)
        if backward:
            self.codes_t = self.codes.view(torch.uint8).t().contiguous().view(self.codes.dtype)
            self.scales_t = self.scales.view(torch.uint8 if scale_dtype == "e8m0" else torch.float32).t().contiguous() \
                .view(self.scales.dtype)

    def forward(self, x, residual=None, checkpoint: bool = False):
        """x, residual: rotated rows (bf16).  Returns (y, h, checkpoint): the
        layer's output, the rotated sum, and what backward needs (or None)."""
        n = q8.harp_rmsnorm_q8(x, residual, None, self.eps, self.scale_dtype, checkpoint=checkpoint)
        y = q8.harp_matmul_q8(n.codes, n.scales, self.codes, self.scales, "bf16")
        y = self.out_proc.apply(y, inverse=True)
        return y, n.h, ((n.ckpt_codes, n.ckpt_scales, n.rstd) if checkpoint else None)

    def backward(self, dy, ckpt, dh=None):
        """dy: gradient of y; dh: that of h's other use.  Returns (gradient of
        x and of residual, gradient of W~ in fp32)."""
        codes, scales, rstd = ckpt
        dy = self.out_proc.apply(dy)                              # y = M_U^T y~
        dw = q8.harp_matmul_q8_wgrad(dy, codes, scales, "f32")
        dc, ds = q8.harp_quantize_q8(dy, 1, self.scale_dtype)
        dn = q8.harp_matmul_q8(dc, ds, self.codes_t, self.scales_t, "bf16")
        dx, _ = q8.harp_rmsnorm_q8_vjp(codes, scales, rstd, dn, None, dh)
        return dx, dw


def random_processor(schedule, d, seed, sigma=0.05, device="cuda") -> Processor:
    """A processor with seeded normal parameters and random signs."""
    from . import inputs
    g_sign, g_theta, g_gauss, _ = inputs.streams(seed)
    theta = torch.from_numpy(inputs.theta_params(g_theta, schedule, d, sigma, 0.1)).to(device)
    gauss = inputs.gauss_mats(g_gauss, schedule)
    blocks, scales = api.harp_materialize_blocks(schedule, d, theta,
                                                 torch.from_numpy(gauss).to(device) if gauss.size else None)
    return Processor(tuple(schedule), d, blocks, scales, torch.from_numpy(inputs.rademacher(g_sign, d)).to(device))


def main() -> int:
    torch.manual_seed(0)
    n, k, rows = 640, 512, 300
    u, v = random_processor((8, 8, 5, 2), n, 1), random_processor((8, 8, 8), k, 2)
    w = torch.randn(n, k, device="cuda") * 0.02
    gamma = 1 + 0.2 * torch.randn(k, device="cuda")
    x, res = torch.randn(rows, k, device="cuda"), torch.randn(rows, k, device="cuda")
    x[:, ::97] *= 50                                              # outlier channels
    h = x + res
    hn = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    want = (hn * gamma) @ w.t()
    layer = Linear8(w.to(torch.bfloat16), u, v, gamma, backward=True)
    bf = torch.bfloat16
    y, _, ckpt = layer.forward(v.apply(x.to(bf)), v.apply(res.to(bf)), checkpoint=True)
    dy = torch.randn(rows, n, device="cuda").to(bf)
    dx, dw = layer.backward(dy, ckpt)
    plain_c, plain_s = q8.harp_quantize_q8(hn.to(bf), 1, layer.scale_dtype)
    wc, ws = q8.harp_quantize_q8((w * gamma).to(bf), q8.BLOCK, layer.scale_dtype)
    plain = q8.harp_matmul_q8(plain_c, plain_s, wc, ws, "bf16")
    rel = lambda a: float((a.float() - want).norm() / want.norm())     # noqa: E731
    print(f"y against fp32: {rel(y):.4f} rotated, {rel(plain):.4f} not rotated; "
          f"|dx| {float(dx.float().norm()):.3f}, |dW~| {float(dw.norm()):.3f}")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
