"""Python binding of the 8-bit operators of include/harp.h (rotated layers in
8 bits), one function per entry point.

A coded matrix is a pair (codes, scales): codes of dtype torch.float8_e4m3fn
and one scale per block of 128 columns, torch.float32 or (powers of two)
torch.float8_e8m0fnu.  Rows are coded in blocks of 1 x 128, weights in blocks
of 128 x 128.  Argument marshalling only, with the rules of api.py: every
check runs first, the GPU check last, then one library call.

stream: the stream that the work goes to (None: the current one).  The caller
makes it wait for the inputs, and the readers of the results for it; memory is
safe either way: results and workspaces made here belong to that stream, and
every tensor may be dropped as soon as the call returns.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _workspace_bytes
from ._lib import lib
from ._streams import launch, new

BLOCK = 128
CODES = torch.float8_e4m3fn
_IO = {torch.float32: _lib.HARP_F32, torch.bfloat16: _lib.HARP_BF16}
_IO_NAME = {"f32": torch.float32, "bf16": torch.bfloat16}
_SCALE = {torch.float32: _lib.HARP_F32, torch.float8_e8m0fnu: _lib.HARP_E8M0}
_SCALE_NAME = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


def _nblk(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _named(table, name, what):
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(map(repr, table))}, got {name!r}")
    return table[name]


def _mat(t, name, dtypes, rows=None, cols=None):
    """A 2-D tensor with contiguous rows: its leading dimension."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must be {'rows' if rows is None else rows} x {'columns' if cols is None else cols}, "
                         f"got {r} x {c}")
    if c < 1:
        raise ValueError(f"{name} has no columns")
    if t.is_contiguous():
        return c
    if c > 1 and r > 0 and t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    if r <= 1:
        return c
    ld = t.stride(0)
    if ld < c:
        raise ValueError(f"{name}: row stride {ld} is smaller than the row length {c}")
    return ld


def _scales(t, name, rows, cols, block_rows, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _SCALE or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'torch.float32 or torch.float8_e8m0fnu'}, got {t.dtype}")
    want = ((rows + block_rows - 1) // block_rows, (cols + 127) // 128)
    if t.shape != want:
        raise ValueError(f"{name} must be {want[0]} x {want[1]} (blocks of {block_rows} x {BLOCK}), "
                         f"got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _vec(t, name, dtype, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements, got {tuple(t.shape)}")


def _on_gpu(*tensors):
    """Every tensor given (None: left out) on one GPU: its index."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise TypeError("every argument must be a GPU tensor (the library has no CPU path)")
            if d != dev:
                if dev >= 0:
                    raise ValueError(f"the arguments are on different GPUs ({dev} and {d})")
                dev = d
    return dev


def _p(t):
    return None if t is None else t.data_ptr()


def _out_mat(t, name, dtype, rows, cols, like, stream):
    """The caller's result matrix, checked, or a new one beside `like`: it and
    its leading dimension."""
    if t is None:
        return new((rows, cols), dtype, like, stream), cols
    return t, _mat(t, name, (dtype,), rows, cols)


def _out_scales(t, name, rows, cols, block_rows, dtype, like, stream):
    if t is None:
        return new(((rows + block_rows - 1) // block_rows, _nblk(cols)), dtype, like, stream)
    _scales(t, name, rows, cols, block_rows, dtype)
    return t


def _work(workspace, need, like, stream):
    """The caller's workspace, or one allocated here when needed, and its bytes."""
    if need < 0:
        raise ValueError("sizes out of range")
    if workspace is not None:
        return workspace, _workspace_bytes(workspace)
    if need == 0:
        return None, 0
    return new(need, torch.uint8, like, stream), need


# ------------------------------------------------------------------ coding
def harp_quantize_q8(x, block_rows: int = 1, scale_dtype: str = "f32", codes=None, scales=None, stream=None):
    """Codes and scales of x (rows x cols, f32/bf16) in blocks of block_rows x
    128: block_rows 1 for activations and checkpoints, 128 for weights.
    Returns (codes, scales)."""
    ldx = _mat(x, "x", _IO)
    rows, cols = x.shape
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows must be 1 or {BLOCK}, got {block_rows}")
    sdt = _named(_SCALE_NAME, scale_dtype, "scale_dtype")
    codes, ldc = _out_mat(codes, "codes", CODES, rows, cols, x, stream)
    scales = _out_scales(scales, "scales", rows, cols, block_rows, sdt, x, stream)
    tensors = (x, codes, scales)
    dev = _on_gpu(*tensors)
    launch(lib().harp_quantize_q8, stream, dev, tensors, _p(x), ldx, _IO[x.dtype], rows, cols, block_rows, _p(codes),
           ldc, _p(scales), _SCALE[sdt])
    return codes, scales


# -------------------------------------------------------------------- norm
class RmsnormQ8(NamedTuple):
    """What harp_rmsnorm_q8 gives: the coded norm, h = x + residual (x itself
    without a residual), and for the backward pass 1/rms and the coding of
    h/rms (without gamma that is codes, scales)."""
    codes: torch.Tensor
    scales: torch.Tensor
    h: torch.Tensor
    rstd: Optional[torch.Tensor]
    ckpt_codes: Optional[torch.Tensor]
    ckpt_scales: Optional[torch.Tensor]


def harp_rmsnorm_q8(x, residual=None, gamma=None, eps: float = 1e-6, scale_dtype: str = "f32",
                    checkpoint: bool = False, h=None, codes=None, scales=None, rstd=None, ckpt_codes=None,
                    ckpt_scales=None, stream=None) -> RmsnormQ8:
    """h = x + residual; the root-mean-square norm of h times gamma, coded in
    blocks of 1 x 128.  checkpoint: also what harp_rmsnorm_q8_vjp needs."""
    ldx = _mat(x, "x", _IO)
    rows, d = x.shape
    sdt = _named(_SCALE_NAME, scale_dtype, "scale_dtype")
    io = x.dtype
    ldr = _mat(residual, "residual", (io,), rows, d) if residual is not None else d
    if gamma is not None:
        _vec(gamma, "gamma", io, d)
    if residual is None:
        if h is not None:
            raise ValueError("h goes with a residual only")
        ldh = d
    else:
        h, ldh = _out_mat(h, "h", io, rows, d, x, stream)
    codes, ldc = _out_mat(codes, "codes", CODES, rows, d, x, stream)
    scales = _out_scales(scales, "scales", rows, d, 1, sdt, x, stream)
    ldk = d
    if checkpoint:
        if rstd is None:
            rstd = new(rows, torch.float32, x, stream)
        else:
            _vec(rstd, "rstd", torch.float32, rows)
        if gamma is not None:
            ckpt_codes, ldk = _out_mat(ckpt_codes, "ckpt_codes", CODES, rows, d, x, stream)
            ckpt_scales = _out_scales(ckpt_scales, "ckpt_scales", rows, d, 1, sdt, x, stream)
    elif rstd is not None:
        raise ValueError("rstd goes with checkpoint=True only")
    if (gamma is None or not checkpoint) and (ckpt_codes is not None or ckpt_scales is not None):
        raise ValueError("ckpt_codes and ckpt_scales go with gamma and checkpoint=True only")
    tensors = (x, residual, gamma, h, codes, scales, rstd, ckpt_codes, ckpt_scales)
    dev = _on_gpu(*tensors)
    launch(lib().harp_rmsnorm_q8, stream, dev, tensors, _p(x), ldx, _p(residual), ldr, _p(gamma), eps, _p(h), ldh,
           _p(codes), ldc, _p(scales), _p(rstd), _p(ckpt_codes), ldk, _p(ckpt_scales), _SCALE[sdt], rows, d, _IO[io])
    if checkpoint and gamma is None:
        ckpt_codes, ckpt_scales = codes, scales
    return RmsnormQ8(codes, scales, x if h is None else h, rstd, ckpt_codes, ckpt_scales)


def harp_rmsnorm_q8_vjp_workspace(rows: int, d: int) -> int:
    """Workspace bytes harp_rmsnorm_q8_vjp needs for dgamma (-1: out of range)."""
    return int(lib().harp_rmsnorm_q8_vjp_workspace(rows, d))


def harp_rmsnorm_q8_vjp(ckpt_codes, ckpt_scales, rstd, dn, gamma=None, dres=None, dh=None, want_dgamma=None,
                        dgamma=None, workspace=None, stream=None):
    """Reverse mode of harp_rmsnorm_q8 from its checkpoint: dn is the gradient
    of the norm's output, dres that of h (the residual's other use).  Returns
    (dh, dgamma); dh is the gradient of x and of residual alike, dgamma (fp32)
    is None unless wanted (by default with gamma)."""
    io = dn.dtype if isinstance(dn, torch.Tensor) else None
    lddn = _mat(dn, "dn", _IO)
    rows, d = dn.shape
    ldc = _mat(ckpt_codes, "ckpt_codes", (CODES,), rows, d)
    _scales(ckpt_scales, "ckpt_scales", rows, d, 1)
    _vec(rstd, "rstd", torch.float32, rows)
    if gamma is not None:
        _vec(gamma, "gamma", io, d)
    lddres = _mat(dres, "dres", (io,), rows, d) if dres is not None else d
    dh, lddh = _out_mat(dh, "dh", io, rows, d, dn, stream)
    if want_dgamma is None:
        want_dgamma = gamma is not None or dgamma is not None
    if not want_dgamma:
        if dgamma is not None:
            raise ValueError("dgamma goes with want_dgamma")
    else:
        if dgamma is None:
            dgamma = new(d, torch.float32, dn, stream)
        else:
            _vec(dgamma, "dgamma", torch.float32, d)
    need = lib().harp_rmsnorm_q8_vjp_workspace(rows, d) if want_dgamma else 0
    workspace, ws_bytes = _work(workspace, need, dn, stream)
    tensors = (dn, ckpt_codes, ckpt_scales, rstd, gamma, dres, dh, dgamma, workspace)
    dev = _on_gpu(*tensors)
    launch(lib().harp_rmsnorm_q8_vjp, stream, dev, tensors, _p(ckpt_codes), ldc, _p(ckpt_scales),
           _SCALE[ckpt_scales.dtype], _p(rstd), _p(gamma), _p(dn), lddn, _p(dres), lddres, _p(dh), lddh, _p(dgamma),
           rows, d, _IO[io], _p(workspace), ws_bytes)
    return dh, dgamma


# ---------------------------------------------------------------- products
def harp_matmul_q8_workspace(rows: int, n: int, k: int) -> int:
    """Workspace bytes harp_matmul_q8 needs (0: none, -1: out of range)."""
    return int(lib().harp_matmul_q8_workspace(rows, n, k))


def harp_matmul_q8(a_codes, a_scales, w_codes, w_scales, out: str = "bf16", y=None, workspace=None, stream=None):
    """y = A W^T of coded matrices: A rows x k in 1 x 128 blocks, W n x k in
    128 x 128 blocks, y rows x n ("f32" or "bf16")."""
    lda = _mat(a_codes, "a_codes", (CODES,))
    rows, k = a_codes.shape
    ldw = _mat(w_codes, "w_codes", (CODES,), None, k)
    n = w_codes.shape[0]
    if n < 1:
        raise ValueError("w_codes has no rows")
    _scales(a_scales, "a_scales", rows, k, 1)
    _scales(w_scales, "w_scales", n, k, BLOCK, a_scales.dtype)
    odt = _named(_IO_NAME, out, "out")
    y, ldy = _out_mat(y, "y", odt, rows, n, a_codes, stream)
    workspace, ws_bytes = _work(workspace, lib().harp_matmul_q8_workspace(rows, n, k), a_codes, stream)
    tensors = (a_codes, a_scales, w_codes, w_scales, y, workspace)
    dev = _on_gpu(*tensors)
    launch(lib().harp_matmul_q8, stream, dev, tensors, _p(a_codes), lda, _p(a_scales), _p(w_codes), ldw, _p(w_scales),
           _SCALE[a_scales.dtype], rows, n, k, _p(y), ldy, _IO[odt], _p(workspace), ws_bytes)
    return y


def harp_matmul_q8_wgrad_workspace(rows: int, n: int, k: int) -> int:
    """Workspace bytes harp_matmul_q8_wgrad needs (0: none, -1: out of range)."""
    return int(lib().harp_matmul_q8_wgrad_workspace(rows, n, k))


def harp_matmul_q8_wgrad(dy, x_codes, x_scales, out: str = "f32", dw=None, workspace=None, stream=None):
    """dW = dY^T X (n x k, "f32" or "bf16") from dy (rows x n, bf16) and the
    coded rows x (rows x k, 1 x 128 blocks) that the product was given."""
    lddy = _mat(dy, "dy", (torch.bfloat16,))
    rows, n = dy.shape
    ldx = _mat(x_codes, "x_codes", (CODES,), rows)
    k = x_codes.shape[1]
    _scales(x_scales, "x_scales", rows, k, 1)
    odt = _named(_IO_NAME, out, "out")
    dw, lddw = _out_mat(dw, "dw", odt, n, k, dy, stream)
    workspace, ws_bytes = _work(workspace, lib().harp_matmul_q8_wgrad_workspace(rows, n, k), dy, stream)
    tensors = (dy, x_codes, x_scales, dw, workspace)
    dev = _on_gpu(*tensors)
    launch(lib().harp_matmul_q8_wgrad, stream, dev, tensors, _p(dy), lddy, _p(x_codes), ldx, _p(x_scales),
           _SCALE[x_scales.dtype], rows, n, k, _p(dw), lddw, _IO[odt], _p(workspace), ws_bytes)
    return dw
