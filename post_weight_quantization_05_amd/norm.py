"""Python binding of the root-mean-square norm that writes 8-bit tokens, and of its gradient (include/gptq_mi355x_int8.h).

Before an integer layer, the residual stream h updated in place:

    y, h, _ = rms_norm(x, weight, residual=h, out=h)            # y: Int8Tensor
    x = int8_matmul(y, w, dtype=torch.bfloat16)

A training step through norm and MX layer, the norm's 8-bit output being the layer's checkpoint:

    y, h, rstd = rms_norm(x, weight, residual=h, fmt="e4m3")    # y: MXTensor
    z = mx_matmul(y, w)
    ...
    dw, _ = mx_grad_weight(dz, y)
    dx, dweight = rms_norm_grad(mx_grad_input(dz, w), h, rstd, weight, dH=dh)   # the gradient of x and of the residual

Every call is asynchronous on `stream` (None = the current stream of the tensors' device), allocates its results and
workspace there, and can be captured into a graph. No call records an autograd graph: the gradient is a call of its own.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._lib import GPTQ_NORM_E4M3, GPTQ_NORM_INT8
from .int8 import Int8Tensor, _apart, _rows, _type
from .int8 import _code_row as _int8_code_row
from .mx import MXTensor, _call, _empty, _need, _result, _scale_row, _stream, _workspace
from .mx import _code_row as _mx_code_row

__all__ = ["NormResult", "rms_norm", "rms_norm_grad"]

_FMT = {"int8": GPTQ_NORM_INT8, "e4m3": GPTQ_NORM_E4M3}


class NormResult(NamedTuple):
    y: Int8Tensor | MXTensor  # the normalized, weighted rows in 8 bits
    h: torch.Tensor           # x + residual (x itself without one)
    rstd: torch.Tensor        # float32 [n]


def _operand(t: torch.Tensor, name: str, like: torch.Tensor, dtype=None) -> int:
    ld = _rows(t, name)
    if t.shape != like.shape or t.get_device() != like.get_device() or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be a {dtype or 'bfloat16 or float32'} tensor of shape {tuple(like.shape)} on "
                         f"{like.device}")
    return ld


def _vector(t: torch.Tensor, name: str, size: int, device: int) -> int:
    if t.get_device() != device or t.dtype is not torch.float32 or t.shape != (size,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(size,)} on device {device}")
    return t.data_ptr()


def rms_norm(X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
             fmt: str = "int8", out: torch.Tensor | None = None, stream=None) -> NormResult:
    """h = X + residual, rounded to fp32 and then to the residual's type; y = h / sqrt(mean h^2 + eps) * weight in 8 bits:
    integers with a scale for each row ("int8", an Int8Tensor) or MX blocks ("e4m3", an MXTensor). X and residual n x d in
    bf16 or fp32, weight fp32. out: where h goes, which may be the residual itself; without a residual h is X and nothing is
    written."""
    try:
        code = _FMT[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"unknown format {fmt!r} ('int8' or 'e4m3')") from None
    ldx, xt = _rows(X, "X"), _type(X)
    n, d = X.shape
    dev = X.get_device()
    w = _vector(weight, "weight", d, dev)
    rp = hp = None
    rt = ldr = ldh = 0
    h = X
    if residual is not None:
        ldr, rt = _operand(residual, "residual", X), _type(residual)
        rp = residual.data_ptr()
        same = False
        if out is not None:  # a single row's stride says nothing: the same bytes are the same row
            same = out is residual or (out.data_ptr() == rp and out.shape == residual.shape
                                       and (n == 1 or out.stride() == residual.stride()))
            _apart(out, "out", X, weight, None if same else residual)
        h, ldh = _result(out, "out", (n, d), residual.dtype, X, stream)
        if same:
            ldh = ldr
        hp = h.data_ptr()
    elif out is not None:
        raise ValueError("out is given without a residual: h is X")
    if code == GPTQ_NORM_INT8:
        codes = _empty((n, _int8_code_row(d)), torch.int8, X, stream)
        scales = _empty((n,), torch.float32, X, stream)
        y = Int8Tensor(codes, scales, d)
    else:
        codes = _empty((n, _mx_code_row(d, "e4m3")), torch.uint8, X, stream)
        scales = _empty((n, _scale_row(d)), torch.uint8, X, stream)
        y = MXTensor(codes, scales, d, "e4m3")
    rstd = _empty((n,), torch.float32, X, stream)
    _call("gptq_rms_norm", dev, X.data_ptr(), xt, ldx, rp, rt, ldr, n, d, w, float(eps), hp, ldh, code, codes.data_ptr(),
          scales.data_ptr(), rstd.data_ptr(), _stream(stream, dev))
    return NormResult(y, h, rstd)


def rms_norm_grad(dY: torch.Tensor, H: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                  dH: torch.Tensor | None = None, out: torch.Tensor | None = None, weight_out: torch.Tensor | None = None,
                  accumulate: bool = False, stream=None):
    """The gradients of X (and alike of the residual), in H's type, and of the weight, fp32, from dY, the gradient of
    rms_norm's y, and its h and rstd. dH: the gradient of h itself, added to X's. accumulate adds the weight's gradient to
    weight_out. Returns (dX, dweight)."""
    ldy, yt = _rows(dY, "dY"), _type(dY)
    n, d = dY.shape
    dev = dY.get_device()
    ldh, ht = _operand(H, "H", dY), _type(H)
    r, w = _vector(rstd, "rstd", n, dev), _vector(weight, "weight", d, dev)
    sp, lds = None, 0
    if dH is not None:
        lds = _operand(dH, "dH", dY, H.dtype)
        sp = dH.data_ptr()
    if accumulate and weight_out is None:
        raise ValueError("accumulate adds to weight_out: pass it")
    if out is not None:
        _apart(out, "out", dY, H, rstd, weight, dH, weight_out)
    dX, ldx = _result(out, "out", (n, d), H.dtype, dY, stream)
    if weight_out is None:
        dw = _empty((d,), torch.float32, dY, stream)
        dwp = dw.data_ptr()
    else:
        _apart(weight_out, "weight_out", dY, H, rstd, weight, dH)
        dw, dwp = weight_out, _vector(weight_out, "weight_out", d, dev)
    need = _need("gptq_rms_norm_grad_workspace_bytes", n, d)
    ws, wp = _workspace(need, dY, stream)
    _call("gptq_rms_norm_grad", dev, dY.data_ptr(), yt, ldy, H.data_ptr(), ht, ldh, r, w, sp, lds, n, d,
          1 if accumulate else 0, dX.data_ptr(), ldx, dwp, wp, need, _stream(stream, dev))
    return dX, dw
