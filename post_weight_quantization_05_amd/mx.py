"""Python binding of the MX (microscaled) operators: quantization to 4 and 8 bits, the quantized linear layer for
prompts and single tokens, and its backward pass from a 4- or 8-bit checkpoint of its input. Names follow the C ABI
(include/gptq_mi355x_mx.h); torch supplies device memory and the stream, HIP kernels do the rest.

A training step through one layer, with only the 8-bit checkpoint kept between its two halves:

    a = mx_quantize(x, "e4m3")                     # the checkpoint is what the product reads
    y = mx_matmul(a, w, bias, relu=True, dtype=torch.bfloat16)
    ...
    dx = mx_grad_input(dy, w, mask=a)              # mask: x came out of a ReLU
    dw, db = mx_grad_weight(dy, a, bias_grad=True)

Every call is asynchronous on `stream` (None = the current stream of the tensors' device), allocates its results and
workspace there, and can be captured into a graph. No call records an autograd graph, whatever its inputs require: the
gradients are calls of their own.
"""
from __future__ import annotations

from dataclasses import dataclass
from functools import lru_cache

import torch

from . import _lib
from ._lib import GPTQ_BF16, GPTQ_F32, GPTQ_MX_E2M1, GPTQ_MX_E4M3, check
from .gptq import _dtype_code, _ld, _on, _req_cuda, _stream as _stream_handle

__all__ = [
    "MXTensor", "mx_quantize", "mx_dequantize", "mx_matmul", "mx_linear", "mx_grad_input", "mx_grad_weight",
]

_FMT = {"e2m1": GPTQ_MX_E2M1, "e4m3": GPTQ_MX_E4M3}
_DTYPE = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}


def _fmt_code(fmt: str) -> int:
    try:
        return _FMT[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"unknown MX format {fmt!r} ('e2m1' or 'e4m3')") from None


def _out_code(dtype) -> int:
    try:
        return _DTYPE[dtype]
    except (KeyError, TypeError):
        raise TypeError(f"unsupported dtype {dtype} (bfloat16 or float32)") from None


def _code_row(cols: int, fmt: str) -> int:
    return -(-cols // 128) * (64 if fmt == "e2m1" else 128)


def _scale_row(cols: int) -> int:
    return -(-cols // 512) * 16


@dataclass
class MXTensor:
    """A matrix of rows x cols in MX form: blocks of 32 consecutive columns of a row share a power of two.

    codes:  uint8 [rows, 64 or 128 bytes for each 128 columns]: two 4-bit E2M1 codes to a byte (even column in the
            low half) or one E4M3 code; zeros behind the last column.
    scales: uint8 [rows, 16 for each 512 columns]: exponent + 127 of each block (255: the block is NaN); zeros
            behind the last block.
    Rows are independent: t.rows_slice(a, b) shares storage."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    fmt: str = "e2m1"

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self):
        return (self.codes.shape[0], self.cols)

    def rows_slice(self, start: int, stop: int) -> "MXTensor":
        return MXTensor(self.codes[start:stop], self.scales[start:stop], self.cols, self.fmt)


# A call's kernels may take only a few microseconds, so the ordinary case passes each check once, on integers, and only
# a failure looks for its reason.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device_index: int) -> int:
    """Handle of `stream`, or of the device's current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device_index)
    return _stream_handle(stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, device: int, *args) -> None:
    """The library's function with that device as the current one, on which its kernels are launched."""
    f = getattr(_lib.load(), name)
    if _current_device() == device:
        check(f(*args), name)
    else:
        with torch.cuda.device(device):
            check(f(*args), name)


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream):
        return like.new_empty(shape, dtype=dtype)


def _mx(t: MXTensor, name: str, device: int | None = None, cols: int | None = None, rows: int | None = None) -> int:
    """Checks an operand's storage; its format code. device: the index that it has to be on."""
    if not isinstance(t, MXTensor):
        raise TypeError(f"{name} must be an MXTensor")
    code = _FMT.get(t.fmt) if isinstance(t.fmt, str) else None
    c, s, d = t.codes, t.scales, t.cols
    n = c.shape[0]
    if (code is not None and c.is_cuda and s.is_cuda and d >= 1 and (cols is None or d == cols)
            and (rows is None or n == rows) and c.dtype == torch.uint8 and s.dtype == torch.uint8
            and c.shape == (n, _code_row(d, t.fmt)) and s.shape == (n, _scale_row(d)) and c.is_contiguous()
            and s.is_contiguous() and c.get_device() == s.get_device()
            and (device is None or c.get_device() == device)):
        return code
    _fmt_code(t.fmt)
    if not (c.is_cuda and s.is_cuda):
        raise ValueError(f"{name} must hold device tensors")
    if d < 1:
        raise ValueError(f"{name} has no columns")
    if cols is not None and d != cols:
        raise ValueError(f"{name} has {d} columns, {cols} expected")
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, {rows} expected")
    if s.device != c.device or (device is not None and c.get_device() != device):
        raise ValueError(f"{name} is on {c.device} and {s.device}, device {device} expected")
    raise ValueError(f"{name} must hold contiguous uint8 codes {(n, _code_row(d, t.fmt))} and scales "
                     f"{(n, _scale_row(d))}")


def _w4(t: MXTensor, name: str, device: int | None = None, cols: int | None = None, rows: int | None = None) -> None:
    if _mx(t, name, device, cols, rows) != GPTQ_MX_E2M1:
        raise ValueError(f"{name} must be an e2m1 MXTensor")


def _result(out, name: str, shape, dtype, like: torch.Tensor, stream):
    """The result's tensor and its leading dimension. like: the first operand."""
    if out is None:
        return _empty(shape, dtype, like, stream), shape[1]
    if not out.is_cuda or out.device != like.device or out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {like.device}")
    if out.numel() and out.data_ptr() == like.data_ptr():
        raise ValueError(f"{name} is an operand: results lie apart from what other workgroups still read")
    return out, _row_stride(out, name)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a row-major matrix; a single row's stride is its width whatever torch reports."""
    ld = _ld(t, name)
    if t.shape[0] <= 1:
        return t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def _matrix(t: torch.Tensor, name: str) -> int:
    """Checks a row-major device matrix (3-D inputs are flattened by the caller); its leading dimension."""
    _req_cuda(t, name)
    if t.dim() != 2 or t.shape[1] < 1:
        raise ValueError(f"{name} must be a 2-D tensor with at least one column")
    if t.shape[1] == 1 and t.stride(1) != 1:
        return _row_stride(t.as_strided(t.shape, (t.stride(0), 1)), name)
    return _row_stride(t, name)


def _workspace(need: int, like: torch.Tensor, stream):
    if need == 0:
        return None, None
    ws = _empty((need,), torch.uint8, like, stream)
    return ws, ws.data_ptr()


@lru_cache(maxsize=1024)
def _need(query: str, *sizes) -> int:
    return getattr(_lib.load(), query)(*sizes)


def _bias_ptr(bias, out: int, like: torch.Tensor):
    if bias is None:
        return None
    if (bias.device != like.device or bias.dtype != torch.float32 or bias.shape != (out,)
            or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 tensor of shape {(out,)} on {like.device}")
    return bias.data_ptr()


def mx_quantize(X: torch.Tensor, fmt: str = "e2m1", stream=None) -> MXTensor:
    """X (n x cols, bf16 or fp32; 3-D inputs are flattened to tokens) -> MXTensor, elements rounded to nearest-even."""
    code = _fmt_code(fmt)
    _req_cuda(X, "X")
    if X.dim() == 3:
        with _on(stream):  # tokens that no view flattens are copied there, and the copy belongs to it
            X = X.reshape(-1, X.shape[-1])
    ld = _matrix(X, "X")
    n, d = X.shape
    xt = _dtype_code(X)
    codes = _empty((n, _code_row(d, fmt)), torch.uint8, X, stream)
    scales = _empty((n, _scale_row(d)), torch.uint8, X, stream)
    dev = X.get_device()
    _call("gptq_mx_quantize", dev, X.data_ptr(), xt, n, d, ld, code, codes.data_ptr(), scales.data_ptr(),
          _stream(stream, dev))
    return MXTensor(codes, scales, d, fmt)


def mx_dequantize(Q: MXTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values Q stands for, exactly (bf16 or fp32)."""
    code, yt = _mx(Q, "Q"), _out_code(dtype)
    c, n, d = Q.codes, Q.codes.shape[0], Q.cols
    Y, ld = _result(out, "out", (n, d), dtype, c, stream)
    dev = c.get_device()
    _call("gptq_mx_dequantize", dev, c.data_ptr(), Q.scales.data_ptr(), code, n, d, Y.data_ptr(), yt, ld,
          _stream(stream, dev))
    return Y


def mx_matmul(A: MXTensor, W: MXTensor, bias: torch.Tensor | None = None, relu: bool = False, dtype=torch.float32,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = A W^T (+ bias, then ReLU when asked): A n x in (e2m1 or e4m3), W out x in (e2m1), Y n x out."""
    code = _mx(A, "A")
    c, n, d = A.codes, A.codes.shape[0], A.cols
    dev = c.get_device()
    _w4(W, "W", dev, d)
    yt = _out_code(dtype)
    no = W.codes.shape[0]
    b = _bias_ptr(bias, no, c)
    Y, ld = _result(out, "out", (n, no), dtype, c, stream)
    need = _need("gptq_mx_matmul_workspace_bytes", n, d, no, code)
    ws, wp = _workspace(need, c, stream)
    _call("gptq_mx_matmul", dev, c.data_ptr(), A.scales.data_ptr(), code, n, d, W.codes.data_ptr(), W.scales.data_ptr(),
          no, b, 1 if relu else 0, Y.data_ptr(), yt, ld, wp, need, _stream(stream, dev))
    return Y


def mx_linear(X: torch.Tensor, W: MXTensor, act: str = "e4m3", bias: torch.Tensor | None = None, relu: bool = False,
              dtype=None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = Q(X) W^T (+ bias, then ReLU): X (n x in, bf16 or fp32) is quantized to `act` on its way into the product,
    the results being those of mx_quantize and mx_matmul. dtype None: X's."""
    code = _fmt_code(act)
    ldx = _matrix(X, "X")
    n, d = X.shape
    dev = X.get_device()
    _w4(W, "W", dev, d)
    dtype = X.dtype if dtype is None else dtype
    xt, yt = _dtype_code(X), _out_code(dtype)
    no = W.codes.shape[0]
    b = _bias_ptr(bias, no, X)
    Y, ld = _result(out, "out", (n, no), dtype, X, stream)
    need = _need("gptq_mx_linear_workspace_bytes", n, d, no, code)
    ws, wp = _workspace(need, X, stream)
    _call("gptq_mx_linear", dev, X.data_ptr(), xt, n, d, ldx, code, W.codes.data_ptr(), W.scales.data_ptr(), no, b,
          1 if relu else 0, Y.data_ptr(), yt, ld, wp, need, _stream(stream, dev))
    return Y


def _grad(dY: torch.Tensor) -> int:
    if dY.dtype != torch.bfloat16:
        raise TypeError(f"unsupported gradient dtype {dY.dtype} (bfloat16)")
    return _matrix(dY, "dY")


def mx_grad_input(dY: torch.Tensor, W: MXTensor, mask: MXTensor | None = None, dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX = dY W (dY n x out bf16, W out x in e2m1), zero wherever `mask` (n x in, the checkpoint of a ReLU's
    outputs) is not positive. An activation that the checkpoint rounded to 0 counts as 0: in e4m3 at least 2.2e5 times
    below its block's largest, in e2m1 up to 1/16 of it."""
    ldy = _grad(dY)
    n, no = dY.shape
    dev = dY.get_device()
    _w4(W, "W", dev, rows=no)
    d = W.cols
    mc = ms = None
    mt = 0
    if mask is not None:
        mt = _mx(mask, "mask", dev, d, n)
        mc, ms = mask.codes.data_ptr(), mask.scales.data_ptr()
    yt = _out_code(dtype)
    dX, ld = _result(out, "out", (n, d), dtype, dY, stream)
    need = _need("gptq_mx_grad_input_workspace_bytes", n, d, no)
    ws, wp = _workspace(need, dY, stream)
    _call("gptq_mx_grad_input", dev, dY.data_ptr(), ldy, n, no, W.codes.data_ptr(), W.scales.data_ptr(), d, mc, ms, mt,
          dX.data_ptr(), yt, ld, wp, need, _stream(stream, dev))
    return dX


def mx_grad_weight(dY: torch.Tensor, A: MXTensor, bias_grad: bool = False, dtype=torch.float32,
                   out: torch.Tensor | None = None, bias_out: torch.Tensor | None = None, accumulate: bool = False,
                   stream=None):
    """dW = dY^T A (dY n x out bf16, A n x in: the checkpoint of the layer's input), and db = dY's column sums in
    fp32 when bias_grad. accumulate adds to `out` (fp32) and `bias_out` instead. Returns (dW, db or None)."""
    ldy = _grad(dY)
    n, no = dY.shape
    dev = dY.get_device()
    code = _mx(A, "A", dev, rows=n)
    d = A.cols
    wt = _out_code(dtype)
    if accumulate and (out is None or (bias_grad and bias_out is None)):
        raise ValueError("accumulate adds to out (and bias_out): pass them")
    if bias_out is not None and not bias_grad:
        raise ValueError("bias_out is given without bias_grad")
    dW, ld = _result(out, "out", (no, d), dtype, dY, stream)
    db = dbp = None
    if bias_grad:
        db = _empty((no,), torch.float32, dY, stream) if bias_out is None else bias_out
        dbp = db.data_ptr() if bias_out is None else _bias_ptr(db, no, dY)
    need = _need("gptq_mx_grad_weight_workspace_bytes", n, d, no)
    ws, wp = _workspace(need, dY, stream)
    _call("gptq_mx_grad_weight", dev, dY.data_ptr(), ldy, n, no, A.codes.data_ptr(), A.scales.data_ptr(), code, d,
          1 if accumulate else 0, dW.data_ptr(), wt, ld, dbp, wp, need, _stream(stream, dev))
    return dW, db
