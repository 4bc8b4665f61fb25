"""Python binding of the MX (microscaled) operators: quantization to 4 and 8 bits, the quantized linear layer for
prompts and single tokens, and its backward pass from a 4- or 8-bit checkpoint of its input. Names follow the C ABI
(include/gptq_mi355x_mx.h); torch supplies device memory and the stream, HIP kernels do the rest.

A training step through one layer, with only the 8-bit checkpoint kept between its two halves:

    a = mx_quantize(x, "e4m3")                     # the checkpoint is what the product reads
    y = mx_matmul(a, w, bias, relu=True, dtype=torch.bfloat16)
    ...
    dx = mx_grad_input(dy, w, mask=a)              # mask: x came out of a ReLU
    dw, db = mx_grad_weight(dy, a, bias_grad=True)

Every call is asynchronous on `stream` (None = the current stream), allocates its results and workspace there, and
can be captured into a graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib
from ._lib import GPTQ_BF16, GPTQ_F32, GPTQ_MX_E2M1, GPTQ_MX_E4M3, check
from .gptq import _dtype_code, _ld, _on, _req_cuda, _stream

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


def _mx(t: MXTensor, name: str, device=None, cols: int | None = None, rows: int | None = None) -> int:
    """Checks an operand's storage; its format code."""
    if not isinstance(t, MXTensor):
        raise TypeError(f"{name} must be an MXTensor")
    code = _fmt_code(t.fmt)
    c, s = t.codes, t.scales
    if not (c.is_cuda and s.is_cuda):
        raise ValueError(f"{name} must hold device tensors")
    if t.cols < 1:
        raise ValueError(f"{name} has no columns")
    if cols is not None and t.cols != cols:
        raise ValueError(f"{name} has {t.cols} columns, {cols} expected")
    n = c.shape[0]
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, {rows} expected")
    if (c.dtype != torch.uint8 or s.dtype != torch.uint8 or c.shape != (n, _code_row(t.cols, t.fmt))
            or s.shape != (n, _scale_row(t.cols)) or not c.is_contiguous() or not s.is_contiguous()):
        raise ValueError(f"{name} must hold contiguous uint8 codes {(n, _code_row(t.cols, t.fmt))} and scales "
                         f"{(n, _scale_row(t.cols))}")
    if s.device != c.device or (device is not None and c.device != device):
        raise ValueError(f"{name} is on {c.device} and {s.device}, {device or c.device} expected")
    return code


def _w4(t: MXTensor, name: str, device=None, cols: int | None = None, rows: int | None = None) -> None:
    if _mx(t, name, device, cols, rows) != GPTQ_MX_E2M1:
        raise ValueError(f"{name} must be an e2m1 MXTensor")


def _result(out, name: str, shape, dtype, device, stream) -> torch.Tensor:
    if out is None:
        with _on(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    if not out.is_cuda or out.device != device or out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    _row_stride(out, name)
    return out


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


def _workspace(need: int, device, stream):
    if need == 0:
        return None, 0
    with _on(stream):
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr()


def _bias_ptr(bias, out: int, device):
    if bias is None:
        return None
    if bias.device != device or bias.dtype != torch.float32 or tuple(bias.shape) != (out,) or not bias.is_contiguous():
        raise ValueError(f"bias must be a contiguous float32 tensor of shape {(out,)} on {device}")
    return bias.data_ptr()


def mx_quantize(X: torch.Tensor, fmt: str = "e2m1", stream=None) -> MXTensor:
    """X (n x cols, bf16 or fp32; 3-D inputs are flattened to tokens) -> MXTensor, elements rounded to nearest-even."""
    code = _fmt_code(fmt)
    _req_cuda(X, "X")
    if X.dim() == 3:
        X = X.reshape(-1, X.shape[-1])
    ld = _matrix(X, "X")
    n, d = X.shape
    xt = _dtype_code(X)
    with _on(stream):
        codes = torch.empty((n, _code_row(d, fmt)), dtype=torch.uint8, device=X.device)
        scales = torch.empty((n, _scale_row(d)), dtype=torch.uint8, device=X.device)
    check(_lib.load().gptq_mx_quantize(X.data_ptr(), xt, n, d, ld, code, codes.data_ptr(), scales.data_ptr(),
                                       _stream(stream)), "gptq_mx_quantize")
    return MXTensor(codes, scales, d, fmt)


def mx_dequantize(Q: MXTensor, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values Q stands for, exactly (bf16 or fp32)."""
    code, yt = _mx(Q, "Q"), _out_code(dtype)
    dev = Q.codes.device
    Y = _result(out, "out", Q.shape, dtype, dev, stream)
    check(_lib.load().gptq_mx_dequantize(Q.codes.data_ptr(), Q.scales.data_ptr(), code, Q.rows, Q.cols, Y.data_ptr(),
                                         yt, _row_stride(Y, "out"), _stream(stream)), "gptq_mx_dequantize")
    return Y


def mx_matmul(A: MXTensor, W: MXTensor, bias: torch.Tensor | None = None, relu: bool = False, dtype=torch.float32,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = A W^T (+ bias, then ReLU when asked): A n x in (e2m1 or e4m3), W out x in (e2m1), Y n x out."""
    code = _mx(A, "A")
    dev = A.codes.device
    _w4(W, "W", dev, A.cols)
    yt = _out_code(dtype)
    n, d, no = A.rows, A.cols, W.rows
    b = _bias_ptr(bias, no, dev)
    Y = _result(out, "out", (n, no), dtype, dev, stream)
    lib = _lib.load()
    ws, wp = _workspace(lib.gptq_mx_matmul_workspace_bytes(n, d, no, code), dev, stream)
    check(lib.gptq_mx_matmul(A.codes.data_ptr(), A.scales.data_ptr(), code, n, d, W.codes.data_ptr(),
                             W.scales.data_ptr(), no, b, int(bool(relu)), Y.data_ptr(), yt, _row_stride(Y, "out"), wp,
                             ws.numel() if ws is not None else 0, _stream(stream)), "gptq_mx_matmul")
    return Y


def mx_linear(X: torch.Tensor, W: MXTensor, act: str = "e4m3", bias: torch.Tensor | None = None, relu: bool = False,
              dtype=None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = Q(X) W^T (+ bias, then ReLU): X (n x in, bf16 or fp32) is quantized to `act` on its way into the product,
    the results being those of mx_quantize and mx_matmul. dtype None: X's."""
    code = _fmt_code(act)
    ld = _matrix(X, "X")
    n, d = X.shape
    dev = X.device
    _w4(W, "W", dev, d)
    dtype = X.dtype if dtype is None else dtype
    xt, yt = _dtype_code(X), _out_code(dtype)
    no = W.rows
    b = _bias_ptr(bias, no, dev)
    Y = _result(out, "out", (n, no), dtype, dev, stream)
    lib = _lib.load()
    ws, wp = _workspace(lib.gptq_mx_linear_workspace_bytes(n, d, no, code), dev, stream)
    check(lib.gptq_mx_linear(X.data_ptr(), xt, n, d, ld, code, W.codes.data_ptr(), W.scales.data_ptr(), no, b,
                             int(bool(relu)), Y.data_ptr(), yt, _row_stride(Y, "out"), wp,
                             ws.numel() if ws is not None else 0, _stream(stream)), "gptq_mx_linear")
    return Y


def _grad(dY: torch.Tensor) -> int:
    if dY.dtype != torch.bfloat16:
        raise TypeError(f"unsupported gradient dtype {dY.dtype} (bfloat16)")
    return _matrix(dY, "dY")


def mx_grad_input(dY: torch.Tensor, W: MXTensor, mask: MXTensor | None = None, dtype=torch.bfloat16,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dX = dY W (dY n x out bf16, W out x in e2m1), zero wherever `mask` (n x in, the checkpoint of a ReLU's
    outputs) is not positive."""
    ld = _grad(dY)
    n, no = dY.shape
    dev = dY.device
    _w4(W, "W", dev, rows=no)
    d = W.cols
    mt = _mx(mask, "mask", dev, d, n) if mask is not None else 0
    yt = _out_code(dtype)
    dX = _result(out, "out", (n, d), dtype, dev, stream)
    lib = _lib.load()
    ws, wp = _workspace(lib.gptq_mx_grad_input_workspace_bytes(n, d, no), dev, stream)
    check(lib.gptq_mx_grad_input(dY.data_ptr(), ld, n, no, W.codes.data_ptr(), W.scales.data_ptr(), d,
                                 mask.codes.data_ptr() if mask is not None else None,
                                 mask.scales.data_ptr() if mask is not None else None, mt, dX.data_ptr(), yt,
                                 _row_stride(dX, "out"), wp, ws.numel() if ws is not None else 0, _stream(stream)),
          "gptq_mx_grad_input")
    return dX


def mx_grad_weight(dY: torch.Tensor, A: MXTensor, bias_grad: bool = False, dtype=torch.float32,
                   out: torch.Tensor | None = None, bias_out: torch.Tensor | None = None, accumulate: bool = False,
                   stream=None):
    """dW = dY^T A (dY n x out bf16, A n x in: the checkpoint of the layer's input), and db = dY's column sums in
    fp32 when bias_grad. accumulate adds to `out` (fp32) and `bias_out` instead. Returns (dW, db or None)."""
    ld = _grad(dY)
    n, no = dY.shape
    dev = dY.device
    code = _mx(A, "A", dev, rows=n)
    d = A.cols
    wt = _out_code(dtype)
    if accumulate and (out is None or (bias_grad and bias_out is None)):
        raise ValueError("accumulate adds to out (and bias_out): pass them")
    if bias_out is not None and not bias_grad:
        raise ValueError("bias_out is given without bias_grad")
    dW = _result(out, "out", (no, d), dtype, dev, stream)
    db = None
    if bias_grad:
        if bias_out is None:
            with _on(stream):
                db = torch.empty(no, dtype=torch.float32, device=dev)
        else:
            _bias_ptr(bias_out, no, dev)
            db = bias_out
    lib = _lib.load()
    ws, wp = _workspace(lib.gptq_mx_grad_weight_workspace_bytes(n, d, no), dev, stream)
    check(lib.gptq_mx_grad_weight(dY.data_ptr(), ld, n, no, A.codes.data_ptr(), A.scales.data_ptr(), code, d,
                                  int(bool(accumulate)), dW.data_ptr(), wt, _row_stride(dW, "out"),
                                  db.data_ptr() if db is not None else None, wp,
                                  ws.numel() if ws is not None else 0, _stream(stream)), "gptq_mx_grad_weight")
    return dW, db
