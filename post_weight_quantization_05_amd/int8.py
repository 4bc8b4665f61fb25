"""Python binding of the 8-bit integer operators: tokens quantized with a scale each, the linear layer whose weights are
GPTQ's integer codes, on quantized or plain tokens. Names follow the C ABI (include/gptq_mi355x_int8.h); torch supplies
device memory and the stream, HIP kernels do the rest.

A layer that GPTQ quantized on the symmetric grid with one grid per row (8 bits or fewer):

    w = int8_weight(gptq_quantize(W, X, bits=8))
    y = int8_matmul(int8_quantize(x), w, bias)       # tokens of a prompt; rms_norm (norm.py) writes such tokens too
    y = int8_linear(x, w, bias)                      # the same in one call, down to a single token

Every call is asynchronous on `stream` (None = the current stream of the tensors' device), allocates its results and
workspace there, and can be captured into a graph. No call records an autograd graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from ._lib import GPTQ_BF16, GPTQ_F32
from .gptq import QuantResult, _dtype_code, _on, _req_cuda
from .mx import _bias_ptr, _call, _empty, _matrix, _need, _out_code, _result, _stream, _workspace

__all__ = ["Int8Tensor", "int8_quantize", "int8_dequantize", "int8_weight", "int8_matmul", "int8_linear"]


_TYPES = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}


def _code_row(cols: int) -> int:
    return (cols + 127) & -128


def _rows(t: torch.Tensor, name: str) -> int:
    """Checks a row-major device matrix; its leading dimension. (The ordinary case in one pass: a call's kernels may take
    only a few microseconds.)"""
    s = t.shape
    if len(s) == 2 and t.is_cuda:
        ld, one = t.stride()
        if one == 1 and ld >= s[1] > 0:
            return ld
    return _matrix(t, name)


def _type(t: torch.Tensor) -> int:
    code = _TYPES.get(t.dtype)
    return _dtype_code(t) if code is None else code


@dataclass
class Int8Tensor:
    """A matrix of rows x cols in 8-bit integers: value(r, c) = codes(r, c) * scales(r).

    codes:  int8 [rows, cols rounded up to 128], zeros behind the last column.
    scales: float32 [rows] (NaN: the whole row is).
    Rows are independent: t.rows_slice(a, b) shares storage."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self):
        return (self.codes.shape[0], self.cols)

    def rows_slice(self, start: int, stop: int) -> "Int8Tensor":
        return Int8Tensor(self.codes[start:stop], self.scales[start:stop], self.cols)


def _int8(t: Int8Tensor, name: str, device: int | None = None, cols: int | None = None) -> None:
    """Checks an operand's storage. device: the index that it has to be on."""
    if not isinstance(t, Int8Tensor):
        raise TypeError(f"{name} must be an Int8Tensor")
    c, s, d = t.codes, t.scales, t.cols
    n, dev = c.shape[0], c.get_device()
    if (dev >= 0 and (device is None or dev == device) and (cols is None or d == cols) and d >= 1
            and c.dtype is torch.int8 and s.dtype is torch.float32 and c.shape == (n, _code_row(d)) and s.shape == (n,)
            and c.is_contiguous() and s.is_contiguous() and s.get_device() == dev):
        return
    if not (c.is_cuda and s.is_cuda):
        raise ValueError(f"{name} must hold device tensors")
    if d < 1:
        raise ValueError(f"{name} has no columns")
    if cols is not None and d != cols:
        raise ValueError(f"{name} has {d} columns, {cols} expected")
    if s.device != c.device or (device is not None and c.get_device() != device):
        raise ValueError(f"{name} is on {c.device} and {s.device}, device {device} expected")
    raise ValueError(f"{name} must hold contiguous int8 codes {(n, _code_row(d))} and float32 scales {(n,)}")


def _extent(t: torch.Tensor):
    """Address of a matrix's (or vector's, or number's) first byte, bytes of a row, bytes from one row to the next, rows."""
    size = t.element_size()
    if t.dim() < 2:
        return t.data_ptr(), t.numel() * size, t.numel() * size, 1
    return t.data_ptr(), t.shape[1] * size, max(t.stride(0), t.shape[1]) * size, t.shape[0]


def _share_memory(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two row-major matrices may share a byte; column ranges of one wider matrix are told apart."""
    pa, wa, sa, na = _extent(a)
    pb, wb, sb, nb = _extent(b)
    if pa + (na - 1) * sa + wa <= pb or pb + (nb - 1) * sb + wb <= pa:
        return False
    if na > 1 and nb > 1 and sa != sb:
        return True
    step = sa if na > 1 else sb
    if na == 1 and nb == 1:
        return True
    off = (pb - pa) % step  # of b's rows within a's
    return off < wa or off + wb > step


def _apart(out, name: str, *operands) -> None:
    """Refuses a given result that shares memory with an operand."""
    if out.numel() == 0 or out.dim() > 2:
        return
    a, _, step, rows = _extent(out)
    b = a + step * rows
    for t in operands:
        if t is None or t.numel() == 0:
            continue
        p = t.data_ptr()
        if p >= b or (t.is_contiguous() and p + t.nbytes <= a):
            continue
        if _share_memory(out, t):
            raise ValueError(f"{name} shares memory with an operand")


def int8_quantize(X: torch.Tensor, stream=None) -> Int8Tensor:
    """X (n x cols, bf16 or fp32; 3-D inputs are flattened to tokens) -> Int8Tensor, a scale for each row and codes
    -127 .. 127 rounded to nearest-even. A row that is not finite becomes NaN."""
    if X.dim() == 3:
        _req_cuda(X, "X")
        with _on(stream):  # tokens that no view flattens are copied there, and the copy belongs to it
            X = X.reshape(-1, X.shape[-1])
    ld, xt = _rows(X, "X"), _type(X)
    n, d = X.shape
    codes = _empty((n, _code_row(d)), torch.int8, X, stream)
    scales = _empty((n,), torch.float32, X, stream)
    dev = X.get_device()
    _call("gptq_int8_quantize", dev, X.data_ptr(), xt, n, d, ld, codes.data_ptr(), scales.data_ptr(), _stream(stream, dev))
    return Int8Tensor(codes, scales, d)


def int8_dequantize(Q: Int8Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values Q stands for, rounded to fp32 and then to dtype (bf16 or fp32)."""
    _int8(Q, "Q")
    yt = _out_code(dtype)
    c, n, d = Q.codes, Q.codes.shape[0], Q.cols
    if out is not None:
        _apart(out, "out", c, Q.scales)
    Y, ld = _result(out, "out", (n, d), dtype, c, stream)
    dev = c.get_device()
    _call("gptq_int8_dequantize", dev, c.data_ptr(), Q.scales.data_ptr(), n, d, Y.data_ptr(), yt, ld, _stream(stream, dev))
    return Y


def int8_weight(result: QuantResult, stream=None) -> Int8Tensor:
    """A layer's weights from what gptq_quantize (or quantize_layer) returned on the symmetric grid with one grid per row.
    Codes and scales are shared where the width is a multiple of 128, and copied into padded rows elsewhere."""
    if not isinstance(result, QuantResult):
        raise TypeError("result must be a QuantResult")
    c, s = result.codes, result.scales
    if result.zeros is not None or c.dtype != torch.int8:
        raise ValueError("the asymmetric grid's codes have zero points: int8 products take the symmetric grid's")
    if s.dim() != 2 or s.shape[1] != 1:
        raise ValueError(f"{s.shape[-1]} grids per row: int8 products take codes with one (group=None)")
    _req_cuda(c, "codes")
    out, d = c.shape
    if s.shape[0] != out or s.dtype != torch.float32 or s.device != c.device or not (c.is_contiguous() and s.is_contiguous()):
        raise ValueError(f"scales must be a contiguous float32 tensor of shape {(out, 1)} on {c.device}, codes contiguous")
    if d % 128 == 0 and c.data_ptr() % 16 == 0:
        return Int8Tensor(c, s.view(out), d)
    padded = _empty((out, _code_row(d)), torch.int8, c, stream)
    dev = c.get_device()
    _call("gptq_int8_pad_codes", dev, c.data_ptr(), out, d, padded.data_ptr(), _stream(stream, dev))
    return Int8Tensor(padded, s.view(out), d)


def int8_matmul(A: Int8Tensor, W: Int8Tensor, bias: torch.Tensor | None = None, relu: bool = False, dtype=torch.float32,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = A W^T (+ bias, then ReLU when asked): A n x in, W out x in, Y n x out. Sums are exact; in fp32 they are multiplied
    by the token's scale, and then by the channel's with bias added in the same step."""
    _int8(A, "A")
    c, n, d = A.codes, A.codes.shape[0], A.cols
    dev = c.get_device()
    _int8(W, "W", dev, d)
    yt = _out_code(dtype)
    no = W.codes.shape[0]
    b = _bias_ptr(bias, no, c)
    if out is not None:
        _apart(out, "out", c, A.scales, W.codes, W.scales, bias)
    Y, ld = _result(out, "out", (n, no), dtype, c, stream)
    need = _need("gptq_int8_matmul_workspace_bytes", n, d, no)
    ws, wp = _workspace(need, c, stream)
    _call("gptq_int8_matmul", dev, c.data_ptr(), A.scales.data_ptr(), n, d, W.codes.data_ptr(), W.scales.data_ptr(), no, b,
          1 if relu else 0, Y.data_ptr(), yt, ld, wp, need, _stream(stream, dev))
    return Y


def int8_linear(X: torch.Tensor, W: Int8Tensor, bias: torch.Tensor | None = None, relu: bool = False, dtype=None,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = Q(X) W^T (+ bias, then ReLU): X (n x in, bf16 or fp32) is quantized on its way into the product, the results
    being those of int8_quantize and int8_matmul. dtype None: X's."""
    ldx, xt = _rows(X, "X"), _type(X)
    n, d = X.shape
    dev = X.get_device()
    _int8(W, "W", dev, d)
    yt = xt
    if dtype is None:
        dtype = X.dtype
    else:
        yt = _out_code(dtype)
    no = W.codes.shape[0]
    b = _bias_ptr(bias, no, X)
    if out is not None:
        _apart(out, "out", X, W.codes, W.scales, bias)
    Y, ld = _result(out, "out", (n, no), dtype, X, stream)
    need = _need("gptq_int8_linear_workspace_bytes", n, d, no)
    ws, wp = _workspace(need, X, stream)
    _call("gptq_int8_linear", dev, X.data_ptr(), xt, n, d, ldx, W.codes.data_ptr(), W.scales.data_ptr(), no, b,
          1 if relu else 0, Y.data_ptr(), yt, ld, wp, need, _stream(stream, dev))
    return Y
