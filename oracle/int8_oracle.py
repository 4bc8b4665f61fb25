"""Numpy fp64 oracle of the 8-bit integer operators and the norm: the definitions of include/gptq_mi355x_int8.h written
out, sharing no code with the GPU path. Roundings to fp32 that the definitions name are made from fp64 values, so they
are single roundings."""
from __future__ import annotations

import numpy as np


def f32(x):
    """x rounded to fp32, as fp64."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def quantize(x: np.ndarray):
    """x (n x d, fp64 of the stored inputs) -> (codes, fp64 whole numbers; scales). A row that is not finite has the
    scale NaN and codes of 0."""
    finite = np.isfinite(x).all(axis=1)
    amax = np.abs(np.where(finite[:, None], x, 0.0)).max(axis=1, initial=0.0)
    scale = f32(np.maximum(amax, f32(1e-12)) / 127)
    q = np.where(finite[:, None], x, 0.0) / scale[:, None]
    codes = np.rint(q)  # ties to even; the quotient's own rounding lies far below the distance to a tie that is none
    return codes, np.where(finite, scale, np.nan)


def values(codes, scales):
    return codes * scales[:, None]


def pad(codes):
    """Codes as they are stored: rows up to the next multiple of 128, zeros behind the last column."""
    n, d = codes.shape
    out = np.zeros((n, -(-d // 128) * 128), np.int8)
    out[:, :d] = codes
    return out


def linear(a, sa, w, sw, bias=None, relu=False):
    y = (a @ w.T) * sa[:, None] * sw
    if bias is not None:
        y = y + bias
    return np.where(y < 0, 0.0, y) if relu else y


def norm(h, weight, eps):
    """(rstd in fp64, u = h * weight rounded to fp32) of the stored sum h."""
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    return rstd, f32(h * weight)


def norm_grad(dy, h, rstd, weight, dh=None):
    g = dy * weight
    m = (g * h).mean(axis=1, keepdims=True)
    r = rstd[:, None]
    dx = r * (g - h * r * r * m)
    return dx if dh is None else dx + dh, (dy * h * r).sum(axis=0)
