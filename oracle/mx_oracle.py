"""Numpy fp64 oracle of the MX (microscaled) operators: the format's definition written out element by element,
sharing no code with the GPU path. See include/gptq_mi355x_mx.h for the format."""
from __future__ import annotations

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    v = np.empty(128)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    return v


E4M3 = _e4m3_values()
TABLE = {"e2m1": E2M1, "e4m3": E4M3[:127]}
LOWEST = {"e2m1": -125, "e4m3": -117}


def block_exponent(amax: float, fmt: str) -> int:
    """Scale exponent of a finite block: floor(log2 amax) - 2 (e2m1), or the least e with amax <= 448 2^e (e4m3)."""
    if amax == 0.0:
        return LOWEST[fmt]
    m, ex = np.frexp(amax)  # amax = m 2^ex, 1/2 <= m < 1
    if fmt == "e2m1":
        e = int(ex) - 3
    else:
        e = int(ex) - 9  # 448 = 0.875 * 2^9
        if m > 0.875:
            e += 1
    return max(e, LOWEST[fmt])


def round_to_table(t: np.ndarray, fmt: str) -> np.ndarray:
    """Code (without sign) of the nearest number of the format to each t >= 0; ties to the even code; saturating."""
    tab = TABLE[fmt]
    up = np.clip(np.searchsorted(tab, t, side="left"), 0, len(tab) - 1)
    dn = np.maximum(up - 1, 0)
    du, dd = tab[up] - t, t - tab[dn]
    pick_up = (du < dd) | ((du == dd) & (up % 2 == 0)) | (t >= tab[-1])
    return np.where(pick_up, up, dn)


def quantize(x: np.ndarray, fmt: str):
    """x (n x d, fp64 of the stored inputs) -> (codes with sign, n x d; scale bytes, n x nb). Codes of a block that
    is not finite are 0, its byte 255."""
    n, d = x.shape
    nb = -(-d // BLOCK)
    codes = np.zeros((n, d), np.uint8)
    scales = np.zeros((n, nb), np.uint8)
    sign_bit = 8 if fmt == "e2m1" else 128
    for b in range(nb):
        s = slice(b * BLOCK, min(d, (b + 1) * BLOCK))
        blk = x[:, s]
        finite = np.isfinite(blk).all(axis=1)
        amax = np.where(finite, np.abs(np.where(np.isfinite(blk), blk, 0.0)).max(axis=1), 0.0)
        e = np.array([block_exponent(a, fmt) for a in amax])
        t = np.abs(np.where(finite[:, None], blk, 0.0)) / np.exp2(e.astype(np.float64))[:, None]
        c = round_to_table(t, fmt) + np.where(np.signbit(blk), sign_bit, 0)
        codes[:, s] = np.where(finite[:, None], c, 0)
        scales[:, b] = np.where(finite, e + 127, 255)
    return codes, scales


def pack(codes: np.ndarray, scales: np.ndarray, fmt: str):
    """The stored form: (codes n x row bytes, scales n x row bytes), zeros behind the last column and block."""
    n, d = codes.shape
    kp, ks = -(-d // 128) * 128, -(-d // 512) * 16
    full = np.zeros((n, kp), np.uint8)
    full[:, :d] = codes
    if fmt == "e2m1":
        full = full[:, 0::2] | (full[:, 1::2] << 4)
    s = np.zeros((n, ks), np.uint8)
    s[:, :scales.shape[1]] = scales
    return full, s


def values(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """The numbers that unpacked codes and scales stand for, fp64."""
    n, d = codes.shape
    if fmt == "e2m1":
        v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    else:
        v = np.where(codes & 128, -1.0, 1.0) * E4M3[codes & 127]
    e = np.repeat(scales, BLOCK, axis=1)[:, :d]
    return np.where(e == 255, np.nan, v * np.exp2(e.astype(np.float64) - 127))


def round_trip(x: np.ndarray, fmt: str) -> np.ndarray:
    return values(*quantize(x, fmt), fmt)


def linear(a: np.ndarray, w: np.ndarray, bias=None, relu=False) -> np.ndarray:
    y = a @ w.T
    if bias is not None:
        y = y + bias
    return np.where(y < 0, 0.0, y) if relu else y


def grad_input(dy: np.ndarray, w: np.ndarray, mask=None) -> np.ndarray:
    dx = dy @ w
    return dx if mask is None else np.where(mask > 0, dx, 0.0)


def grad_weight(dy: np.ndarray, a: np.ndarray):
    return dy.T @ a, dy.sum(axis=0)
