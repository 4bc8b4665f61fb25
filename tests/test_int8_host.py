"""8-bit integer operators and the norm without a GPU: the oracle against hand-worked rows and differences, the C ABI's
refusals (every check runs on the host before anything is launched), and what the Python layer refuses."""
import os
import re

import numpy as np
import pytest
import torch

import post_weight_quantization_05_amd as G
from oracle import int8_oracle as I8
from post_weight_quantization_05_amd import _lib, int8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gptq_mi355x_int8.h")

needs_lib = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")
INVALID, WORKSPACE = -1, -5


# ---- the oracle ---------------------------------------------------------------------------------------------
def test_hand_rows():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -127.0, 0.49], [0.0] * 6, [1e-13, -1e-15, 0, 0, 0, 0], [1, np.inf, 0, 0, 0, 0],
                  [np.nan, 1, 2, 3, 4, 5]])
    c, s = I8.quantize(x)
    np.testing.assert_array_equal(c[0], [127, 0, 2, -2, -127, 0])  # scale 1: ties to even
    assert s[0] == 1 and s[1] == np.float32(1e-12 / 127)
    np.testing.assert_array_equal(c[1], 0)
    np.testing.assert_array_equal(c[2], [13, 0, 0, 0, 0, 0])  # below the least scale
    assert np.isnan(s[3:]).all() and not c[3:].any()
    assert I8.pad(c).shape == (5, 128) and not I8.pad(c)[:, 6:].any()


def test_round_trip_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = I8.f32(rng.standard_normal((50, 200)) * np.exp2(rng.integers(-20, 20, size=(50, 1))))
    c, s = I8.quantize(x)
    assert np.abs(c).max() == 127
    assert (np.abs(I8.values(c, s) - x) <= 0.5 * s[:, None] * (1 + 2.0 ** -40)).all()


def test_norm_gradient_against_differences():
    """Central differences of sum(dy * norm(h)): the error of a step t is t^2 / 6 of the third derivative (some 1e-9 here)
    plus rounding of the two losses over t (1e-13 / 1e-4)."""
    rng = np.random.default_rng(2)
    n, d, eps, t = 4, 7, 1e-3, 1e-4
    h, dy, w = rng.standard_normal((n, d)), rng.standard_normal((n, d)), rng.standard_normal(d)

    def loss(h, w):
        return float((dy * (h * w / np.sqrt((h * h).mean(1, keepdims=True) + eps))).sum())

    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    dx, dw = I8.norm_grad(dy, h, rstd, w)
    for i in range(n):
        for j in range(d):
            e = np.zeros_like(h)
            e[i, j] = t
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * t) - dx[i, j]) <= 1e-6
    for j in range(d):
        e = np.zeros_like(w)
        e[j] = t
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * t) - dw[j]) <= 1e-6


# ---- the C ABI ----------------------------------------------------------------------------------------------
def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(gptq_[a-z0-9_]+)\s*\(", text)))


@needs_lib
def test_exports_every_declared_symbol():
    lib = _lib.load()
    names = _declared()
    assert len(names) == 11, names
    for n in names:
        assert hasattr(lib, n) and n in _lib.SIGNATURES, n


@needs_lib
def test_row_lengths_and_workspaces():
    lib = _lib.load()
    for cols, b in ((1, 128), (128, 128), (129, 256), (11008, 11008)):
        assert lib.gptq_int8_code_bytes_per_row(cols) == b
    for bad in (0, -5, 65537):
        assert lib.gptq_int8_code_bytes_per_row(bad) == 0
    assert lib.gptq_int8_linear_workspace_bytes(-1, 8, 8) == 0
    assert lib.gptq_int8_matmul_workspace_bytes(4, 8, 0) == 0
    assert lib.gptq_rms_norm_grad_workspace_bytes(4, 65537) == 0


P = 4096  # an aligned address that is never read: every call below is refused


def _refused(fn, good, changes):
    for idx, value, status in changes:
        a = list(good)
        a[idx] = value
        assert fn(*a) == status, (fn.__name__, idx, value)


@needs_lib
def test_quantize_refusals():
    lib = _lib.load()
    good = [P, 0, 4, 64, 64, P, P, None]
    _refused(lib.gptq_int8_quantize, good, [
        (0, None, INVALID), (0, P + 2, INVALID), (1, 2, INVALID), (2, -1, INVALID), (2, 1 << 31, INVALID), (3, 0, INVALID),
        (3, 65537, INVALID), (4, 63, INVALID), (5, None, INVALID), (5, P + 8, INVALID), (6, None, INVALID),
        (6, P + 2, INVALID)])
    good = [P, P, 4, 64, P, 1, 64, None]
    _refused(lib.gptq_int8_dequantize, good, [
        (0, None, INVALID), (0, P + 4, INVALID), (1, None, INVALID), (1, P + 1, INVALID), (2, -1, INVALID), (3, 0, INVALID),
        (4, None, INVALID), (4, P + 1, INVALID), (5, 5, INVALID), (6, 63, INVALID)])
    good = [P, 4, 64, P, None]
    _refused(lib.gptq_int8_pad_codes, good, [
        (0, None, INVALID), (1, 0, INVALID), (1, (1 << 20) + 1, INVALID), (2, 0, INVALID), (2, 65537, INVALID),
        (3, None, INVALID), (3, P + 8, INVALID)])
    assert lib.gptq_int8_quantize(None, 0, 0, 64, 64, None, None, None) == 0  # no rows: nothing to do
    assert lib.gptq_int8_dequantize(None, None, 0, 64, None, 0, 64, None) == 0


@needs_lib
def test_product_refusals():
    lib = _lib.load()
    n, d, out = 20, 11008, 67  # few tiles with a long sum: the one that takes a workspace if any does
    need = lib.gptq_int8_matmul_workspace_bytes(n, d, out)
    good = [P, P, n, d, P, P, out, P, 0, P, 0, out, P, need, None]
    bad = [(0, None, INVALID), (0, P + 8, INVALID), (1, None, INVALID), (1, P + 2, INVALID), (2, -1, INVALID),
           (3, 0, INVALID), (3, 65537, INVALID), (4, None, INVALID), (4, P + 1, INVALID), (5, None, INVALID),
           (6, 0, INVALID), (6, (1 << 20) + 1, INVALID), (7, P + 2, INVALID), (8, 2, INVALID), (9, None, INVALID),
           (9, P + 2, INVALID), (10, 3, INVALID), (11, out - 1, INVALID)]
    if need:
        bad += [(12, None, WORKSPACE), (12, P + 16, WORKSPACE), (13, need - 1, WORKSPACE)]
    _refused(lib.gptq_int8_matmul, good, bad)
    need = lib.gptq_int8_linear_workspace_bytes(300, 64, 8)
    assert need >= 300 * 128 + 300 * 4
    good = [P, 1, 300, 64, 64, P, P, 8, P, 1, P, 1, 8, P, need, None]
    _refused(lib.gptq_int8_linear, good, [
        (0, None, INVALID), (0, P + 1, INVALID), (1, 9, INVALID), (2, -1, INVALID), (3, 0, INVALID), (4, 63, INVALID),
        (5, None, INVALID), (5, P + 2, INVALID), (6, None, INVALID), (7, 0, INVALID), (8, P + 1, INVALID), (9, -1, INVALID),
        (10, None, INVALID), (11, 2, INVALID), (12, 7, INVALID), (13, None, WORKSPACE), (13, P + 16, WORKSPACE),
        (14, need - 1, WORKSPACE)])


@needs_lib
def test_norm_refusals():
    lib = _lib.load()
    #       X  xt ldx R  rt ldr n  d   w  eps   H  ldh fmt codes scales rstd stream
    good = [P, 1, 64, P, 1, 64, 4, 64, P, 1e-6, 2 * P, 64, 0, P, P, P, None]
    _refused(lib.gptq_rms_norm, good, [
        (0, None, INVALID), (0, P + 1, INVALID), (1, 2, INVALID), (2, 63, INVALID), (3, P + 1, INVALID), (4, 2, INVALID),
        (5, 63, INVALID), (6, -1, INVALID), (7, 0, INVALID), (7, 65537, INVALID), (8, None, INVALID), (8, P + 2, INVALID),
        (9, 0.0, INVALID), (9, -1.0, INVALID), (9, float("nan"), INVALID), (9, float("inf"), INVALID), (9, 1e-31, INVALID),
        (10, None, INVALID), (10, 2 * P + 1, INVALID), (11, 63, INVALID), (12, 2, INVALID), (13, None, INVALID),
        (13, P + 8, INVALID), (14, None, INVALID), (14, P + 2, INVALID), (15, P + 2, INVALID)])
    in_place = list(good)
    in_place[10], in_place[11] = P, 65  # the residual's address with other rows
    assert lib.gptq_rms_norm(*in_place) == INVALID
    e4m3 = list(good)
    e4m3[12], e4m3[14] = 1, P + 4  # MX scale bytes start at 16-byte aligned addresses
    assert lib.gptq_rms_norm(*e4m3) == INVALID
    need = lib.gptq_rms_norm_grad_workspace_bytes(4000, 64)
    assert need > 0
    #       dY yt ldy h  ht ldh rstd w dH ldd n  d  acc dX ldx dw ws need stream
    good = [P, 0, 64, P, 1, 64, P, P, P, 64, 4000, 64, 0, P, 64, P, P, need, None]
    _refused(lib.gptq_rms_norm_grad, good, [
        (0, None, INVALID), (0, P + 2, INVALID), (1, 2, INVALID), (2, 63, INVALID), (3, None, INVALID), (3, P + 1, INVALID),
        (4, -1, INVALID), (5, 63, INVALID), (6, None, INVALID), (7, None, INVALID), (7, P + 2, INVALID), (8, P + 1, INVALID),
        (9, 63, INVALID), (10, -1, INVALID), (11, 0, INVALID), (12, 2, INVALID), (13, None, INVALID), (13, P + 1, INVALID),
        (14, 63, INVALID), (15, None, INVALID), (15, P + 2, INVALID), (16, None, WORKSPACE), (16, P + 16, WORKSPACE),
        (17, need - 1, WORKSPACE)])
    empty = list(good)
    empty[10], empty[12] = 0, 1
    assert lib.gptq_rms_norm_grad(*empty) == 0  # no rows to add


# ---- the Python layer ---------------------------------------------------------------------------------------
def test_python_refuses_host_tensors_and_bad_arguments():
    x = torch.zeros(4, 64)
    q = G.Int8Tensor(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4), 64)
    for call in (lambda: G.int8_quantize(x), lambda: G.int8_dequantize(q), lambda: G.int8_matmul(q, q),
                 lambda: G.int8_linear(x, q), lambda: G.rms_norm(x, torch.ones(64)),
                 lambda: G.rms_norm(x, torch.ones(64), fmt="e2m1"),
                 lambda: G.rms_norm_grad(x, x, torch.ones(4), torch.ones(64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.int8_matmul(x, q)
    with pytest.raises(TypeError):
        G.int8_weight(x)
    assert q.shape == (4, 64) and q.rows_slice(1, 3).rows == 2


def test_weights_of_other_grids_are_refused():
    c, s, g = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4, 1), torch.zeros(128, dtype=torch.int32)
    loss = torch.zeros(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="zero points"):
        G.int8_weight(G.QuantResult(c.view(torch.uint8), s, g, loss, zeros=torch.zeros(4, 1, dtype=torch.int32)))
    with pytest.raises(ValueError, match="grids per row"):
        G.int8_weight(G.QuantResult(c, torch.zeros(4, 2), g, loss))
    with pytest.raises(ValueError, match="device"):
        G.int8_weight(G.QuantResult(c, s, g, loss))


def test_shared_memory_is_found():
    base = torch.zeros(20, 50)
    share = int8._share_memory
    assert share(base, base) and share(base[:5], base[4:])
    assert not share(base[:5], base[5:])
    assert not share(base[:, :20], base[:, 20:]) and share(base[:, :21], base[:, 20:])
    assert not share(base[:, 20:], base[:, :20]) and share(base[3:9, 20:], base[:, :21])
    assert share(base[3], base) and not share(base[3, 10:20], base[3, 20:30])
    assert not share(base[3:4, 10:20], base[:, 20:])
    assert not share(torch.zeros(4, 4), torch.zeros(4, 4))
    # rows of another length: taken to share memory where they lie among each other
    assert share(base[:, :20], base.view(10, 100)[:, 20:30])
