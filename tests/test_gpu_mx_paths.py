"""GPU parity of the MX products on the paths that only some sizes take: sums over slices of k that another launch joins
(with everything the join applies), workgroups that pass from one tile to the next inside the result, launches that take a
call in pieces, scales that differ from block to block, and every scale byte.

How many slices a size gets follows from the workspace that the library asks for, and is asserted, so that a changed rule
cannot leave these tests without their path. References are formed in fp64 on the device; bounds are those of
test_gpu_mx.py.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_05_amd as G
from oracle import mx_oracle as MX
from post_weight_quantization_05_amd import _lib

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

STEP = 2.0 ** -23  # a product's or an addition's error, relative to the sum of magnitudes so far
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FMT = {"e2m1": 0, "e4m3": 1}


def _check(y, ref, mag, k):
    """|y - ref| <= (k + 2) steps of mag + the result's rounding; NaN where the reference is."""
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    bound = (k + 2) * STEP * mag + ref.abs() * HALF[y.dtype] + 1e-38
    err = torch.where(ok, (y.double() - ref).abs(), 0.0)
    worst = float(torch.where(ok, err / bound, 0.0).max())
    assert worst <= 1.0, f"{worst:.3g} of the bound"
    ref, mag = torch.where(ok, ref, 0.0), torch.where(ok, mag, 0.0)
    # errors of a random sum add up like a random walk; at least 16 products enter each addition
    assert float(err.norm()) <= np.sqrt(k / 16 + 4) * STEP * float(mag.norm()) + HALF[y.dtype] * float(ref.norm())


def _up(v, to):
    return -(-v // to) * to


def _matmul_slices(n, d, out, fmt):
    need = _lib.load().gptq_mx_matmul_workspace_bytes(n, d, out, FMT[fmt])
    return max(1, need // (n * out * 4))


def _grad_input_slices(n, d, out):
    need = _lib.load().gptq_mx_grad_input_workspace_bytes(n, d, out)
    rest = need - _up(out * _up(d, 128) * 2, 256) - _up(n * _up(out, 128) * 2, 256)
    return max(1, rest // (n * d * 4))


def _grad_weight_slices(n, d, out):
    need = _lib.load().gptq_mx_grad_weight_workspace_bytes(n, d, out)
    rest = need - _up(n * _up(d, 128) * 2, 256) - _up(n * _up(out, 128) * 2, 256)
    assert 2 * -(-n // 256) < d  # the column sums' part is less than one slice
    return max(1, rest // (out * d * 4))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(g, n, d, fmt, relu=False, nan=()):
    x = torch.randn((n, d), generator=g, device="cuda")
    x[:, d // 3] *= 20
    if relu:
        x = torch.relu(x)
    for r, c in nan:
        x[r, c] = float("nan")
    q = G.mx_quantize(x, fmt)
    return q, G.mx_dequantize(q, torch.float32).double()


def _weights(g, out, d):
    q = G.mx_quantize(torch.randn((out, d), generator=g, device="cuda") * 0.02, "e2m1")
    return q, G.mx_dequantize(q, torch.float32).double()


def _gradient(g, n, out):
    return (torch.randn((n, out), generator=g, device="cuda") * 1e-3).bfloat16()


# ---- sums over slices -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,out,slices", [(700, 11008, 600, 2), (300, 6300, 200, 2), (20, 11008, 67, 3)])
def test_matmul_slices(n, d, out, slices, y, fmt):
    print(f"[mx matmul slices] {n}x{d}x{out} {fmt} -> {y}", flush=True)
    assert _matmul_slices(n, d, out, fmt) == slices
    g = _gen(n)
    a, a64 = _tokens(g, n, d, fmt, nan=[(3, d - 1)])
    w, w64 = _weights(g, out, d)
    bias = torch.randn(out, generator=g, device="cuda")
    ref, mag = a64 @ w64.t(), torch.nan_to_num(a64).abs() @ w64.abs().t()
    _check(G.mx_matmul(a, w, dtype=DT[y]), ref, mag, d)
    ref, mag = ref + bias.double(), mag + bias.double().abs()
    wide = torch.full((n, out + 5), 7.0, dtype=DT[y], device="cuda")
    G.mx_matmul(a, w, bias=bias, dtype=DT[y], out=wide[:, 3:3 + out])
    _check(wide[:, 3:3 + out], ref, mag, d + 1)
    G.mx_matmul(a, w, bias=bias, relu=True, dtype=DT[y], out=wide[:, 3:3 + out])
    _check(wide[:, 3:3 + out], torch.where(ref < 0, 0.0, ref), mag, d + 1)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + out:] == 7).all()


GRADS = [(200, 520, 4096, 4), (130, 333, 2100, 2), (2040, 1910, 2100, 2)]  # tiles of 64, 64 and 128


@pytest.mark.parametrize("mask", [None, "e2m1", "e4m3"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,out,slices", GRADS)
def test_grad_input_slices(n, d, out, slices, y, mask):
    print(f"[mx grad_input slices] {n}x{d}x{out} mask {mask} -> {y}", flush=True)
    assert _grad_input_slices(n, d, out) == slices
    g = _gen(n + d)
    dy = _gradient(g, n, out)
    w, w64 = _weights(g, out, d)
    m, m64 = _tokens(g, n, d, mask, relu=True, nan=[(0, 0), (n - 1, d - 1), (n // 2, 70)]) if mask else (None, None)
    ref, mag = dy.double() @ w64, dy.double().abs() @ w64.abs()
    if mask:
        ref = torch.where(m64 > 0, ref, 0.0)
    got = G.mx_grad_input(dy, w, mask=m, dtype=DT[y])
    _check(got, ref, mag, out)
    wide = torch.full((n, d + 3), 7.0, dtype=DT[y], device="cuda")
    G.mx_grad_input(dy, w, mask=m, dtype=DT[y], out=wide[:, 1:1 + d])
    assert torch.equal(wide[:, 1:1 + d], got) and (wide[:, 0] == 7).all() and (wide[:, 1 + d:] == 7).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("out,d,n,slices", GRADS)
def test_grad_weight_slices(n, d, out, slices, fmt):
    print(f"[mx grad_weight slices] {n}x{d}x{out} {fmt}", flush=True)
    assert _grad_weight_slices(n, d, out) == slices
    g = _gen(n + d)
    dy = _gradient(g, n, out)
    a, a64 = _tokens(g, n, d, fmt, relu=True)
    ref, mag = dy.double().t() @ a64, dy.double().abs().t() @ a64.abs()
    sums, smag = dy.double().sum(0), dy.double().abs().sum(0)
    for y in ("f32", "bf16"):
        dw, db = G.mx_grad_weight(dy, a, bias_grad=True, dtype=DT[y])
        _check(dw, ref, mag, n)
        assert float(((db.double() - sums).abs() - sums.abs() * HALF[torch.float32] - n * 2.0 ** -52 * smag).max()) <= 0
    wide, total = torch.full((out, d + 3), 0.5, device="cuda"), torch.full((out,), -0.25, device="cuda")
    G.mx_grad_weight(dy, a, bias_grad=True, out=wide[:, 1:1 + d], bias_out=total, accumulate=True)
    _check(wide[:, 1:1 + d], ref + 0.5, mag + 0.5, n + 1)
    assert (wide[:, 0] == 0.5).all() and (wide[:, 1 + d:] == 0.5).all()
    off = (total.double() - (sums - 0.25)).abs()
    assert float((off - 0.5 * HALF[torch.float32] - n * 2.0 ** -52 * (smag + 1)).max()) <= 0


# ---- workgroups that pass from tile to tile -------------------------------------------------------------------
# 17 x 18 tiles of 256, more than the chip has places for, most of them inside the result
HANDOVER = (4350, 4600, 600)


@pytest.mark.parametrize("mask", [None, "e2m1", "e4m3"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_grad_input_from_tile_to_tile(y, mask):
    n, d, out = HANDOVER
    print(f"[mx grad_input handover] mask {mask} -> {y}", flush=True)
    g = _gen(7)
    dy = _gradient(g, n, out)
    w, w64 = _weights(g, out, d)
    m, m64 = _tokens(g, n, d, mask, relu=True, nan=[(0, 0), (n - 1, d - 1), (700, 3000), (4000, 40)]) if mask else (None, None)
    ref, mag = dy.double() @ w64, dy.double().abs() @ w64.abs()
    if mask:
        ref = torch.where(m64 > 0, ref, 0.0)
    _check(G.mx_grad_input(dy, w, mask=m, dtype=DT[y]), ref, mag, out)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_grad_weight_from_tile_to_tile(y, fmt):
    out, d, n = HANDOVER
    print(f"[mx grad_weight handover] {fmt} -> {y}", flush=True)
    g = _gen(8)
    dy = _gradient(g, n, out)
    a, a64 = _tokens(g, n, d, fmt, relu=True)
    ref, mag = dy.double().t() @ a64, dy.double().abs().t() @ a64.abs()
    _check(G.mx_grad_weight(dy, a, dtype=DT[y])[0], ref, mag, n)
    if y == "f32":
        total = torch.full((out, d), 0.5, device="cuda")
        G.mx_grad_weight(dy, a, out=total, accumulate=True)
        _check(total, ref + 0.5, mag + 0.5, n + 1)


def test_matmul_not_finite_in_the_largest_4_bit_tile():
    """d long enough for tiles of 256 of either operand."""
    g = _gen(9)
    x, v = torch.randn((4100, 2000), generator=g, device="cuda"), torch.randn((4200, 2000), generator=g, device="cuda")
    x[17, 1999], x[4099, 0], v[5, 300], v[4199, 1999] = float("nan"), float("inf"), float("inf"), float("nan")
    for y in ("f32", "bf16"):
        got = torch.isnan(G.mx_matmul(G.mx_quantize(x, "e2m1"), G.mx_quantize(v, "e2m1"), relu=True, dtype=DT[y]))
        want = torch.zeros_like(got)
        want[[17, 4099]] = True
        want[:, [5, 4199]] = True
        assert torch.equal(got, want)


# ---- calls in pieces ------------------------------------------------------------------------------------------
def test_quantize_in_pieces():
    """More rows than one launch takes (2^25 of up to 512 columns)."""
    n, d = (1 << 25) + 5, 32
    X = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((9, d), generator=_gen(10), device="cuda").bfloat16()
    X[-9:] = tail
    q, want = G.mx_quantize(X, "e2m1"), G.mx_quantize(tail, "e2m1")
    assert torch.equal(q.codes[-9:], want.codes) and torch.equal(q.scales[-9:], want.scales)
    assert not q.codes[:-9].any()
    v = G.mx_dequantize(q, out=X)
    assert torch.equal(v[-9:], G.mx_dequantize(want)) and not v[:-9].any()


@pytest.mark.parametrize("mask", [None, "e4m3"])
@pytest.mark.parametrize("out", [64, 60])  # dY read as it is, and from a padded copy
def test_grad_input_in_pieces(out, mask):
    """More rows than one launch takes (2^20)."""
    n, d = (1 << 20) + 700, 64
    g = _gen(11)
    dy = _gradient(g, n, out)
    w, w64 = _weights(g, out, d)
    m, m64 = _tokens(g, n, d, mask, relu=True) if mask else (None, None)
    ref, mag = dy.double() @ w64, dy.double().abs() @ w64.abs()
    if mask:
        ref = torch.where(m64 > 0, ref, 0.0)
    _check(G.mx_grad_input(dy, w, mask=m), ref, mag, out)


def test_matmul_in_pieces():
    """More tiles than one launch takes (2^20): the second piece's tokens."""
    n, d, out = 16384 + 300, 64, 1 << 20
    g = _gen(12)
    a, a64 = _tokens(g, n, d, "e2m1")
    w, w64 = _weights(g, out, d)
    y = G.mx_matmul(a, w, dtype=torch.bfloat16)
    for rows in (slice(0, 40), slice(16384 - 40, 16384 + 40), slice(n - 40, n)):
        _check(y[rows], a64[rows] @ w64.t(), a64[rows].abs() @ w64.abs().t(), d)


# ---- scales ---------------------------------------------------------------------------------------------------
def _equal_rows(values, exponents, fmt, rows):
    """rows equal rows of element values ({column: value}, zeros elsewhere) with the blocks' scale exponents."""
    d, tab = 32 * len(exponents), MX.TABLE[fmt]
    c = np.zeros((rows, d), np.uint8)
    for col, v in values.items():
        k, = np.where(tab == abs(v))
        c[:, col] = int(k[0]) | ((8 if fmt == "e2m1" else 128) if v < 0 else 0)
    return _stored(c, np.tile(np.asarray(exponents) + 127, (rows, 1)).astype(np.uint8), fmt)


def _stored(c, s, fmt):
    codes, scales = MX.pack(c, s, fmt)
    return (G.MXTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), c.shape[1], fmt),
            MX.values(c, s, fmt))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("n", [1, 16, 17, 300])
def test_blocks_of_far_scales_do_not_lose_each_other(n, fmt):
    """2^s - 2^s in one block, 2.25 in another of the same 64 or 128 columns: partial sums are multiples of 1/4 below
    2^(s + 1), which fp32 holds in any order up to s = 21."""
    for s in (0, 3, 6, 10, 14, 17, 20):
        for big, small in ((0, 1), (1, 0), (0, 2), (3, 0), (1, 3), (2, 3)):
            e = [0] * 4
            e[big] = s
            a, a64 = _equal_rows({32 * big: 1.0, 32 * big + 1: 1.0, 32 * small + 5: 1.5}, e, fmt, n)
            w, w64 = _equal_rows({32 * big: 1.0, 32 * big + 1: -1.0, 32 * small + 5: 1.5}, [0] * 4, "e2m1", 40)
            assert (G.mx_matmul(a, w) == 2.25).all() and (a64 @ w64.T == 2.25).all(), (s, big, small)
            a, _ = _equal_rows({32 * big: 1.0, 32 * big + 1: 1.0, 32 * small + 5: 1.5}, [0] * 4, fmt, n)
            w, _ = _equal_rows({32 * big: 1.0, 32 * big + 1: -1.0, 32 * small + 5: 1.5}, e, "e2m1", 40)
            assert (G.mx_matmul(a, w) == 2.25).all(), (s, big, small)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("n,d,out", [(8, 1024, 300), (100, 1024, 300), (1030, 700, 2100), (4100, 2000, 4200)])
def test_products_and_gradients_with_scales_of_every_size(n, d, out, fmt):
    """Blocks whose sizes are spread over 2^16 to either side."""
    print(f"[mx scales] {n}x{d}x{out} {fmt}", flush=True)
    g = _gen(n + d)

    def spread(rows):
        e = torch.randint(-16, 17, (rows, -(-d // 32)), generator=g, device="cuda").float()
        return torch.randn((rows, d), generator=g, device="cuda") * torch.exp2(e).repeat_interleave(32, 1)[:, :d]

    a, w = G.mx_quantize(spread(n), fmt), G.mx_quantize(spread(out), "e2m1")
    a64, w64 = (G.mx_dequantize(t, torch.float32).double() for t in (a, w))
    dy = _gradient(g, n, out)
    _check(G.mx_matmul(a, w), a64 @ w64.t(), a64.abs() @ w64.abs().t(), d)
    dx = G.mx_grad_input(dy, w, mask=a, dtype=torch.float32)
    _check(dx, torch.where(a64 > 0, dy.double() @ w64, 0.0), dy.double().abs() @ w64.abs(), out)
    dw, _ = G.mx_grad_weight(dy, a)
    _check(dw, dy.double().t() @ a64, dy.double().abs().t() @ a64.abs(), n)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_every_scale_byte_and_code(fmt):
    """Dequantized, each code under each scale byte is its value rounded once to the result's type; and the product
    takes the byte for the same power of two."""
    signs = 16 if fmt == "e2m1" else 256
    c = np.tile((np.arange(256) % signs).astype(np.uint8), (256, 1))
    s = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 8))
    q, v = _stored(c, s, fmt)
    want = torch.from_numpy(v)
    assert torch.equal(G.mx_dequantize(q, torch.float32).cpu().nan_to_num(7.5), want.float().nan_to_num(7.5))
    # values have at most 4 significant bits, so rounding to fp32 first changes nothing about bf16
    assert torch.equal(G.mx_dequantize(q).float().cpu().nan_to_num(7.5), want.float().bfloat16().float().nan_to_num(7.5))
    for rows in (8, 40):
        for byte in (0, 1, 2, 9, 10, 11, 60, 127, 200, 250, 254):
            a, _ = _equal_rows({3: 1.0}, [0], fmt, rows)
            a.scales[:, 0] = byte
            w, _ = _equal_rows({3: 1.0}, [0], "e2m1", 5)
            other = min(max(254 - byte, 0), 254)
            w.scales[:, 0] = other
            assert (G.mx_matmul(a, w) == 2.0 ** (byte + other - 254)).all(), (byte, other)


# ---- the layer is the quantization and the product ------------------------------------------------------------
@pytest.mark.parametrize("act", ["e2m1", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 4096), (1, 11008), (3, 1001), (8, 4096), (9, 4096), (16, 512), (16, 4100), (17, 600), (300, 640)])
def test_linear_is_quantize_and_matmul(n, d, x, act):
    g = _gen(n + d)
    X = (torch.randn((n, d), generator=g, device="cuda") * 3).to(DT[x])
    w, _ = _weights(g, 130, d)
    bias = torch.randn(130, generator=g, device="cuda")
    for y in ("f32", "bf16"):
        want = G.mx_matmul(G.mx_quantize(X, act), w, bias=bias, relu=True, dtype=DT[y])
        assert torch.equal(G.mx_linear(X, w, act=act, bias=bias, relu=True, dtype=DT[y]), want)
