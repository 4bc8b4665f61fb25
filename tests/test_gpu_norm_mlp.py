"""The residual MLP example: its gradients, and that it runs from prompts to single tokens."""
import pytest
import torch

import post_weight_quantization_05_amd as G

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)


def _through(x, value):
    """value forwards, x's gradient backwards: what the 8-bit roundings do."""
    return x + (value - x).detach()


@pytest.mark.parametrize("n,width,hidden", [(48, 96, 160), (130, 256, 512)])
def test_gradients(n, width, hidden):
    """Against autograd in fp64 through the values that the forward pass kept. Between the given gradient and a result
    lie at most seven roundings to bf16 (three a block: du, dy, dx), each 2^-9 of its vector's norm or less. They are
    independent of each other and pass through the same products as the gradients, so to a factor of two their part of
    a result is sqrt(7) 2^-9: 2^-6 bounds both. Sums in fp32 add far less."""
    from examples.norm_mlp import NormMlp

    g = torch.Generator(device="cuda").manual_seed(n)
    model = NormMlp(width, hidden, seed=3)
    for t in model.gain:
        t += 0.2 * torch.randn(t.shape, generator=g, device="cuda")
    for t in model.b:
        t += 0.1 * torch.randn(t.shape, generator=g, device="cuda")
    x = torch.randn((n, width), generator=g, device="cuda").bfloat16()
    d = (torch.randn((n, width), generator=g, device="cuda") * 1e-2).bfloat16()
    model.forward(x)
    dW, db, dgain, dx = model.backward(d)

    gain = [t.double().requires_grad_() for t in model.gain]
    W = [G.mx_dequantize(q, torch.float32).double().requires_grad_() for q in model.Q]
    b = [t.double().requires_grad_() for t in model.b]
    entered = x.double().requires_grad_()
    h, add = entered, 0.0
    for i, (y8, h8, _, a8) in enumerate(model.kept):
        h = _through(h + add, h8.double())
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * gain[i]
        y = _through(y, G.mx_dequantize(y8, torch.float32).double())
        a8 = G.mx_dequantize(a8, torch.float32).double()
        u = y @ W[2 * i].t() + b[2 * i]
        a = _through(u * (a8 > 0), a8)
        add = a @ W[2 * i + 1].t() + b[2 * i + 1]
    ((h + add) * d.double()).sum().backward()
    for got, ref in list(zip(dW, W)) + list(zip(db, b)) + list(zip(dgain, gain)) + [(dx, entered)]:
        assert got.shape == ref.grad.shape
        err = float((got.double() - ref.grad).norm() / ref.grad.norm())
        assert err <= 2.0 ** -6, err


def test_runs_and_serves():
    from examples.norm_mlp import IntegerMlp, train

    losses, model, x = train(steps=3, n=200)
    assert len(losses) == 3 and all(v == v for v in losses)
    before = x.clone()
    served = IntegerMlp(model, x)
    h, out = served(x)
    assert torch.equal(x, before) and h.shape == out.shape == x.shape and torch.isfinite(out).all()
    for rows in (slice(0, 1), slice(7, 12), slice(150, 200)):  # rows do not depend on each other, nor on the kernel
        a, b = served(x[rows])
        assert torch.equal(a, h[rows]) and torch.equal(b, out[rows])
