"""What a call on a given stream does with torch is done there (no GPU needed: the library and the stream's context are
stood in for, and the torch functions that are called are recorded)."""
import contextlib
import types

import pytest
import torch
from torch.overrides import TorchFunctionMode

from post_weight_quantization_05_amd import _lib, gptq, mx

COPIES = {"reshape", "contiguous", "clone", "to", "flatten"}
ALLOCATIONS = {"empty", "new_empty", "zeros", "new_zeros"}


class _Recorder(TorchFunctionMode):
    """Names of the torch functions called, and whether a stream's context was entered at the time."""

    def __init__(self):
        super().__init__()
        self.depth, self.calls = 0, []

    @contextlib.contextmanager
    def on(self, stream):
        self.depth += 1
        try:
            yield
        finally:
            self.depth -= 1

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.calls.append((func.__name__, self.depth > 0))
        return func(*args, **(kwargs or {}))

    def outside(self, names):
        return [c for c, inside in self.calls if c in names and not inside]

    def inside(self, names):
        return [c for c, inside in self.calls if c in names and inside]


class _Library:
    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith("_bytes") else 0


@pytest.fixture
def recorder(monkeypatch):
    r = _Recorder()
    for m in (gptq, mx):
        monkeypatch.setattr(m, "_on", r.on)
        monkeypatch.setattr(m, "_req_cuda", lambda t, name: None)
    monkeypatch.setattr(mx, "_current_device", lambda: -1, raising=False)  # get_device() of a host tensor
    monkeypatch.setattr(_lib, "load", lambda path=None: _Library())
    return r


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_mx_quantize_flattens_tokens_on_its_stream(recorder, fmt):
    x = torch.zeros(4, 3, 64).transpose(0, 1)  # no view flattens its tokens: they are copied
    with recorder:
        q = mx.mx_quantize(x, fmt, stream=types.SimpleNamespace(cuda_stream=1))
    assert q.shape == (12, 64)
    assert not recorder.outside(COPIES | ALLOCATIONS) and recorder.inside(COPIES), recorder.calls


def test_hessian_accumulate_flattens_tokens_on_its_stream(recorder):
    x = torch.zeros(4, 3, 64).transpose(0, 1)
    state = gptq.HessianState(64, device="cpu")
    with recorder:
        gptq.hessian_accumulate(x, state, stream=types.SimpleNamespace(cuda_stream=1))
    assert not recorder.outside(COPIES | ALLOCATIONS) and recorder.inside(COPIES), recorder.calls


class _OnDevice1(torch.Tensor):
    """A host tensor that says it lies on device 1."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


def _calls():
    def t(shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice1)

    a = mx.MXTensor(t((40, 128)), t((40, 16)), 64, "e4m3")
    w = mx.MXTensor(t((8, 64)), t((8, 16)), 64, "e2m1")
    x, dy = t((40, 64), torch.bfloat16), t((40, 8), torch.bfloat16)
    s = types.SimpleNamespace(cuda_stream=1)
    return {
        "gptq_mx_quantize": lambda: mx.mx_quantize(x, stream=s),
        "gptq_mx_dequantize": lambda: mx.mx_dequantize(a, stream=s),
        "gptq_mx_matmul": lambda: mx.mx_matmul(a, w, stream=s),
        "gptq_mx_linear": lambda: mx.mx_linear(x, w, stream=s),
        "gptq_mx_grad_input": lambda: mx.mx_grad_input(dy, w, mask=a, stream=s),
        "gptq_mx_grad_weight": lambda: mx.mx_grad_weight(dy, a, bias_grad=True, stream=s),
    }


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("name", list(_calls()))
def test_mx_calls_run_on_their_tensors_device(monkeypatch, recorder, name, current):
    """The library launches on the current device: a call on another device's tensors makes that one current."""
    device, seen = [current], []

    @contextlib.contextmanager
    def use(d):
        device.append(d)
        yield
        device.pop()

    class Library(_Library):
        def __getattr__(self, f):
            if f.endswith("_bytes"):
                return lambda *a: 256
            return lambda *a: seen.append((f, device[-1])) or 0

    monkeypatch.setattr(_lib, "load", lambda path=None: Library())
    monkeypatch.setattr(mx, "_current_device", lambda: device[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "device", use)
    mx._need.cache_clear()
    _calls()[name]()
    mx._need.cache_clear()
    assert seen == [(name, 1)] and device == [current]


def test_mx_results_are_no_operands(monkeypatch, recorder):
    """A result written over an operand would race with the workgroups that still read it."""
    monkeypatch.setattr(mx, "_current_device", lambda: 1)

    def t(shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice1)

    w = mx.MXTensor(t((64, 64)), t((64, 16)), 64, "e2m1")
    x = t((40, 64), torch.bfloat16)
    s = types.SimpleNamespace(cuda_stream=1)
    for call in (lambda out: mx.mx_linear(x, w, out=out, stream=s), lambda out: mx.mx_grad_input(x, w, out=out, stream=s)):
        with pytest.raises(ValueError, match="operand"):
            call(x)
        assert call(torch.zeros_like(x)).shape == x.shape
