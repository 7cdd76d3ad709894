"""Operands that the 8-bit layer's, the top logits' and the distillation's calls refuse: pointers off
their elements' alignment, and tensors of different devices (no GPU needed)."""

import pytest
import torch

from post_weight_quantization_02_gb300 import gptq as G
from tests.test_student_cpu import BACKWARD, BOTH, GRAD, INVALID, LINEAR, LOSS, P, QUANT, TOP, call


@pytest.mark.parametrize("name,defaults,fields", [
    ("gptq_fp8_quantize", QUANT, ["scales"]),
    ("gptq_fp8_linear", LINEAR, ["ws_"]),
    ("gptq_fp8_linear_backward", BACKWARD, ["ws_"]),
    ("gptq_top_logits", TOP, ["v", "i", "lse"]),
    ("gptq_distill_loss", LOSS, ["tv", "ti", "w", "loss", "lse"]),
    ("gptq_distill_backward", GRAD, ["lse", "tv", "ti", "w", "g"]),
    ("gptq_distill_loss_grad", BOTH, ["tv", "ti", "w", "loss"]),
])
def test_misaligned_pointers(name, defaults, fields):
    for f in fields:
        for off in (1, 2):
            assert call(name, defaults, {f: P + off}) == INVALID, f
            assert "aligned" in G.gptq_last_error()


@pytest.mark.parametrize("name,defaults", [("gptq_distill_loss", LOSS), ("gptq_distill_backward", GRAD),
                                           ("gptq_distill_loss_grad", BOTH)])
def test_temperature_whose_exponent_factor_overflows(name, defaults):
    """log2(e) / T has to be a finite float32 number: 4.8e38, of T = 3e-39, is not, 3.2e38 is."""
    assert call(name, defaults, dict(T=3e-39)) == INVALID
    assert call(name, defaults, dict(T=4.5e-39, rows=0)) != INVALID     # (no GPU: no status word)


class Operand:
    """What the binding looks at in a CUDA tensor."""

    def __init__(self, device, shape, dtype=torch.float32):
        self._index, self.shape, self.dtype = device, torch.Size(shape), dtype
        self.device, self.is_cuda, self.requires_grad = torch.device("cuda", device), True, False

    def dim(self):
        return len(self.shape)

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.append(n)
            n *= s
        return tuple(reversed(out))

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P

    def get_device(self):
        return self._index


F8, I32, U8 = torch.float8_e4m3fn, torch.int32, torch.uint8
CALLS = {
    G.gptq_fp8_quantize: dict(x=(40, 256), form="blocks", codes=((40, 256), F8), scales=(1, 2)),
    G.gptq_fp8_linear: dict(x=(40, 256), codes=((128, 256), F8), scales=(1, 2), y=(40, 128),
                            ws=((1 << 20,), U8)),
    G.gptq_fp8_linear_backward: dict(dy=(40, 128), x=(40, 256), codes=((128, 256), F8), scales=(1, 2),
                                     dx=(40, 256), dw=(128, 256), ws=((1 << 20,), U8)),
    G.gptq_top_logits: dict(logits=(3, 500), k=7, values=(3, 7), indices=((3, 7), I32), lse=(3,)),
    G.gptq_distill_loss: dict(logits=(3, 500), values=(3, 7), indices=((3, 7), I32), weights=(3,),
                              loss=(3,), lse=(3,)),
    G.gptq_distill_backward: dict(logits=(3, 500), lse=(3,), values=(3, 7), indices=((3, 7), I32),
                                  grad_loss=(3,), weights=(3,), dlogits=(3, 500)),
    G.gptq_distill_loss_grad: dict(logits=(3, 500), values=(3, 7), indices=((3, 7), I32), weights=(3,),
                                   loss=(3,), dlogits=(3, 500)),
}


class Recorder:
    """Stands for the library: every call succeeds and is counted."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def fn(*args):
            self.calls += 1
            return G.GPTQ_OK
        return fn


@pytest.fixture
def fake(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(G, "lib", lambda: recorder)
    monkeypatch.setattr(G, "_stream_of", lambda stream, t: 0)
    monkeypatch.setattr(torch.autograd.graph, "increment_version", lambda t: None)
    monkeypatch.setattr(G, "_devices", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return recorder


def operands(spec, devices):
    out = {}
    for name, s in spec.items():
        if not isinstance(s, tuple):
            out[name] = s
            continue
        shape, dtype = s if isinstance(s[0], tuple) else (s, torch.float32)
        out[name] = Operand(devices.get(name, devices[None]), shape, dtype)
    return out


@pytest.mark.parametrize("fn", CALLS, ids=lambda f: f.__name__)
def test_operands_of_several_devices(fake, fn):
    spec = CALLS[fn]
    fn(**operands(spec, {None: 0}))
    assert fake.calls == 1
    for name, s in spec.items():
        if isinstance(s, tuple):
            with pytest.raises(ValueError, match="device"):
                fn(**operands(spec, {None: 0, name: 1}))
    with pytest.raises(ValueError, match="current device"):
        fn(**operands(spec, {None: 1}))
    assert fake.calls == 1
