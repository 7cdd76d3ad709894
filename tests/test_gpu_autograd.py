"""Automatic differentiation of the 8-bit layer and of the distillation loss where the plain answer
would be a wrong one: what was saved has been written to, a second derivative, a tangent, a gradient
that is not computed.  Each is an error."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

from post_weight_quantization_02_gb300 import DistilledHead, Fp8Linear, TopLogits, distill_loss, top_logits

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def randn(seed, *shape, device, dtype=F32, scale=1.0):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)


def make_layer(device, grad=True):
    w = randn(1, 200, 260, device=device, scale=0.02).requires_grad_(grad)
    return w, Fp8Linear.from_weight(w, keep=True)


def make_loss(device, rows=6):
    logits = randn(2, rows, 900, device=device)
    return logits, top_logits(randn(3, rows, 900, device=device, scale=3), 20)


# ------------------------------------------------------------------ saved tensors that are written to

def test_refresh_before_backward(lib, cuda_device):
    """The input gradient needs the codes of the forward pass."""
    w, layer = make_layer(cuda_device)
    x = randn(4, 9, 260, device=cuda_device).requires_grad_()
    y = layer(x)
    with torch.no_grad():
        w.mul_(-3)
    layer.refresh()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = layer(x)                                   # and a new forward pass has them
    (dx,) = torch.autograd.grad(y.sum(), (x,))
    assert torch.equal(dx, layer.backward(torch.ones_like(y), x.detach())[0])


def test_refresh_before_backward_of_the_weight(lib, cuda_device):
    """The weight's gradient does not."""
    w, layer = make_layer(cuda_device)
    x = randn(4, 9, 260, device=cuda_device)
    y = layer(x)
    with torch.no_grad():
        w.mul_(-3)
    layer.refresh()
    (dw,) = torch.autograd.grad(y.sum(), (w,))
    assert torch.equal(dw, layer.backward(torch.ones_like(y), x, need_dx=False)[1])


def test_gradient_in_place_before_backward(lib, cuda_device):
    logits, teacher = make_loss(cuda_device)
    logits.requires_grad_()
    loss = distill_loss(logits, teacher)
    flat = logits.detach()
    lib.gptq_distill_loss_grad(flat, teacher.values, teacher.indices, dlogits=flat)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()


def test_written_tensors_are_marked(lib, cuda_device):
    """Every call that writes into its caller's tensors."""
    dev = cuda_device
    x, dy = randn(5, 40, 260, device=dev), randn(6, 40, 200, device=dev)
    codes, scales = lib.gptq_fp8_quantize(randn(7, 200, 260, device=dev))
    logits, t = make_loss(dev)
    n = logits.shape[0]
    e = lambda *shape, dtype=F32: torch.zeros(*shape, dtype=dtype, device=dev)
    calls = [
        (lambda **o: lib.gptq_fp8_quantize(x, "rows", **o),
         dict(codes=e(40, 272, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :260], scales=e(3, 40))),
        (lambda **o: lib.gptq_fp8_linear(x, codes, scales, **o), dict(y=e(40, 200))),
        (lambda **o: lib.gptq_fp8_linear_backward(dy, x, codes, scales, **o),
         dict(dx=e(40, 260), dw=e(200, 260))),
        (lambda **o: lib.gptq_top_logits(logits, 5, **o),
         dict(values=e(n, 5), indices=e(n, 5, dtype=torch.int32), lse=e(n))),
        (lambda **o: lib.gptq_distill_loss(logits, t.values, t.indices, **o), dict(loss=e(n), lse=e(n))),
        (lambda **o: lib.gptq_distill_backward(logits, t.lse, t.values, t.indices, **o),
         dict(dlogits=e(n, 900))),
        (lambda **o: lib.gptq_distill_loss_grad(logits, t.values, t.indices, **o),
         dict(loss=e(n), dlogits=e(n, 900))),
    ]
    for call, outs in calls:
        before = {k: v._version for k, v in outs.items()}
        call(**outs)
        assert all(v._version > before[k] for k, v in outs.items()), outs.keys()
    with torch.inference_mode():                    # tensors without a version
        lib.gptq_fp8_linear(x, codes, scales, y=e(40, 200))


def test_what_is_saved(lib, cuda_device):
    """Activations are kept for the weight's gradient only, codes for the input's only."""
    def kept(x, layer):
        seen = []
        def pack(t):
            seen.append(t.data_ptr())
            return t
        with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
            layer(x)
        return x.data_ptr() in seen, layer.codes.data_ptr() in seen
    x = randn(4, 9, 260, device=cuda_device)
    frozen, trained = make_layer(cuda_device, False)[1], make_layer(cuda_device)[1]
    assert kept(x, trained) == (True, False)
    x.requires_grad_()
    assert kept(x, frozen) == (False, True)
    assert kept(x, trained) == (True, True)


# ------------------------------------------------------------------ derivatives that do not exist

def test_second_derivatives(lib, cuda_device):
    """A gradient taken for a second derivative is the gradient, and differentiating it an error,
    also where only the weight or the saved input would have a second-order term."""
    w, layer = make_layer(cuda_device)
    x = randn(4, 9, 260, device=cuda_device).requires_grad_()
    logits, teacher = make_loss(cuda_device)
    logits.requires_grad_()
    for out, inp in ((lambda: layer(x).square().sum(), x), (lambda: layer(x).sum(), x),
                     (lambda: layer(x).sum(), w), (lambda: distill_loss(logits, teacher).sum(), logits)):
        (ref,) = torch.autograd.grad(out(), (inp,))
        (grad,) = torch.autograd.grad(out(), (inp,), create_graph=True)
        assert torch.equal(grad, ref)
        with pytest.raises(RuntimeError, match="second derivative"):
            (inp.sum() + grad.square().sum()).backward()


def test_tangents(lib, cuda_device):
    w, layer = make_layer(cuda_device, False)
    x = randn(4, 9, 260, device=cuda_device)
    logits, teacher = make_loss(cuda_device)
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        calls = [lambda: layer(dual), lambda: DistilledHead(w).logits(dual),
                 lambda: distill_loss(fwd.make_dual(logits, torch.ones_like(logits)), teacher)]
        layer_w = Fp8Linear(layer.codes, layer.scales, fwd.make_dual(w, torch.ones_like(w)))
        calls.append(lambda: layer_w(x))
        for call in calls:
            with pytest.raises(NotImplementedError, match="jvp"):
                call()
        layer(x)                                    # nothing here has a tangent


def test_gradients_of_weights_and_teacher(lib, cuda_device):
    """The loss has a gradient for the student's logits alone; asking for another is refused."""
    logits, teacher = make_loss(cuda_device)
    logits.requires_grad_()
    w = torch.rand(6, device=cuda_device)
    ref = distill_loss(logits, teacher, 1.0, w)
    w.requires_grad_()
    with pytest.raises(ValueError, match="weights"):
        distill_loss(logits, teacher, 1.0, w)
    values = TopLogits(teacher.values.clone().requires_grad_(), teacher.indices, teacher.lse)
    with pytest.raises(ValueError, match="teacher"):
        distill_loss(logits, values)
    assert torch.equal(distill_loss(logits, teacher, 1.0, w.detach()), ref)
    with torch.no_grad():
        assert torch.equal(distill_loss(logits, values, 1.0, w), ref)
