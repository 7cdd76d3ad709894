"""A linear layer in 8-bit floating point with a scale for every 128 values.

``Fp8Linear`` keeps a weight as e4m3 codes in 128 x 128 blocks (``gptq_fp8_quantize``) and
multiplies activations, quantised in 1 x 128 groups on the way in, on the tensor cores
(``gptq_fp8_linear``).  It can be made from a dense weight or from a packed GPTQ checkpoint
(``QuantizedLayer``), and it is differentiable once, in reverse mode: the gradients of its input
and of its weight are 8-bit products too (``gptq_fp8_linear_backward``; the quantisers count as the
identity).
Every call only enqueues; ``gptq.gptq_async_status`` reports device-side failures.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.forward_ad import unpack_dual

from . import gptq as G
from .api import QuantizedLayer

__all__ = ["Fp8Linear"]


def _matrix(t: torch.Tensor) -> torch.Tensor:
    """t as a matrix of contiguous rows that do not overlap (a broadcast gradient is copied)."""
    t = t.reshape(-1, t.shape[-1])
    rows, cols = t.shape
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        t = t.contiguous()
    return t


def _differentiated(t: Optional[torch.Tensor]) -> bool:
    """Whether t takes part in automatic differentiation, of either mode (a call that has no
    forward mode has to say so)."""
    return t is not None and ((torch.is_grad_enabled() and t.requires_grad)
                              or unpack_dual(t).tangent is not None)


class _Gradient(torch.autograd.Function):
    """A gradient that a call computed, tied to what it has a derivative in, which is not
    computed: taking it is an error."""

    @staticmethod
    def forward(ctx, gradient, *inputs):
        return gradient

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the 8-bit layer and the distillation loss have no second derivative")


def _once(gradient: Optional[torch.Tensor], *inputs: Optional[torch.Tensor]):
    """What a backward pass returns: under create_graph, where it is recorded, not a constant."""
    if gradient is None or not torch.is_grad_enabled():
        return gradient
    return _Gradient.apply(gradient, *inputs)


class _Fp8LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, codes, scales, dtype):
        # the weight's gradient needs no codes: they may change before it is taken (the calls ask
        # for a weight of the layer's shape all the same); the input's needs no activations
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        ctx.save_for_backward(x if need_dw else None, codes if need_dx else None,
                              scales if need_dx else None)
        ctx.unread = None if need_dx else (codes, scales)
        ctx.weight = weight
        ctx.weight_dtype = None if weight is None else weight.dtype
        ctx.x_shape, ctx.x_dtype = x.shape, x.dtype
        return G.gptq_fp8_linear(x, codes, scales, dtype=dtype)

    @staticmethod
    def backward(ctx, dy):
        x, codes, scales = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if codes is None:
            codes, scales = ctx.unread
        upstream, dy = dy, _matrix(dy)
        dx = None
        if need_dx:
            dx = torch.empty(ctx.x_shape, dtype=ctx.x_dtype, device=dy.device)
        dx, dw = G.gptq_fp8_linear_backward(dy, x, codes, scales,
                                            need_dx=need_dx, need_dw=need_dw, dx=dx,
                                            dw_dtype=ctx.weight_dtype or torch.float32)
        return _once(dx, upstream, ctx.weight), _once(dw, upstream, x), None, None, None


class Fp8Linear:
    """y = x W^T with W [d_out, d_in] in 8-bit blocks.

    ``codes`` float8_e4m3fn [d_out, d_in] (rows of a multiple of 16 bytes) and ``scales``
    float32 [ceil(d_out / 128), ceil(d_in / 128)].  ``weight``, if kept, is the dense weight
    that the gradient belongs to (``refresh`` turns it into codes again after a step).
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor,
                 weight: Optional[torch.Tensor] = None):
        self.codes, self.scales, self.weight = codes, scales, weight
        self.d_out, self.d_in = codes.shape

    @classmethod
    def from_weight(cls, weight: torch.Tensor, keep: bool = False) -> "Fp8Linear":
        """From a dense weight (bf16 or fp32); ``keep`` holds on to it for training."""
        codes, scales = G.gptq_fp8_quantize(weight.detach(), "blocks")
        return cls(codes, scales, weight if keep else None)

    @classmethod
    def from_checkpoint(cls, layer: QuantizedLayer, bits: int) -> "Fp8Linear":
        """From a packed GPTQ layer: its weight as the codes and scales say, in 8-bit blocks."""
        return cls.from_weight(G.gptq_dequantize(layer.qweight, layer.scales, layer.qzeros,
                                                 layer.g_idx, bits))

    def refresh(self) -> None:
        """The codes of the kept weight, after it changed.  An input gradient of an earlier call
        has to be taken before (it raises afterwards)."""
        if self.weight is None:
            raise ValueError("no weight was kept")
        G.gptq_fp8_quantize(self.weight.detach(), "blocks", self.codes, self.scales)

    def __call__(self, x: torch.Tensor, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """``x`` [..., d_in] (bf16 or fp32) to [..., d_out] in ``dtype`` (x's by default)."""
        flat = _matrix(x)
        dtype = dtype or x.dtype
        if _differentiated(x) or _differentiated(self.weight):
            y = _Fp8LinearFunction.apply(flat, self.weight, self.codes, self.scales, dtype)
        else:
            y = G.gptq_fp8_linear(flat, self.codes, self.scales, dtype=dtype)
        return y.reshape(*x.shape[:-1], self.d_out)

    def backward(self, dy: torch.Tensor, x: torch.Tensor, need_dx: bool = True,
                 need_dw: bool = True) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
        """(dx, dw) for the gradient ``dy`` of the output, without automatic differentiation."""
        dx, dw = G.gptq_fp8_linear_backward(_matrix(dy), _matrix(x) if need_dw else None,
                                            self.codes, self.scales, need_dx, need_dw)
        return (None if dx is None else dx.reshape(*dy.shape[:-1], self.d_in)), dw
