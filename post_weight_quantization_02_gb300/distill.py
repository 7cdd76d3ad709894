"""Distilling a compressed model from its full-precision teacher's top logits.

A teacher's logits are reduced to the k largest of each position (``top_logits``) and kept;
``distill_loss`` is the Kullback-Leibler divergence from their softmax to the student's, and
``DistilledHead`` runs a whole step of a student whose output head is in 8 bits: hidden states
to logits, logits to loss and gradient in one pass over them, and the gradient back to the
hidden states and the head's weight.  Everything only enqueues;
``gptq.gptq_async_status`` reports device-side failures.
"""

from __future__ import annotations

import dataclasses
from typing import Optional, Tuple

import torch

from . import gptq as G
from .fp8 import Fp8Linear, _matrix, _once

__all__ = ["TopLogits", "top_logits", "distill_loss", "DistilledHead"]


@dataclasses.dataclass
class TopLogits:
    """The k largest logits of each position."""

    values: torch.Tensor    # float32 [n, k], descending
    indices: torch.Tensor   # int32 [n, k]; -1: no entry
    lse: torch.Tensor       # float32 [n], log-sum-exp of all the position's logits


def top_logits(logits: torch.Tensor, k: int) -> TopLogits:
    """What a student needs of a teacher's ``logits`` [..., vocab] (bf16 or fp32)."""
    return TopLogits(*G.gptq_top_logits(_matrix(logits), k))


class _DistillFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, values, indices, temperature, weights):
        loss, lse = G.gptq_distill_loss(logits, values, indices, temperature, weights)
        ctx.save_for_backward(logits, lse, values, indices, weights)
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, grad_loss):
        logits, lse, values, indices, weights = ctx.saved_tensors
        d = G.gptq_distill_backward(logits, lse, values, indices, grad_loss.float().contiguous(),
                                    ctx.temperature, weights)
        return _once(d, logits, grad_loss), None, None, None, None


def distill_loss(logits: torch.Tensor, teacher: TopLogits, temperature: float = 1.0,
                 weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each position's loss, float32 [n], differentiable in ``logits`` [..., vocab] alone;
    ``weights`` float32 [n] multiply it, and a position of weight 0 does not count."""
    for t, name in ((weights, "weights"), (teacher.values, "the teacher's values")):
        if torch.is_grad_enabled() and t is not None and t.requires_grad:
            raise ValueError(f"{name}: the loss has no gradient in them (detach them)")
    return _DistillFunction.apply(_matrix(logits), teacher.values, teacher.indices,
                                  float(temperature), weights)


class DistilledHead:
    """A student's output head in 8 bits, trained against a teacher's top logits.

    ``weight`` [vocab, hidden] is the dense weight (updated by the caller's optimiser from the
    gradients that ``step`` returns; then ``refresh``)."""

    def __init__(self, weight: torch.Tensor, temperature: float = 1.0):
        self.linear = Fp8Linear.from_weight(weight, keep=True)
        self.temperature = float(temperature)

    def logits(self, hidden: torch.Tensor) -> torch.Tensor:
        with torch.no_grad():
            return self.linear(hidden)

    def step(self, hidden: torch.Tensor, teacher: TopLogits,
             weights: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(loss [n], gradient of ``hidden``, gradient of the weight) of the sum of the losses.
        The logits are replaced by their gradient in place."""
        with torch.no_grad():
            logits = _matrix(self.logits(hidden))
            loss, dlogits = G.gptq_distill_loss_grad(logits, teacher.values, teacher.indices,
                                                     self.temperature, weights, dlogits=logits)
            dhidden, dweight = self.linear.backward(dlogits, _matrix(hidden))
        return loss, dhidden.reshape(hidden.shape), dweight

    def refresh(self) -> None:
        self.linear.refresh()


def main() -> None:
    """A small head, disturbed, is pulled back towards its teacher: prints the loss as it falls."""
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    hidden = randn(2048, 1024).bfloat16()
    true = randn(16384, 1024) * 0.1
    teacher = top_logits(hidden.float() @ true.T, 64)
    weight = true + 0.05 * randn(16384, 1024)
    head = DistilledHead(weight)
    share = torch.full((2048,), 1 / 2048, device="cuda")
    for step in range(20):
        loss, _, dweight = head.step(hidden, teacher, share)
        if step % 5 == 0:
            print(f"step {step}: loss {float(loss.sum()):.4f}")
        weight -= 0.5 * dweight
        head.refresh()
    G.gptq_async_status()
    print(f"last: loss {float(head.step(hidden, teacher, share)[0].sum()):.4f}")


if __name__ == "__main__":
    main()
