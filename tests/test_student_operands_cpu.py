"""Operands that the 8-bit layer's, the top logits' and the distillation's calls refuse: pointers off
their elements' alignment (no GPU needed)."""

import pytest

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
