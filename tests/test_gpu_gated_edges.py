"""GPU tests of the gated block at the edges of what its calls allow: operands
narrowed where nothing else is prepared, single misaligned factors."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import test_gpu_gated as G
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

# fp32 x or W under 16-bit compute and no factors to prepare: without a rank, and where few rows read both factors as
# they are stored
CASTS = [
    (5, 136, 72, 0, BF16, F32, BF16, None, "silu"), (300, 264, 136, 0, BF16, F32, BF16, BF16, "gelu"),
    (40, 136, 72, 0, F32, F16, F16, None, "silu"), (300, 264, 136, 0, F32, BF16, BF16, BF16, "gelu_tanh"),
    (260, 136, 72, 0, F16, F32, F32, F32, "silu"),
    (20, 136, 72, 16, BF16, F32, BF16, None, "silu"), (1, 264, 136, 16, F16, F32, F16, F16, "gelu"),
    (120, 264, 136, 32, F32, F16, F16, None, "gelu_tanh"), (33, 72, 264, 64, F32, BF16, BF16, BF16, "silu"),
    (20, 136, 72, 16, F32, F32, BF16, None, "silu"),
]


def _name(c):
    return "-".join(str(v).replace("torch.", "") for v in c)


@pytest.mark.parametrize("case", CASTS, ids=_name)
def test_operands_narrowed_alone(case):
    G.test_forward(case)


@pytest.mark.parametrize("case", [
    (20, 72, 64, 16, F32, BF16, BF16, BF16, "silu", ""), (1, 136, 72, 32, F32, F16, F16, F16, "gelu", ""),
    (100, 264, 136, 16, F32, BF16, BF16, F32, "gelu_tanh", "w"), (128, 72, 264, 5, F32, F16, F16, F16, "silu", ""),
    (40, 72, 64, 0, F32, BF16, BF16, BF16, "silu", "w"),
], ids=_name)
def test_backward_that_narrows_x_alone(case):
    G.test_backward(case)


@pytest.mark.parametrize("M", [3, 20, 200])
@pytest.mark.parametrize("which", ["up_gate", "up_value", "down_gate", "down_value"])
@pytest.mark.parametrize("wdt", [BF16, F32])
def test_one_factor_off_16_bytes(M, which, wdt):
    """A factor that starts between two 16-byte boundaries is read as its aligned twin is."""
    say("misaligned", M, which, wdt)
    t = G._inputs(M, 136, 72, 16, BF16, wdt, BF16)
    want = L.lora_gated_linear(*G._args(t), 1.5, keep=True)
    odd = torch.empty(t[which].numel() + 1, dtype=BF16, device="cuda")[1:].view(t[which].shape)
    odd.copy_(t[which])
    assert odd.data_ptr() % 16 == 2
    t[which] = odd
    for a, b in zip(L.lora_gated_linear(*G._args(t), 1.5, keep=True), want):
        assert torch.equal(a, b)
