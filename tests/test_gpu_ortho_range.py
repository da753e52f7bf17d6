"""GPU tests of the orthogonalized update far from unit size: norms around and
far below eps, coefficients that shrink or grow the iterate, zero updates."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import ortho_ref as O
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = O.F16, O.BF16, O.F32

# up to 16, 32, 64 and 128 (one and several chunks a workgroup), and dense
SHAPES = [(8, 200), (300, 24), (40, 170), (100, 9000), (150, 300), (520, 250)]


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-7, 1.0])
def test_zero(R, C, dt, eps):
    """A zero update gives zeros, whatever eps is."""
    say("ortho range, zero", R, C, dt, eps)
    z = torch.zeros(R, C, dtype=dt, device="cuda")
    for steps in (1, 5):
        assert torch.equal(L.orthogonalize(z, steps=steps, eps=eps), z)
