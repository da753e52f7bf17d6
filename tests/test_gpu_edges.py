"""GPU tests of the 8-bit and update calls at their edges: empty axes, and
updates that are not finite."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _z(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt, device="cuda")


def _codes(n, k):
    q = torch.zeros(n, k, dtype=torch.uint8, device="cuda").view(L.E4M3)
    return q, _z(-(-n // 128), -(-k // 128), dt=F32)


@pytest.mark.parametrize("M", [3, 200])
def test_layer_without_features(M):
    """K = 0: y is the bias, the gradients of what exists are zero.  N = 0: dx is zero."""
    say("edges, K = 0 and N = 0", M)
    wq, ws = _codes(48, 0)
    b = torch.randn(48, device="cuda").to(BF16)
    y = L.fp8_lora_linear(_z(M, 0), wq, ws, _z(4, 0), _z(48, 4) + 1, 1.0, b)
    assert torch.equal(y, b.expand(M, 48))
    dx, dd, du = L.fp8_lora_linear_backward(_z(M, 0), _codes(0, 48)[0], ws, _z(4, 0), _z(48, 4) + 1, 1.0, _z(M, 48) + 1)
    assert dx.shape == (M, 0) and dd.shape == (4, 0) and torch.equal(du, _z(48, 4))
    wq, ws = _codes(0, 64)
    assert L.fp8_lora_linear(_z(M, 64), wq, ws, _z(4, 64), _z(0, 4), 1.0).shape == (M, 0)
    dx, dd, du = L.fp8_lora_linear_backward(_z(M, 64) + 1, _codes(64, 0)[0], ws, _z(4, 64) + 1, _z(0, 4), 1.0, _z(M, 0))
    torch.cuda.synchronize()
    assert torch.equal(dx, _z(M, 64)) and torch.equal(dd, _z(4, 64)) and du.shape == (0, 4)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,C", [(8, 64), (64, 8), (24, 9000), (100, 300), (300, 200), (520, 700)])
@pytest.mark.parametrize("coef", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0)])
def test_update_that_is_not_finite(R, C, dt, coef):
    """One NaN or infinity anywhere makes every element of the update NaN."""
    say("edges, not finite", R, C, dt, coef)
    for bad in (float("nan"), float("inf"), float("-inf")):
        g = torch.ones(R, C, dtype=dt, device="cuda")
        g[R // 3, C // 2] = bad
        assert torch.isnan(L.orthogonalize(g, coefficients=coef)).all(), bad


@pytest.mark.parametrize("dt", [BF16, F32])
def test_16_bit_layer_without_features(dt):
    """The same of the layer over a weight as it is."""
    say("edges, K = 0 and N = 0, plain weight", dt)
    z = lambda *s: _z(*s, dt=dt)
    dx, dd, du = L.lora_linear_backward(z(3, 0), z(48, 0), z(4, 0), z(48, 4) + 1, 1.0, z(3, 48) + 1)
    assert dx.shape == (3, 0) and dd.shape == (4, 0) and torch.equal(du, z(48, 4))
    dx, dd, du = L.lora_linear_backward(z(3, 64) + 1, z(0, 64), z(4, 64) + 1, z(0, 4), 1.0, z(3, 0))
    torch.cuda.synchronize()
    assert torch.equal(dx, z(3, 64)) and torch.equal(dd, z(4, 64)) and du.shape == (0, 4)
