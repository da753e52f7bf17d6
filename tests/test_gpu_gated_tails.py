"""GPU tests of the activations' tails in fp32: act(g) and its slope keep their
relative accuracy down to fp32's smallest normal value."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F32 = torch.float32
# gates over which the activation falls from 1e-30 to 0
TAIL = {"silu": (-70.0, -125.0), "gelu": (-11.0, -14.5), "gelu_tanh": (-9.0, -13.0)}


def _gates(act, n):
    lo, hi = TAIL[act]
    far = torch.tensor([-200.0, -1e3, -1e5, -2e6, -1e10, -1e20, -1e30, -3e38], device="cuda")
    return torch.cat([torch.linspace(lo, hi, n - far.numel(), device="cuda"), far])


def _off(act, g, v):
    """Bound: 2^-20 of the value (2^-19 of a slope) and, as R.act_error has it, the tanh form's 2^-22 |u|, three times
    in the slope, whose factors p, 1 - p and u' all come from u; results below 2^-126 may be flushed."""
    rel = R.ACT
    if act == "gelu_tanh":
        rel = rel + 3 * 2.0 ** -22 * (1.5957691216057308 * (g + 0.044715 * g ** 3)).abs().clamp(max=130.0)
    return 2 * rel * v.abs() + 2.0 ** -126


@pytest.mark.parametrize("act", sorted(TAIL))
@pytest.mark.parametrize("M", [1, 40, 300])
def test_value(act, M):
    say("tail, value", act, M)
    n = 1000
    g = _gates(act, n)
    x = torch.zeros(M, 8, device="cuda")
    x[:, 0] = 1.0
    wg, wv = torch.zeros(n, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    wg[:, 0], wv[:, 0] = g, 1.0
    none, up = torch.zeros(0, 8, device="cuda"), torch.zeros(n, 0, device="cuda")
    y = L.lora_gated_linear(x, wg, wv, none, up, none, up, 1.0, activation=act)
    a = R.act(act, g.double())[0]
    assert ((a.abs() > 2.0 ** -126) & (a.abs() < 2.0 ** -119)).sum() >= 5
    assert ((y.double() - a).abs() <= _off(act, g.double(), a)).all()


@pytest.mark.parametrize("act", sorted(TAIL))
def test_gradients(act):
    """The slope (dg over dy value) and the value (dv over dy), read back through dx over an identity."""
    say("tail, gradients", act)
    n = 1000
    g = _gates(act, n)[None].expand(3, n).contiguous()
    a, slope = R.act(act, g.double())
    slope = torch.where(g.abs() > 1e30, 0.0, slope)   # (the 64-bit form overflows there)
    assert ((slope.abs() > 2.0 ** -126) & (slope.abs() < 2.0 ** -119)).sum() >= 5
    one = torch.ones(3, n, device="cuda")
    eye, zero = torch.eye(n, device="cuda"), torch.zeros(n, n, device="cuda")
    none, up = torch.zeros(0, n, device="cuda"), torch.zeros(n, 0, device="cuda")
    for wts, want in (((eye, zero), slope), ((zero, eye), a)):
        dx = L.lora_gated_linear_backward(torch.zeros(3, n, device="cuda"), zero, zero, none, up, none, up, 1.0, one, g,
                                          one, activation=act, want_ddown=False, want_dup=False, w_gate_t=wts[0],
                                          w_value_t=wts[1])[0]
        bad = (dx.double() - want).abs() > _off(act, g.double(), want)
        assert not bad.any(), (g[bad][:5], dx[bad][:5], want[bad][:5])
