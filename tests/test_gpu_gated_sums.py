"""GPU tests of the gated block's fp32 products over long sums: summed in blocks of
b = 512, n products are off by about sqrt(b / 2 + n / 2b) 2^-25 of the result.

Each fused step rounds a partial sum once, by at most half an ulp: 2^-24 of it at
most, 2^-24.8 in the mean square.  The terms are independent, so a partial sum of
k of them has sqrt(k / n) of the result's norm, and the squares of the roundings
add up to (b / 2 + n / 2b) 2^-49.6: 5.6e-7 for n = 8192, 5.9e-7 for 16384.  The
bound here is 8e-7; as chains of a quarter of n they were off by 1.1e-6 and more."""
import math

import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests import test_gpu_gated as G
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F32 = torch.float32
BOUND = 8e-7


def _off(a, b):
    return float(torch.linalg.norm(a.double() - b) / torch.linalg.norm(b))


@pytest.mark.parametrize("M,N", [(1, 512), (12, 512), (20, 512), (32, 264), (40, 520), (300, 512), (1200, 1032), (517, 2056)])
def test_projections(M, N):
    K = 8192
    say("long sums, forward", M, N, L.lora_gated_plan(M, N, K, L.F32))
    t = G._inputs(M, N, K, 8, F32, F32, F32, F32)
    y, gate, value, h = L.lora_gated_linear(*G._args(t), 1.5, t["bias_gate"], t["bias_value"], keep=True)
    for k, got in (("gate", gate), ("value", value)):
        ref = R.project(t["x"], t["w_" + k], t["down_" + k], t["up_" + k], 1.5, t["bias_" + k], F32)[0]
        assert _off(got, ref) <= BOUND, (k, _off(got, ref))


@pytest.mark.parametrize("M,K", [(1, 512), (12, 512), (20, 520), (32, 264), (40, 512), (300, 512), (1500, 1024)])
def test_dx(M, K):
    """dx is one sum over the features of both projections."""
    N = 8192
    say("long sums, dx", M, K, L.lora_gated_plan(M, N, K, L.F32, True))
    t = G._inputs(M, N, K, 8, F32, F32, F32)
    dy, gate, value = G._rand(7, M, N), G._rand(8, M, N), G._rand(9, M, N)
    dx = L.lora_gated_linear_backward(*G._args(t), 1.5, dy, gate, value, want_ddown=False, want_dup=False)[0]
    a, slope = R.act("silu", gate.double())
    ref = 0.0
    for k, d in (("gate", dy.double() * value.double() * slope), ("value", dy.double() * a)):
        gh = 1.5 * (d @ t["up_" + k].double())
        ref = ref + d @ t["w_" + k].double() + gh @ t["down_" + k].double()
    assert _off(dx, ref) <= BOUND, _off(dx, ref)
