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


@pytest.mark.parametrize("size", [(4, 72, 64), (70, 72, 64), (64, 136, 4104), (517, 520, 72), (2100, 4104, 72)], ids=_name)
@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("hit", ["gate", "value"])
def test_an_infinite_h_stays_with_its_projection(size, dt, hit):
    """h of one projection overflows its type: that projection is infinite with the sign of up, the other is what it
    is without the overflow, to the bit."""
    say("infinite h", size, dt, hit)
    M, N, K = size
    other = "value" if hit == "gate" else "gate"
    t = G._inputs(M, N, K, 3, dt, dt, dt)
    big = {F16: 100.0, BF16: 2.0 ** 70, F32: 2.0 ** 70}[dt]
    t["x"] = (t["x"].abs() + 1.0).clamp(max=4.0)
    t["x"][1::2] *= big   # every other token's h overflows
    t["down_" + hit][0] = {F16: 6e4, BF16: 2.0 ** 70, F32: 2.0 ** 70}[dt]
    t["down_" + hit][1:] = 0.0
    t["down_" + other][:] = 0.0
    t["up_" + hit][:, 0] = t["up_" + hit][:, 0].sign() + (t["up_" + hit][:, 0] == 0)
    # (the even tokens of fp16 overflow too: 64 x 6e4 at least)
    rows = slice(0, None) if dt == F16 else slice(1, None, 2)
    kw = dict(activation="silu", keep=True)
    y, gate, value, h = L.lora_gated_linear(*G._args(t), 1.0, **kw)
    kept = {"gate": gate, "value": value}
    clean = dict(t)
    clean["down_" + hit] = torch.zeros_like(t["down_" + hit])
    _, gate0, value0, _ = L.lora_gated_linear(*G._args(clean), 1.0, **kw)
    assert torch.isfinite(kept[other]).all()
    assert torch.equal(kept[other], value0 if hit == "gate" else gate0)
    want = float("inf") * t["up_" + hit][:, 0].sign().double()
    assert torch.equal(kept[hit][rows].double(), want.expand_as(kept[hit][rows]))
    if hit == "gate":   # act(inf) v, and -inf times 0
        up = want > 0
        ref = torch.where(value[rows] == 0, float("nan"), float("inf") * value[rows].double().sign())
        assert torch.equal(y[rows][:, up].double().nan_to_num(nan=7.0), ref[:, up].nan_to_num(nan=7.0))
        assert torch.isnan(y[rows][:, ~up]).all()
