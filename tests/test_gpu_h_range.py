"""GPU tests of h = round(x.down^T) where it leaves its type's range or x holds
infinities: it is what the definition in 64 bits rounds to, and zero past the
rank, whatever path computes it."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests import test_gpu_gated as G
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
SIZES = [(3, 72), (70, 264), (200, 72), (517, 136), (2100, 72), (300, 4104)]   # rows, K


def _rounded(h, c):
    out = R.nearest(torch.where(torch.isfinite(h), h, 0.0), c)
    out = torch.where(out.abs() > torch.finfo(c).max, float("inf") * out.sign(), out)
    return torch.where(torch.isfinite(h), out, h)


def _same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=0.0), b.nan_to_num(nan=0.0))


def _h_of_both(t, r, dt, rp):
    """h as lora_linear and as the gated block leave it."""
    a = (t["x"], t["w_gate"], t["down_gate"], t["up_gate"])
    _, ws = L.lora_linear(*a, 1.0, return_workspace=True)
    yield "linear", L.lora_saved_h(ws, *a)
    h = L.lora_gated_linear(*G._args(t), 1.0, keep=True)[3]
    yield "gate", h[:, :rp]
    t = dict(t)
    for k in ("w", "down", "up"):
        t[k + "_gate"], t[k + "_value"] = t[k + "_value"], t[k + "_gate"]
    yield "value", L.lora_gated_linear(*G._args(t), 1.0, keep=True)[3][:, rp:]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("r", [1, 5, 24, 40, 100, 200])
def test_overflow(M, K, r):
    """bf16: sums of products that pass fp32's range, of one sign and of both."""
    say("h overflow", M, K, r)
    rp = R.r_pad(r, BF16)
    t = G._inputs(M, 72, K, r, BF16, BF16, BF16)
    for s in (2.0 ** 62, 2.0 ** 70, 2.0 ** 90):
        t["x"][1::2] = t["x"][1::2].sign() * s
        t["down_gate"][0] = 2.0 ** 70 * t["down_gate"][0].sign()
        h64 = t["x"].double() @ t["down_gate"].double().t()
        want = _rounded(h64, BF16)
        for name, h in _h_of_both(t, r, BF16, rp):
            assert _same(h[:, :r].double(), want), (name, s)
            assert not h[:, r:].any(), (name, s)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("r", [1, 5, 16, 40, 100, 200])
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_infinite_x(M, K, r, dt):
    say("h of infinities", M, K, r, dt)
    rp = R.r_pad(r, dt)
    t = G._inputs(M, 72, K, r, dt, dt, dt)
    clean = {n: h.clone() for n, h in _h_of_both(t, r, dt, rp)}
    assert not (t["down_gate"] == 0).any()
    t["x"][1, 3] = float("inf")
    t["x"][2, 5] = -float("inf")
    t["x"][M - 1, 7], t["x"][M - 1, 60] = float("inf"), float("inf")
    hit = sorted({1, 2, M - 1})
    want = t["x"].double() @ t["down_gate"].double().t()
    rest = [m for m in range(M) if m not in hit]
    for name, h in _h_of_both(t, r, dt, rp):
        assert not torch.isfinite(want[hit]).any()
        assert _same(h[hit, :r].double(), want[hit]), name
        assert not h[:, r:].any(), name
        assert torch.equal(h[rest], clean[name][rest]), name
