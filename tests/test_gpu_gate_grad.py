"""GPU tests of dg and dv, the gradients of the gated block's two projections: in
16 bits they are the exact values' roundings, to the bit, over every gate.

They are read back through dx: without a rank, with x in fp32, one projection's
weight the identity and the other's zero, dx is that projection's d (whose
products with zeros need finite values, so the inputs keep both gradients
finite)."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests.gpu_cases import say
from tests.test_gpu_gated import _rand

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
ACTS = ["silu", "gelu", "gelu_tanh"]


def _grads(act, dy, gate, value):
    """(dg, dv) as the backward rounds them, in 64 bits."""
    M, N = gate.shape
    c = gate.dtype
    eye, zero = torch.eye(N, dtype=c, device="cuda"), torch.zeros(N, N, dtype=c, device="cuda")
    none, up = torch.zeros(0, N, dtype=c, device="cuda"), torch.zeros(N, 0, dtype=c, device="cuda")
    x = torch.zeros(M, N, device="cuda")
    out = []
    for a, b in ((eye, zero), (zero, eye)):
        dx = L.lora_gated_linear_backward(x, zero, zero, none, up, none, up, 1.0, dy, gate, value, activation=act,
                                          want_ddown=False, want_dup=False, w_gate_t=a, w_value_t=b)[0]
        assert dx.dtype == F32
        out.append(dx.double())
    return out


def _check(act, dy, gate, value):
    c = gate.dtype
    a, slope = R.act(act, gate.double())
    w = (dy.double() * value.double()).abs()
    d64 = dy.double() * value.double() * slope, dy.double() * a
    # What 64 bits leave open: each evaluation (a quotient, an exponential, a few products and one sum, whose terms
    # are at most 1.2 near its zero) is off by some 2^-53 of itself, 2^-48 bounds it, and 2^-50 of dy value where the
    # sum's terms cancel.  It matters at ties only: beside a gate g below 2^-53 the slope is 1/2 + g / 2 (gelu: + 0.8 g),
    # which 64 bits round to 1/2, while dy value / 2 has 16 bits and is a tie of bf16 once in 2^8 (the same above the
    # gates where the slope or act(g) / g is 1 to 64 bits).
    off = 2.0 ** -48 * d64[0].abs() + torch.where(gate.double().abs() < 2.0, 2.0 ** -50 * w, 0.0), 2.0 ** -48 * d64[1].abs()
    top = torch.finfo(c).max
    assert all((R.nearest(d, c).abs() <= top).all() for d in d64)
    for name, got, d, o in zip(("dg", "dv"), _grads(act, dy, gate, value), d64, off):
        # (dx is an fp32 result: below 2^-126 it may be flushed)
        lo, hi = R.nearest(d - o, c), R.nearest(d + o, c)
        assert int((lo != hi).sum()) <= gate.numel() // 64
        bad = torch.where(d.abs() < 2.0 ** -126, got.abs() > 2.0 ** -126, (got != lo) & (got != hi))
        assert not bad.any(), (name, int(bad.sum()), gate[bad][:4], dy[bad][:4], value[bad][:4], got[bad][:4], d[bad][:4])


def _every(c):
    """Every finite value of a 16-bit type, 256 x 256 (infinities and NaNs as zeros)."""
    g = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(c).view(256, 256)
    return torch.where(torch.isfinite(g), g, torch.zeros_like(g))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("c", [F16, BF16])
@pytest.mark.parametrize("wide", [False, True], ids=["dy16", "dy32"])
def test_every_gate(act, c, wide):
    say("gate grad, every gate", act, c, wide)
    gate = _every(c)
    for seed in range(3):
        dy = _rand(seed, 256, 256).clamp(-3, 3) / (gate.float().abs() / 1000.0).clamp(min=1.0)
        _check(act, dy.to(F32 if wide else c), gate, _rand(seed + 9, 256, 256).to(c))


@pytest.mark.parametrize("M,N", [(1, 8), (5, 72), (3, 264), (65, 264), (130, 136)])
@pytest.mark.parametrize("c", [F16, BF16])
def test_odd_sizes(M, N, c):
    say("gate grad, sizes", M, N, c)
    for act in ACTS:
        _check(act, _rand(1, M, N).to(c), (2.0 * _rand(2, M, N)).to(c), _rand(3, M, N).to(c))


@pytest.mark.parametrize("act,at", [("silu", -1.2784645), ("gelu", -0.7517915), ("gelu_tanh", -0.7524614)])
@pytest.mark.parametrize("c", [F16, BF16])
def test_slopes_that_cancel(act, at, c):
    """Every gate next to the activation's minimum, where the slope is a difference of like terms: thousands of
    elements of each 16384 lie within fp32's error of a border."""
    say("gate grad, slope 0", act, c)
    gate = torch.full((256, 256), at, device="cuda").to(c)
    assert float(R.act(act, gate.double())[1].abs().max()) < 2e-3
    for wide in (False, True):
        _check(act, _rand(4, 256, 256).to(F32 if wide else c), gate, _rand(5, 256, 256).to(c))


# where the activation and its slope fall below the smallest normal fp32 value: gates from, to
FAR = {"silu": (-80.0, -140.0), "gelu": (-12.0, -14.5), "gelu_tanh": (-9.5, -12.5)}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("c,dy,v", [(BF16, 1e30, 1e7), (BF16, 3e37, 1.0), (BF16, 1.0, 3e37), (F16, 3e37, 100.0),
                                    (F16, 1e32, 1.0)])
def test_far_gates(act, c, dy, v):
    """Tiny slopes times large factors."""
    say("gate grad, far gates", act, c, dy, v)
    lo, hi = FAR[act]
    gate = torch.linspace(lo, hi, 128 * 128, device="cuda").view(128, 128).to(c)
    dyt = (_rand(6, 128, 128).clamp(-2, 2) * dy).to(BF16 if c == BF16 else F32)
    vt = (_rand(7, 128, 128).clamp(-2, 2) * v).to(c)
    a, slope = R.act(act, gate.double())
    top = float(torch.finfo(c).max)
    # (both gradients finite: what would pass the type's range is made zero)
    past = ((dyt.double() * vt.double() * slope).abs() > top / 2) | ((dyt.double() * a).abs() > top / 2)
    dyt = torch.where(past, torch.zeros_like(dyt), dyt)
    _check(act, dyt, gate, vt)


@pytest.mark.parametrize("act,lo,hi", [("silu", -24.0, -60.0), ("gelu", -6.5, -11.0), ("gelu_tanh", -5.0, -8.5)])
@pytest.mark.parametrize("wide", [False, True], ids=["dy16", "dy32"])
def test_products_past_the_range(act, lo, hi, wide):
    """dy value passes fp32's range and the slope brings it back."""
    say("gate grad, dy v past the range", act, wide)
    gate = torch.linspace(lo, hi, 128 * 128, device="cuda").view(128, 128).to(BF16)
    a, slope = R.act(act, gate.double())
    dy = (_rand(8, 128, 128).sign() * (1.0 + torch.rand(128, 128, device="cuda")) * 1e25).to(F32 if wide else BF16)
    # a value that brings dg to about 1e35
    v = (1e35 / (dy.double().abs() * slope.abs())).clamp(max=1e38).to(BF16)
    assert ((dy.double() * v.double()).abs() > 3.5e38).any()
    _check(act, dy, gate, v)
