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


def _z(*s, dt):
    return torch.zeros(*s, dtype=dt, device="cuda")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("given", ["", "h", "w", "wh"])
def test_backward_without_features(dt, M, given):
    """K = 0: no dx, no gradient of the downs, zeros for the ups (h is zero).  N = 0: zeros for dx and the downs."""
    say("gated backward, empty axes", dt, M, given)
    rp = 16 if dt == BF16 else 32

    def call(N, K):
        w = (_z(N, K, dt=dt), _z(N, K, dt=dt))
        factors = (_z(4, K, dt=dt) + 1, _z(N, 4, dt=dt) + 1) * 2
        kw = {"w_gate_t": _z(K, N, dt=dt), "w_value_t": _z(K, N, dt=dt)} if "w" in given else {}
        if "h" in given:
            kw["h"] = _z(M, 2 * rp, dt=dt)
        d = _z(M, N, dt=dt) + 1
        return L.lora_gated_linear_backward(_z(M, K, dt=dt) + 1, *w, *factors, 1.5, d, d, d, **kw)

    dx, ddg, dug, ddv, duv = call(48, 0)
    assert dx.shape == (M, 0) and ddg.shape == (4, 0) and ddv.shape == (4, 0)
    assert torch.equal(dug, _z(48, 4, dt=dt)) and torch.equal(duv, _z(48, 4, dt=dt))
    dx, ddg, dug, ddv, duv = call(0, 64)
    assert dug.shape == (0, 4) and duv.shape == (0, 4)
    assert torch.equal(dx, _z(M, 64, dt=dt)) and torch.equal(ddg, _z(4, 64, dt=dt)) and torch.equal(ddv, _z(4, 64, dt=dt))


def test_nothing_wanted():
    t = G._inputs(70, 72, 64, 4, BF16, BF16, BF16)
    _, gate, value, h = L.lora_gated_linear(*G._args(t), 1.0, keep=True)
    got = L.lora_gated_linear_backward(*G._args(t), 1.0, gate, gate, value, h=h, want_dx=False, want_ddown=False,
                                       want_dup=False)
    assert got == (None,) * 5


@pytest.mark.parametrize("M,N,K", [(0, 48, 64), (5, 0, 64), (5, 48, 0), (200, 48, 0), (200, 0, 64)])
def test_int8_without_rows_or_features(M, N, K):
    say("int8, empty axes", M, N, K)
    q, s = L.int8_quantize_rows(_z(M, K, dt=BF16))
    assert q.shape == (M, K) and torch.equal(s, torch.full_like(s, 2.0 ** -100 / 127.0))
    a, sa = L.int8_quantize_rows(_z(N, K, dt=F32))
    b = torch.randn(N, device="cuda").to(BF16)
    y = L.int8_linear(q, s, a, sa, b)
    assert torch.equal(y, b.expand(M, N))
    y = L.int8_gated_linear(q, s, a, sa, a, sa, b, b, activation="silu", out_dtype=F32)
    want = (b.double() * b.double().sigmoid() * b.double()).expand(M, N)
    assert ((y.double() - want).abs() <= 2.0 ** -19 * want.abs()).all()


@pytest.mark.parametrize("c", [F16, BF16])
@pytest.mark.parametrize("wide", ["down", "up"])
@pytest.mark.parametrize("M", [1, 20, 200])
@pytest.mark.parametrize("r", [5, 16])
def test_factors_of_two_dtypes(c, wide, M, r):
    """One factor of each projection in fp32, the other in 16 bits: what is kept and the gradients are those of the
    rounded factor, but for the dtype of the fp32 factor's gradient."""
    say("factors of two dtypes", c, wide, M, r)
    t = G._inputs(M, 136, 72, r, c, c, F32)
    for n in ("gate", "value"):
        k = ("up_" if wide == "down" else "down_") + n
        t[k] = t[k].to(c)
    low = {k: v.to(c) if v is not None else None for k, v in t.items()}
    y, gate, value, h = L.lora_gated_linear(*G._args(t), 1.5, keep=True)
    y0, gate0, value0, h0 = L.lora_gated_linear(*G._args(low), 1.5, keep=True)
    assert y.dtype == F32 and y0.dtype == c
    for a, b in ((gate, gate0), (value, value0), (h, h0)):
        assert torch.equal(a, b)
    dy = G._rand(3, M, 136).to(c)
    for kept in (None, h):
        got = L.lora_gated_linear_backward(*G._args(t), 1.5, dy, gate, value, h=kept)
        want = L.lora_gated_linear_backward(*G._args(low), 1.5, dy, gate, value, h=kept)
        dts = (c,) + ((F32, c) if wide == "down" else (c, F32)) * 2
        for g, w, dt in zip(got, want, dts):
            assert g.dtype == dt and torch.equal(g.to(c), w)
