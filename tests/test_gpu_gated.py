"""GPU tests of the gated feed-forward block, forward and backward, against its
definition in 64 bits: every path (few rows, each tile, K splits), odd ranks,
every dtype policy, and gradients against differences too."""
import math

import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E = 2.0 ** -24


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def _inputs(M, N, K, r, xdt, wdt, adt, bdt=None, seed=0):
    sd = 1.0 / math.sqrt(max(K, 1))
    t = {"x": (_rand(seed, M, K) * torch.exp(0.5 * _rand(seed + 1, M, 1))).to(xdt)}
    for i, n in enumerate(("gate", "value")):
        t["w_" + n] = _rand(seed + 10 + i, N, K, std=sd).to(wdt)
        t["down_" + n] = _rand(seed + 20 + i, r, K, std=sd).to(adt)
        t["up_" + n] = _rand(seed + 30 + i, N, r, std=0.3 / math.sqrt(max(r, 1))).to(adt)
        t["bias_" + n] = None if bdt is None else _rand(seed + 40 + i, N, std=0.3).to(bdt)
    return t


def _args(t):
    return [t[k] for k in ("x", "w_gate", "w_value", "down_gate", "up_gate", "down_value", "up_value")]


# rows, features, K, rank, x, W and factors' dtypes, bias, activation
FORWARD = [
    (1, 8, 8, 1, F16, F16, F16, None, "silu"), (1, 1025, 1032, 16, BF16, BF16, BF16, None, "silu"),
    (2, 33, 72, 5, F16, F16, F16, F16, "gelu"), (16, 520, 264, 16, BF16, BF16, BF16, BF16, "gelu_tanh"),
    (17, 100, 1032, 17, F16, F16, F16, None, "silu"), (32, 257, 136, 33, BF16, BF16, BF16, None, "gelu"),
    (33, 72, 2056, 64, F16, F16, F16, F16, "silu"), (64, 130, 4104, 100, BF16, BF16, BF16, None, "gelu_tanh"),
    (129, 1001, 520, 128, F16, F16, F16, F16, "gelu"), (128, 48, 264, 256, BF16, BF16, BF16, BF16, "silu"),
    (300, 2056, 1040, 5, F16, F16, F16, None, "silu"), (517, 515, 328, 129, BF16, BF16, BF16, None, "gelu"),
    (777, 1030, 136, 200, F16, F16, F16, F16, "gelu_tanh"), (2100, 4100, 264, 16, BF16, BF16, BF16, BF16, "silu"),
    (2050, 4097, 136, 40, F16, F16, F16, F16, "gelu"), (4100, 2064, 72, 256, BF16, BF16, BF16, None, "gelu_tanh"),
    (300, 264, 136, 0, BF16, BF16, BF16, BF16, "silu"), (5, 264, 136, 0, F16, F16, F16, None, "gelu"),
    (20, 136, 72, 16, BF16, F32, F32, F32, "silu"), (260, 520, 264, 24, F32, F32, F16, None, "silu"),
    (200, 264, 136, 8, F16, F32, F16, F16, "gelu_tanh"), (600, 1032, 136, 64, BF16, BF16, F32, None, "gelu"),
    (1, 64, 72, 3, F32, F32, F32, None, "gelu"), (31, 100, 520, 32, F32, F32, F32, F32, "silu"),
    (200, 333, 264, 40, F32, F32, F32, F32, "gelu_tanh"), (517, 2056, 136, 5, F32, F32, F32, None, "silu"),
    (40, 64, 4096, 16, F32, F32, F32, None, "silu"), (50, 72, 0, 4, BF16, BF16, BF16, BF16, "silu"),
    (3, 72, 0, 0, F16, F16, F16, F16, "silu"), (1100, 1101, 264, 7, F16, F16, F16, None, "silu"),
    (1024, 2048, 264, 3, F32, F32, F32, None, "silu"),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_forward(case):
    M, N, K, r, xdt, wdt, adt, bdt, act = case
    t = _inputs(M, N, K, r, xdt, wdt, adt, bdt)
    code = [L.dtype_code(v) for v in t.values() if v is not None]
    c_dt, o_dt = L.resolve_dtypes(code)
    c, o = L.torch_dtype(c_dt), L.torch_dtype(o_dt)
    say("gated forward", case, L.lora_gated_plan(M, N, K, c_dt))
    scale = 1.5
    n = M * N
    buf = torch.full((n + 65,), 7.0, dtype=o, device="cuda")
    out = buf[1:1 + n].view(M, N)
    y, gate, value, h = L.lora_gated_linear(*_args(t), scale, t["bias_gate"], t["bias_value"], activation=act, out=out,
                                            keep=True)
    assert y is out and bool((buf[:1] == 7.0).all()) and bool((buf[1 + n:] == 7.0).all())
    assert torch.equal(y, L.lora_gated_linear(*_args(t), scale, t["bias_gate"], t["bias_value"], activation=act))
    p, e = {}, {}
    for i, k in enumerate(("gate", "value")):
        p[k], e[k], hr, eh = R.project(t["x"], t["w_" + k], t["down_" + k], t["up_" + k], scale, t["bias_" + k], c)
        kept = (gate, value)[i]
        assert kept.dtype == c
        bad = (kept.double() - p[k]).abs() > e[k] + R.U[c] * (p[k].abs() + e[k]) + R.TINY[c]
        assert not bad.any(), (k, int(bad.sum()))
        if r:
            rp = R.r_pad(r, c)
            assert h.shape == (M, 2 * rp) and h.dtype == c
            half = h[:, i * rp:(i + 1) * rp].double()
            assert not half[:, r:].any()
            assert ((half[:, :r] - hr).abs() <= eh).all()
    if r == 0:
        assert h is None
    ref = R.act(act, p["gate"])[0] * p["value"]
    bad = (y.double() - ref).abs() > R.block_bound(act, p["gate"], e["gate"], p["value"], e["value"], ref, o)
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_over_its_range(act):
    """One feature per g from far below to far above, through an identity projection in fp32."""
    say("activation range", act)
    g = torch.cat([torch.linspace(-30, 30, 4006, device="cuda"), torch.logspace(-30, 4, 500, device="cuda"),
                   -torch.logspace(-30, 4, 500, device="cuda"),
                   torch.tensor([0.0, -0.0, 86.9, 87.1, 200.0, -86.9, -87.1, -200.0, 3e38, -3e38], device="cuda")])
    n = g.numel()
    x = torch.zeros(1, 8, device="cuda")
    x[0, 0] = 1.0
    w_gate, w_value = torch.zeros(n, 8, device="cuda"), torch.zeros(n, 8, device="cuda")
    w_gate[:, 0], w_value[:, 0] = g, 1.0
    none, up = torch.zeros(0, 8, device="cuda"), torch.zeros(n, 0, device="cuda")
    y, kept, _, _ = L.lora_gated_linear(x, w_gate, w_value, none, up, none, up, 1.0, activation=act, keep=True)
    assert torch.equal(kept[0], g + 0.0)
    a, slope = R.act(act, g.double())
    big = g.abs() > 1e30   # (64-bit slope forms overflow there)
    # (below u = -87 the logistic factor counts as 0: |g| p(u) is at most 87 exp(-87) = 1.43e-36 < 2^-119 there)
    assert ((y[0].double() - a).abs() <= R.act_error(act, g.double()) + 2.0 ** -119).all()
    dy = torch.ones(1, n, device="cuda")
    # (the slopes come back through dx over an identity weight, 1024 at a time)
    idx = torch.arange(n, device="cuda")
    got = torch.empty(n, device="cuda", dtype=torch.float64)
    for k in range(0, n, 1024):
        part = idx[k:k + 1024]
        eye = torch.zeros(part.numel() + (-part.numel()) % 8, n, device="cuda")
        eye[torch.arange(part.numel(), device="cuda"), part] = 1.0
        kk = eye.shape[0]
        dxk = L.lora_gated_linear_backward(torch.zeros(1, kk, device="cuda"), torch.zeros(n, kk, device="cuda"),
                                           torch.zeros(n, kk, device="cuda"), torch.zeros(0, kk, device="cuda"), up,
                                           torch.zeros(0, kk, device="cuda"), up, 1.0, dy, kept, torch.ones_like(kept),
                                           activation=act, want_ddown=False, want_dup=False, w_gate_t=eye,
                                           w_value_t=torch.zeros_like(eye))[0]
        got[part] = dxk[0, :part.numel()].double()
    ok = (got - slope).abs() <= 2.0 ** -19 * (1.0 + g.abs().double().clamp(max=100.0))
    assert ok[~big].all() and torch.isfinite(got).all()


def test_values_that_are_not_finite():
    """A NaN or an infinity reaches its own outputs only."""
    say("not finite")
    for M in (4, 70):
        t = _inputs(M, 72, 64, 4, BF16, BF16, BF16)
        clean = L.lora_gated_linear(*_args(t), 1.0)
        t["x"][1, 3], t["x"][2, 5] = float("nan"), float("inf")
        y = L.lora_gated_linear(*_args(t), 1.0)
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_an_infinite_gate(act, dt):
    """act(inf) is inf; -inf times 0 is a NaN, as in the formulas."""
    say("infinite gate", act, dt)
    for M in (3, 70):
        t = _inputs(M, 64, 64, 2, dt, dt, dt, dt)
        t["bias_gate"][5], t["bias_gate"][6] = float("inf"), -float("inf")
        y = L.lora_gated_linear(*_args(t), 1.0, t["bias_gate"], t["bias_value"], activation=act)
        v = R.project(t["x"], t["w_value"], t["down_value"], t["up_value"], 1.0, t["bias_value"], dt)[0]
        assert torch.equal(y[:, 5].double(), float("inf") * torch.sign(v[:, 5])) and torch.isnan(y[:, 6]).all()
        assert torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 7:]).all()


# rows, features, K, rank, x, W, factors' and dy's dtypes, activation, what is given
BACKWARD = [
    (1, 8, 8, 1, F16, F16, F16, F16, "silu", "wh"), (1, 1032, 520, 16, BF16, BF16, BF16, BF16, "silu", "wh"),
    (7, 264, 136, 5, F16, F16, F16, F16, "gelu", ""), (32, 72, 264, 33, BF16, BF16, BF16, BF16, "gelu_tanh", "w"),
    (33, 136, 72, 16, F16, F16, F16, F16, "silu", "h"), (130, 520, 264, 100, BF16, BF16, BF16, BF16, "gelu", "wh"),
    (300, 2064, 1040, 5, F16, F16, F16, F16, "silu", "wh"), (517, 264, 2056, 129, BF16, BF16, BF16, BF16, "silu", ""),
    (2100, 136, 4104, 64, BF16, BF16, BF16, BF16, "gelu_tanh", "wh"), (4100, 72, 2064, 256, F16, F16, F16, F16, "gelu", "h"),
    (777, 1032, 1032, 16, BF16, BF16, F32, F32, "silu", "wh"), (200, 264, 136, 24, BF16, F32, F32, F32, "gelu", ""),
    (260, 136, 264, 8, F32, F32, F16, F16, "silu", "w"), (260, 136, 264, 8, F32, BF16, BF16, BF16, "silu", ""),
    (300, 264, 136, 0, BF16, BF16, BF16, BF16, "silu", "w"),
    (1, 72, 64, 3, F32, F32, F32, F32, "gelu", "wh"), (31, 136, 520, 32, F32, F32, F32, F32, "silu", ""),
    (200, 328, 264, 40, F32, F32, F32, F32, "gelu_tanh", "wh"), (517, 136, 1032, 200, F32, F32, F32, F32, "silu", ""),
    (64, 2048, 72, 16, BF16, BF16, BF16, BF16, "silu", "wh"), (1500, 264, 1544, 20, BF16, BF16, BF16, BF16, "silu", "wh"),
    (1030, 72, 2056, 40, F32, F32, F32, F32, "gelu", "w"), (5, 72, 8200, 8, F16, F16, F16, F16, "silu", "wh"),
    (20, 72, 8200, 40, BF16, BF16, F32, F32, "gelu_tanh", ""), (1024, 136, 4096, 16, F32, F32, F32, F32, "silu", "w"),
]


def _backward(t, scale, dy, kept, act, given, c, **kw):
    if "w" in given:
        kw["w_gate_t"], kw["w_value_t"] = (t[k].to(c).t().contiguous() for k in ("w_gate", "w_value"))
    if "h" in given:
        kw["h"] = kept[2]
    return L.lora_gated_linear_backward(*_args(t), scale, dy, kept[0], kept[1], activation=act, **kw)


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_backward(case):
    M, N, K, r, xdt, wdt, adt, gdt, act, given = case
    t = _inputs(M, N, K, r, xdt, wdt, adt)
    c_dt, _ = L.resolve_dtypes([L.dtype_code(v) for v in t.values() if v is not None] + [L.dtype_code(torch.empty(0, dtype=gdt))])
    c = L.torch_dtype(c_dt)
    say("gated backward", case, L.lora_gated_plan(M, N, K, c_dt, True))
    scale, u = 1.5, R.U[c]
    _, gate, value, h = L.lora_gated_linear(*_args(t), scale, activation=act, keep=True)
    kept = (gate.to(c), value.to(c), h if h is None or h.dtype == c else h.to(c))
    dy = (_rand(77, M, N) * torch.exp(0.5 * _rand(78, M, 1))).to(gdt)
    dx, *grads = _backward(t, scale, dy, kept, act, given, c)
    assert dx.dtype == xdt and all(g.dtype == adt for g in grads)
    again = _backward(t, scale, dy, kept, act, given, c)
    assert all(torch.equal(a, b) for a, b in zip((dx, *grads), again))

    # the definition: d rounded once from 64 bits.  The kernel rounds its own fp32 value, which lies on the other
    # side of a border now and then: off by 2 u |d| there, never by more than that plus its own error.
    a, slope = R.act(act, kept[0].double())
    d64 = {"gate": dy.double() * kept[1].double() * slope, "value": dy.double() * a}
    err = {"gate": (dy.double() * kept[1].double()).abs() * 2.0 ** -19 * (1.0 + kept[0].double().abs()),
           "value": dy.double().abs() * R.act_error(act, kept[0].double())}
    rp = R.r_pad(r, c)
    ref_dx, bnd_dx = 0.0, 0.0
    for i, n in enumerate(("gate", "value")):
        d = R.nearest(d64[n], c)
        off = err[n] * (1 + u) + 2 * u * d.abs() + R.TINY[c]
        wc = t["w_" + n].to(c).double()
        ref_dx = ref_dx + d @ wc
        bnd_dx = bnd_dx + (off + (2 * N + r + 4) * E * d.abs()) @ wc.abs()
        if not r:
            continue
        dc, uc = t["down_" + n].to(c).double(), t["up_" + n].to(c).double()
        gh, eg = R.low_rank(scale * d, uc, c)
        goff = eg + scale * (off @ uc.abs()) + 2 * u * gh.abs() + R.TINY[c]
        ref_dx = ref_dx + gh @ dc
        bnd_dx = bnd_dx + (goff + (2 * N + 2 * r + 4) * E * gh.abs()) @ dc.abs()
        xc = t["x"].to(c).double()
        dd, du = grads[2 * i], grads[2 * i + 1]
        ref = gh.t() @ xc
        bnd = (goff + (M + 4) * E * gh.abs()).t() @ xc.abs()
        bad = (dd.double() - ref).abs() > bnd + R.U[adt] * (ref.abs() + bnd) + R.TINY[adt]
        assert not bad.any(), ("d_down", n, int(bad.sum()))
        hr, hoff = R.low_rank(xc, dc.t(), c)
        if "h" in given:
            hr, hoff = kept[2][:, i * rp:i * rp + r].double(), 0.0 * hr
        ref = scale * (d.t() @ hr)
        bnd = scale * ((off + (M + 4) * E * d.abs()).t() @ (hr.abs() + hoff) + d.abs().t() @ hoff) + 2 * E * ref.abs()
        bad = (du.double() - ref).abs() > bnd + R.U[adt] * (ref.abs() + bnd) + R.TINY[adt]
        assert not bad.any(), ("d_up", n, int(bad.sum()))
    bad = (dx.double() - ref_dx).abs() > bnd_dx + R.U[xdt] * (ref_dx.abs() + bnd_dx) + R.TINY[xdt]
    assert not bad.any(), ("dx", int(bad.sum()))
    # all of it together, far below the worst case: the output's rounding, and the few d on the other side of a border
    norm = torch.linalg.norm
    assert norm(dx.double() - ref_dx) <= (R.U[xdt] + 0.5 * u + 40 * E) * norm(ref_dx) + 1e-30


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [5, 70])
def test_gradients_against_differences(act, M):
    """<gradient, direction> against a central difference of the 64-bit loss sum(y dy) along it."""
    say("gated differences", act, M)
    N, K, r, scale = 72, 64, 4, 1.5
    t = _inputs(M, N, K, r, F32, F32, F32)
    dy = _rand(5, M, N)
    _, gate, value, h = L.lora_gated_linear(*_args(t), scale, activation=act, keep=True)
    dx, ddg, dug, ddv, duv = L.lora_gated_linear_backward(*_args(t), scale, dy, gate, value, activation=act, h=h)
    grads = {"x": dx, "down_gate": ddg, "up_gate": dug, "down_value": ddv, "up_value": duv}

    def loss(v):
        p = [v["x"] @ v["w_" + n].t() + scale * ((v["x"] @ v["down_" + n].t()) @ v["up_" + n].t())
             for n in ("gate", "value")]
        return float((R.act(act, p[0])[0] * p[1] * dy.double()).sum())

    full = {k: v.double() for k, v in t.items() if v is not None}
    for k, g in grads.items():
        u = _rand(91, *g.shape).double()
        eps = 1e-5
        lo, hi = dict(full), dict(full)
        lo[k], hi[k] = full[k] - eps * u, full[k] + eps * u
        want, got = (loss(hi) - loss(lo)) / (2 * eps), float((g.double() * u).sum())
        # differences: eps^2 of third derivatives; gradients: fp32 sums and kept values
        assert abs(got - want) <= 1e-5 * float(g.double().norm() * u.norm()), (k, got, want)


def test_wanted_gradients_alone():
    t = _inputs(70, 72, 64, 16, BF16, BF16, BF16)
    _, gate, value, h = L.lora_gated_linear(*_args(t), 1.0, keep=True)
    dy = _rand(6, 70, 72).to(BF16)
    full = L.lora_gated_linear_backward(*_args(t), 1.0, dy, gate, value, h=h)
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        say("gated want", want)
        got = L.lora_gated_linear_backward(*_args(t), 1.0, dy, gate, value, h=h, want_dx=want[0], want_ddown=want[1],
                                           want_dup=want[2])
        for g, f, w in zip(got, full, (want[0], want[1], want[2], want[1], want[2])):
            assert (g is None) == (not w) and (g is None or torch.equal(g, f))


def test_empty():
    t = _inputs(0, 72, 64, 4, BF16, BF16, BF16)
    y, gate, value, h = L.lora_gated_linear(*_args(t), 1.0, keep=True)
    assert y.shape == (0, 72) and h.shape == (0, 32)
    dx, *grads = L.lora_gated_linear_backward(*_args(t), 1.0, torch.zeros(0, 72, dtype=BF16, device="cuda"), gate, value, h=h)
    assert dx.shape == (0, 64) and not any(g.any() for g in grads)
