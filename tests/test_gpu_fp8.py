"""GPU tests of the 8-bit base-weight operators against their definitions in
64 bits: codes and scales bit for bit, products within the bound of their own
roundings, gradients against the formulas and against differences."""
import numpy as np
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import fp8_ref as R
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _rand(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64) * std


def _bits(q):
    return q.cpu().view(torch.uint8).numpy()


# ---- quantization ------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (17, 272), (16, 256), (130, 400), (5, 4112)])
def test_rows_bit_for_bit(M, K, dt):
    x = (_rand(M * 7 + K, M, K) * torch.exp(_rand(K, M, 1))).to(dt)
    say("fp8 rows", M, K, dt)
    q, s = L.fp8_quantize_rows(x.cuda())
    codes, scales = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(q), codes)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("N,K,transposed", [(16, 16, True), (1, 16, False), (129, 144, False), (272, 400, True),
                                            (128, 256, True), (333, 128, False)])
def test_tiles_bit_for_bit(N, K, transposed, dt):
    w = _rand(N + K, N, K, std=0.02).to(dt)
    say("fp8 tiles", N, K, transposed, dt)
    q, s, qt = L.fp8_quantize_weight(w.cuda(), transposed=transposed)
    codes, scales = R.quantize_tiles(w)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(q), codes)
    assert (qt is not None) == transposed
    if transposed:
        assert np.array_equal(_bits(qt), codes.T)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_rows_at_every_ratio(dt):
    """Every 8-bit-significand value against every group maximum of that kind:
    the quotients that lie on, or a rounding of the scale away from, a border."""
    top = torch.arange(128, 256, dtype=torch.float64) / 64
    val = torch.arange(128, 256, dtype=torch.float64)
    rows = []
    for sh in (0, 3, 9, 15):   # down into e4m3's subnormal values
        v = (val / 64 * 2.0 ** -sh)
        rows.append(torch.minimum(v[None, :], top[:, None]))
    x = torch.cat(rows)
    x[:, 0] = top.repeat(4)   # the group's maximum
    x[::2] = -x[::2]
    x = x.to(dt)
    say("fp8 rows, every ratio", dt)
    q, s = L.fp8_quantize_rows(x.cuda())
    codes, scales = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(q), codes)


def test_rows_zeros_tiny_and_largest():
    x = torch.zeros(6, 256, dtype=F32)
    x[0, 128:] = 3.0                      # a zero group beside another
    x[1] = 2.0 ** -140                    # subnormal, below the floor
    x[2, 5] = torch.finfo(F32).max
    x[3, 7] = -0.0
    x[4] = 2.0 ** -100 * (1 + torch.arange(256) / 512)
    x[5] = torch.finfo(F32).tiny
    say("fp8 rows, zeros, tiny, largest")
    q, s = L.fp8_quantize_rows(x.cuda())
    codes, scales = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(q), codes)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_rows_not_finite(dt):
    x = torch.ones(4, 384, dtype=dt)
    x[1, 130] = float("inf")
    x[2, 5] = float("nan")
    x[3, 383] = float("-inf")
    say("fp8 rows, not finite", dt)
    q, s = L.fp8_quantize_rows(x.cuda())
    v, s = q.cpu().to(F32), s.cpu()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[1, 1] = bad[2, 0] = bad[3, 2] = True
    for m in range(4):
        for b in range(3):
            group = v[m, b * 128:(b + 1) * 128]
            if bad[m, b]:
                assert not np.isfinite(s[b, m].item()) and bool(torch.isnan(group).all()), (m, b)
            else:
                assert np.isfinite(s[b, m].item()) and torch.equal(group, torch.full_like(group, 448.0)), (m, b)


# ---- the product ---------------------------------------------------------------------

def _quantized(seed, M, N, K):
    x = _rand(seed, M, K).to(F32) * torch.exp(_rand(seed + 1, M, 1)).to(F32)
    w = _rand(seed + 2, N, K, std=K ** -0.5).to(F32)
    q, s = L.fp8_quantize_rows(x.cuda())
    wq, wsc, _ = L.fp8_quantize_weight(w.cuda())
    xv = R.rows_value(_bits(q), s.cpu().numpy())
    wv = R.tiles_value(_bits(wq), wsc.cpu().numpy())
    return q, s, wq, wsc, xv, wv


PRODUCTS = [(1, 1, 16), (1, 128, 128), (2, 17, 144), (7, 129, 272), (16, 1040, 4112), (33, 64, 1040), (64, 64, 2064),
            (65, 200, 128), (130, 260, 144), (257, 300, 528), (300, 520, 4112), (513, 1032, 272), (1100, 2056, 160),
            (2100, 4104, 144)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_product(M, N, K, dt):
    say("fp8 product", M, N, K, dt)
    q, s, wq, wsc, xv, wv = _quantized(M + N + K, M, N, K)
    bias = _rand(5, N).to(dt) if (M + N) % 2 else None
    y = L.fp8_linear(q, s, wq, wsc, None if bias is None else bias.cuda(), out_dtype=dt)
    exact = xv @ wv.T
    mass = np.abs(xv) @ np.abs(wv).T
    if bias is not None:
        exact = exact + R.f64(bias)
        mass = mass + np.abs(R.f64(bias))
    err = np.abs(R.f64(y) - exact)
    bound = R.product_bound(exact, mass, 128 + -(-K // 128) + 8, dt)
    assert np.all(err <= bound), (float((err / bound).max()))


def test_product_of_scales_far_apart():
    """Row and tile scales of very different sizes in neighbouring groups."""
    M, N, K = 70, 300, 656
    say("fp8 product, scales far apart")
    q, s, wq, wsc, _, _ = _quantized(11, M, N, K)
    s = s * torch.exp2(torch.randint(-20, 20, s.shape, generator=torch.Generator().manual_seed(1)).float()).cuda()
    wsc = wsc * torch.exp2(torch.randint(-9, 9, wsc.shape, generator=torch.Generator().manual_seed(2)).float()).cuda()
    xv, wv = R.rows_value(_bits(q), s.cpu().numpy()), R.tiles_value(_bits(wq), wsc.cpu().numpy())
    y = L.fp8_linear(q, s, wq, wsc, out_dtype=F32)
    exact, mass = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.all(np.abs(R.f64(y) - exact) <= R.product_bound(exact, mass, 128 + 6 + 8, F32))


def test_product_leaves_other_rows_alone():
    """A token row that is not finite gives its own outputs only, and an output
    buffer's neighbours stay as they were."""
    M, N, K = 37, 144, 272
    say("fp8 product, one row not finite")
    x = _rand(3, M, K).to(BF16)
    w = _rand(4, N, K, std=0.1).to(BF16)
    wq, wsc, _ = L.fp8_quantize_weight(w.cuda())
    clean = L.fp8_linear(*L.fp8_quantize_rows(x.cuda()), wq, wsc)
    x[9, 200] = float("nan")
    x[20, 0] = float("inf")
    room = torch.full((M + 2, N), 7.0, dtype=BF16, device="cuda")
    y = L.fp8_linear(*L.fp8_quantize_rows(x.cuda()), wq, wsc, out=room[1:M + 1])
    torch.cuda.synchronize()
    assert torch.isnan(y[9]).all() and torch.isnan(y[20]).all()
    keep = [m for m in range(M) if m not in (9, 20)]
    assert torch.equal(y[keep], clean[keep])
    assert (room[0] == 7).all() and (room[-1] == 7).all()


# ---- the LoRA forward and backward ---------------------------------------------------

def _layer(seed, M, N, K, r, dt, adt, bias=False):
    t = dict(x=_rand(seed, M, K).to(dt), w=_rand(seed + 1, N, K, std=K ** -0.5).to(F32),
             down=_rand(seed + 2, r, K, std=K ** -0.5).to(adt), up=_rand(seed + 3, N, r, std=0.3).to(adt),
             dy=_rand(seed + 4, M, N).to(dt), bias=_rand(seed + 5, N).to(dt) if bias else None)
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def _round(v, dt):
    """64 bits to a 16-bit type in one rounding (torch's conversion rounds to 32 bits first)."""
    bits, low = (11, -14) if dt == F16 else (8, -126)
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, low) - (bits - 1))
    return np.round(v / step) * step


LAYERS = [(1, 32, 16, 1), (1, 1040, 2064, 16), (16, 272, 1040, 5), (33, 144, 272, 16), (130, 400, 528, 64),
          (200, 272, 2064, 100), (300, 528, 400, 256), (1030, 1040, 528, 24)]


@pytest.mark.parametrize("M,N,K,r", LAYERS)
@pytest.mark.parametrize("dt,adt", [(F16, F16), (BF16, BF16), (BF16, F32), (F32, F32)])
def test_forward(M, N, K, r, dt, adt):
    say("fp8 forward", M, N, K, r, dt, adt)
    t = _layer(M + K, M, N, K, r, dt, adt, bias=r % 2 == 0)
    wq, wsc, _ = L.fp8_quantize_weight(t["w"])
    scale = 1.5
    y, ws = L.fp8_lora_linear(t["x"], wq, wsc, t["down"], t["up"], scale, t["bias"], return_workspace=True)
    out = F32 if F32 in (dt, adt) else dt
    assert y.dtype == out
    codes, s = R.quantize_rows(t["x"])
    xv, wv = R.rows_value(codes, s), R.tiles_value(_bits(wq), wsc.cpu().numpy())
    xe, de, ue = R.f64(t["x"]), R.f64(t["down"].to(dt)), R.f64(t["up"].to(dt))
    h = L.fp8_lora_saved_h(ws, t["x"], t["down"], t["up"], t["bias"])
    assert (h[:, r:] == 0).all()
    h = R.f64(h[:, :r])
    want_h = xe @ de.T
    if dt == F32:
        assert np.all(np.abs(h - want_h) <= 2.0 ** -23 * (K + 4) * (np.abs(xe) @ np.abs(de).T))
    else:
        assert np.array_equal(h, _round(want_h, dt))
    exact = xv @ wv.T + scale * (h @ ue.T)
    mass = np.abs(xv) @ np.abs(wv).T + scale * (np.abs(h) @ np.abs(ue).T)
    if t["bias"] is not None:
        exact, mass = exact + R.f64(t["bias"]), mass + np.abs(R.f64(t["bias"]))
    err = np.abs(R.f64(y) - exact)
    bound = R.product_bound(exact, mass, 128 + -(-K // 128) + r + 8, out)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("M,N,K,r", LAYERS)
@pytest.mark.parametrize("dt,adt", [(F16, F16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("saved", [False, True])
def test_backward(M, N, K, r, dt, adt, saved):
    say("fp8 backward", M, N, K, r, dt, adt, saved)
    t = _layer(M + N, M, N, K, r, dt, adt)
    wq, wsc, wqt = L.fp8_quantize_weight(t["w"], transposed=True)
    scale = 0.75
    h = None
    if saved:
        _, ws = L.fp8_lora_linear(t["x"], wq, wsc, t["down"], t["up"], scale, return_workspace=True)
        h = L.fp8_lora_saved_h(ws, t["x"], t["down"], t["up"])
    dx, dd, du = L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], scale, t["dy"], h=h)
    assert (dx.dtype, dd.dtype, du.dtype) == (dt, adt, adt)
    codes, s = R.quantize_rows(t["dy"])
    gv, wv = R.rows_value(codes, s), R.tiles_value(_bits(wq), wsc.cpu().numpy())
    xe, ge, de, ue = R.f64(t["x"]), R.f64(t["dy"]), R.f64(t["down"].to(dt)), R.f64(t["up"].to(dt))
    hx, gx = xe @ de.T, scale * (ge @ ue)
    # fp32 compute keeps h and gh in fp32 (their own sums' errors are part of the bound)
    hr, gr = (hx, gx) if dt == F32 else (_round(hx, dt), _round(gx, dt))
    eh = 2.0 ** -23 * (K + 4) * (np.abs(xe) @ np.abs(de).T) if dt == F32 else 0 * hx
    eg = 2.0 ** -23 * (N + 4) * scale * (np.abs(ge) @ np.abs(ue)) if dt == F32 else 0 * gx
    for name, got, exact, mass, slack, terms in (
            ("dx", dx, gv @ wv + gr @ de, np.abs(gv) @ np.abs(wv) + np.abs(gr) @ np.abs(de), eg @ np.abs(de),
             128 + -(-N // 128) + r + 8),
            ("d_down", dd, gr.T @ xe, np.abs(gr).T @ np.abs(xe), eg.T @ np.abs(xe), M + 8),
            ("d_up", du, scale * (ge.T @ hr), scale * (np.abs(ge).T @ np.abs(hr)), scale * (np.abs(ge).T @ eh), M + 8)):
        err = np.abs(R.f64(got) - exact)
        bound = R.product_bound(exact, mass, terms, got.dtype) + slack
        assert np.all(err <= bound), (name, float((err / bound).max()))


def test_backward_against_differences():
    """dDown and dUp against central differences of the fp32 forward, whose
    quantized product they do not pass through; dx through a layer whose
    weight and dy are exact in e4m3 (no quantization error)."""
    M, N, K, r, scale = 6, 32, 48, 3, 0.5
    say("fp8 backward against differences")
    t = _layer(21, M, N, K, r, F32, F32)
    w = torch.from_numpy(R.VALUES[np.random.RandomState(0).randint(80, 100, (N, K))]).to(F32)
    w[0, 0] = 448.0   # scale 1: every weight is its own code
    dy = torch.from_numpy(R.VALUES[np.random.RandomState(1).randint(30, 60, (M, N))]).to(F32)
    dy[:, 0] = 448.0
    wq, wsc, wqt = L.fp8_quantize_weight(w.cuda(), transposed=True)
    assert torch.equal(wsc.cpu(), torch.ones(1, 1))
    t["dy"] = dy.cuda()
    dx, dd, du = L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], scale, t["dy"])

    def loss(x, down, up):   # the layer's formula in 64 bits, no quantization of x
        y = x @ w.double().numpy().T + scale * (x @ down.T) @ up.T
        return float((y * dy.double().numpy()).sum())

    x, d, u = (R.f64(t[k]) for k in ("x", "down", "up"))
    rng = np.random.RandomState(2)
    for name, got, at in (("dx", dx, 0), ("d_down", dd, 1), ("d_up", du, 2)):
        args = [x, d, u]
        for _ in range(12):
            i = tuple(rng.randint(0, n) for n in args[at].shape)
            eps = 1e-4
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[at][i] += eps
            lo[at][i] -= eps
            diff = (loss(*hi) - loss(*lo)) / (2 * eps)
            # bilinear in each argument: the difference is exact up to 64-bit
            # cancellation (2^-53 |loss| / eps); the kernel's sums are fp32
            tol = 1e-10 * abs(loss(*args)) / eps * 1e-2 + 2.0 ** -20 * (abs(diff) + float(np.abs(R.f64(got)).max()))
            assert abs(diff - R.f64(got)[i]) <= tol, (name, i, diff, R.f64(got)[i])


def test_backward_parts_and_rank_zero():
    M, N, K, r = 40, 144, 272, 8
    say("fp8 backward, parts")
    t = _layer(31, M, N, K, r, BF16, BF16)
    wq, wsc, wqt = L.fp8_quantize_weight(t["w"], transposed=True)
    full = L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], 1.0, t["dy"])
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        part = L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], 1.0, t["dy"], want_dx=bool(want[0]),
                                          want_ddown=bool(want[1]), want_dup=bool(want[2]))
        for w, p, f in zip(want, part, full):
            assert (p is None) == (not w)
            if w:
                assert torch.equal(p, f)
    none = torch.empty(0, K, dtype=BF16, device="cuda"), torch.empty(N, 0, dtype=BF16, device="cuda")
    y = L.fp8_lora_linear(t["x"], wq, wsc, *none, 1.0)
    assert torch.equal(y, L.fp8_linear(*L.fp8_quantize_rows(t["x"]), wq, wsc))
    dx, dd, du = L.fp8_lora_linear_backward(t["x"], wqt, wsc, *none, 1.0, t["dy"])
    assert torch.equal(dx, L.fp8_linear(*L.fp8_quantize_rows(t["dy"]), wqt, wsc.t().contiguous()))
    assert dd.numel() == 0 and du.numel() == 0


def test_empty_calls():
    say("fp8 empty calls")
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")
    wq, wsc, wqt = L.fp8_quantize_weight(z(144, 272) + 1, transposed=True)
    q, s = L.fp8_quantize_rows(z(0, 272))
    assert q.shape == (0, 272) and s.shape == (3, 0)
    assert L.fp8_linear(q, s, wq, wsc).shape == (0, 144)
    assert L.fp8_lora_linear(z(0, 272), wq, wsc, z(4, 272), z(144, 4), 1.0).shape == (0, 144)
    dx, dd, du = L.fp8_lora_linear_backward(z(0, 272), wqt, wsc, z(4, 272), z(144, 4), 1.0, z(0, 144))
    torch.cuda.synchronize()
    assert dx.shape == (0, 272) and (dd == 0).all() and (du == 0).all()
    q, s = L.fp8_quantize_rows(z(3, 0))
    w0, s0, _ = L.fp8_quantize_weight(z(144, 0))
    b = _rand(1, 144).to(BF16).cuda()
    assert torch.equal(L.fp8_linear(q, s, w0, s0, b), b.expand(3, 144))


def test_side_stream_and_graph():
    """The calls run on the current stream, and a captured forward and backward
    replay to the eager results, with eager work between the replays."""
    M, N, K, r = 48, 272, 528, 8
    say("fp8 side stream and graph")
    t = _layer(41, M, N, K, r, BF16, BF16, bias=True)
    wq, wsc, wqt = L.fp8_quantize_weight(t["w"], transposed=True)
    call = lambda: (L.fp8_lora_linear(t["x"], wq, wsc, t["down"], t["up"], 0.5, t["bias"]),
                    *L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], 0.5, t["dy"]))
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = call()
    x0 = t["x"].clone()
    for k in range(3):
        t["x"].copy_(x0 * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        eager = call()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), k


def test_offsets_past_32_bits():
    """More than 2^31 elements of x: the last rows come out as they do alone."""
    M, K, N, tail = 270000, 8192, 144, 40
    say("fp8 offsets past 32 bits")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    for i in range(0, M, 30000):
        x[i:i + 30000] = torch.randn(min(30000, M - i), K, generator=g, device="cuda")
    w = _rand(6, N, K, std=K ** -0.5).to(BF16).cuda()
    wq, wsc, _ = L.fp8_quantize_weight(w)
    q, s = L.fp8_quantize_rows(x)
    last = x[M - tail:].clone()
    del x
    q1, s1 = L.fp8_quantize_rows(last)
    assert torch.equal(q[M - tail:].view(torch.uint8), q1.view(torch.uint8))
    assert torch.equal(s[:, M - tail:], s1)
    y = L.fp8_linear(q, s, wq, wsc, out_dtype=F32)[M - tail:]
    xv, wv = R.rows_value(_bits(q1), s1.cpu().numpy()), R.tiles_value(_bits(wq), wsc.cpu().numpy())
    exact, mass = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.all(np.abs(R.f64(y) - exact) <= R.product_bound(exact, mass, 128 + K // 128 + 8, F32))


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("c", [F16, BF16])
def test_fp32_activations_with_16_bit_factors(M, c):
    """x and dy in fp32 beside 16-bit factors: the codes come from them as
    stored, the bypass from them rounded to the compute dtype, y and dx are fp32."""
    N, K, r, scale = 272, 528, 12, 0.5
    say("fp8 fp32 activations", M, c)
    t = _layer(61, M, N, K, r, F32, c)
    wq, wsc, wqt = L.fp8_quantize_weight(t["w"], transposed=True)
    y = L.fp8_lora_linear(t["x"], wq, wsc, t["down"], t["up"], scale)
    dx, dd, du = L.fp8_lora_linear_backward(t["x"], wqt, wsc, t["down"], t["up"], scale, t["dy"])
    assert (y.dtype, dx.dtype, dd.dtype, du.dtype) == (F32, F32, c, c)
    wv = R.tiles_value(_bits(wq), wsc.cpu().numpy())
    xv, gv = R.rows_value(*R.quantize_rows(t["x"])), R.rows_value(*R.quantize_rows(t["dy"]))
    xc, gc = R.f64(t["x"].to(c)), R.f64(t["dy"].to(c))
    de, ue = R.f64(t["down"]), R.f64(t["up"])
    h, gh = _round(xc @ de.T, c), _round(scale * (gc @ ue), c)
    for name, got, exact, mass, terms in (
            ("y", y, xv @ wv.T + scale * (h @ ue.T), np.abs(xv) @ np.abs(wv).T + scale * (np.abs(h) @ np.abs(ue).T),
             128 + 5 + r + 8),
            ("dx", dx, gv @ wv + gh @ de, np.abs(gv) @ np.abs(wv) + np.abs(gh) @ np.abs(de), 128 + 3 + r + 8),
            ("d_down", dd, gh.T @ xc, np.abs(gh).T @ np.abs(xc), M + 8),
            ("d_up", du, scale * (gc.T @ h), scale * (np.abs(gc).T @ np.abs(h)), M + 8)):
        err = np.abs(R.f64(got) - exact)
        bound = R.product_bound(exact, mass, terms, got.dtype)
        assert np.all(err <= bound), (name, float((err / bound).max()))
