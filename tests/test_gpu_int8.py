"""GPU tests of the 8-bit integer operators against their definitions in 64 bits:
codes and scales exactly, products within the roundings that the definition
leaves, on every path (few rows, each tile, K splits) and at ragged sizes."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def _guarded(shape, dt, off=1):
    """An output whose rows start off elements past an aligned address, between marked elements."""
    n = shape[0] * shape[1]
    buf = torch.full((n + 64 + off,), 7.0, dtype=dt, device="cuda")
    return buf, buf[off:off + n].view(shape)


def _untouched(buf, off, n):
    return bool((buf[:off] == 7.0).all()) and bool((buf[off + n:] == 7.0).all())


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (17, 1040), (5, 4096), (2, 4112), (9, 8192), (4, 8208), (3, 20000),
                                 (300, 272), (0, 64), (4, 0)])
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_rows(M, K, dt):
    say("int8 rows", M, K, dt)
    x = (_rand(M * 7 + K, M, K) * torch.exp(_rand(1, M, 1))).to(dt)
    if M > 2 and K:
        x[1] = 0.0
        x[2] *= 2.0 ** -14 if dt == F16 else 2.0 ** -110
    q, s = L.int8_quantize_rows(x)
    qr, sr = R.int8_rows(x) if K else (torch.zeros(M, 0, dtype=torch.int8, device="cuda"),
                                       torch.full((M,), 2.0 ** -100 / 127.0, device="cuda"))
    assert torch.equal(s, sr) and torch.equal(q, qr)


def test_rows_on_the_borders():
    """Every quotient c + 1/2 and its neighbours: scales that are powers of two make exact ties."""
    for dt in (F16, BF16, F32):
        say("int8 ties", dt)
        t = torch.arange(-127, 127, device="cuda").float() + 0.5
        row = torch.cat([torch.tensor([127.0, -127.0], device="cuda"), t])
        near = torch.cat([row, torch.nextafter(row, torch.full_like(row, 1e9)), torch.nextafter(row, -torch.full_like(row, 1e9))])
        near[256], near[512] = 127.0, 127.0   # (nothing past the largest)
        near = near.clamp(-127.0, 127.0)
        x = torch.cat([near, torch.zeros((-near.numel()) % 16, device="cuda")])
        x = torch.stack([x * 2.0 ** e for e in (-8, 0, 6)] + [x * 0.3, x * 1.7]).to(dt)
        q, s = L.int8_quantize_rows(x)
        qr, sr = R.int8_rows(x)
        assert torch.equal(s, sr) and torch.equal(q, qr)


def test_rows_that_are_not_finite():
    x = _rand(3, 4, 64)
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    for dt in (F16, BF16, F32):
        q, s = L.int8_quantize_rows(x.to(dt))
        assert torch.isinf(s[1]) and torch.isnan(s[2]) and not q[1:3].any() and torch.isfinite(s[[0, 3]]).all()
        y = L.int8_linear(q, s, *L.int8_quantize_rows(_rand(4, 24, 64)), out_dtype=F32)
        assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3]]).all()


# rows, features, K
SHAPES = [(1, 1, 16), (1, 8192, 4096), (2, 33, 64), (7, 130, 1040), (16, 257, 144), (17, 100, 80), (31, 515, 2064),
          (32, 64, 16), (33, 48, 4096), (64, 512, 8192), (65, 67, 272), (129, 1000, 528), (200, 3001, 208),
          (300, 2056, 1040), (777, 1025, 1040), (1030, 2500, 144), (2100, 2057, 528), (4100, 4097, 272), (40, 24, 0),
          (3, 24, 0), (600, 700, 16), (5, 8200, 80), (20, 8193, 64),
          (500, 1500, 528), (900, 1800, 2064)]


def _operands(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    def r(n):
        return torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8)
    s = torch.exp(_rand(seed, M)) * 0.01
    return r(M), s, r(N), torch.exp(_rand(seed + 1, N)) * 0.01, r(N), torch.exp(_rand(seed + 2, N)) * 0.01


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    q, s, w, ws, _, _ = _operands(M, N, K, M + N + K)
    for dt, bdt in ((BF16, None), (F16, F32), (F32, BF16)):
        say("int8 product", M, N, K, dt, bdt, L.int8_linear_plan(M, N, K))
        b = None if bdt is None else _rand(9, N).to(bdt)
        g, eg = R.int8_project(q, s, w, ws, b)
        if dt == F16:   # (sums of any codes reach past its range)
            s, f = s * 2.0 ** -12, 2.0 ** -12
            g, eg = R.int8_project(q, s, w, ws, b)
        buf, out = _guarded((M, N), dt)
        y = L.int8_linear(q, s, w, ws, b, out=out)
        bad = (y.double() - g).abs() > eg + R.U[dt] * (g.abs() + eg) + R.TINY[dt]
        assert y is out and not bad.any(), int(bad.sum())
        assert _untouched(buf, 1, M * N)
        assert torch.equal(y, L.int8_linear(q, s, w, ws, b, out_dtype=dt))


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated(M, N, K, act):
    q, s, wg, sg, wv, sv = _operands(M, N, K, M + N + K)
    top = max(1.0, 128.0 * 128.0 * K ** 0.5)
    s = s / top * 300.0   # (projections of a few units: both sides of the activation)
    for dt, bdt in ((BF16, None), (F16, F16), (F32, F32)):
        say("int8 gated", M, N, K, act, dt, bdt, L.int8_gated_plan(M, N, K))
        bg, bv = (None, None) if bdt is None else (_rand(8, N).to(bdt), _rand(9, N).to(bdt))
        g, eg = R.int8_project(q, s, wg, sg, bg)
        v, ev = R.int8_project(q, s, wv, sv, bv)
        ref = R.act(act, g)[0] * v
        buf, out = _guarded((M, N), dt)
        y = L.int8_gated_linear(q, s, wg, sg, wv, sv, bg, bv, activation=act, out=out)
        bad = (y.double() - ref).abs() > R.block_bound(act, g, eg, v, ev, ref, dt)
        assert not bad.any(), int(bad.sum())
        assert _untouched(buf, 1, M * N)
        assert torch.equal(y, L.int8_gated_linear(q, s, wg, sg, wv, sv, bg, bv, activation=act, out_dtype=dt))


def test_sums_are_exact():
    """The longest contraction of the largest codes fills 31 bits; few rows and a tile agree to the bit."""
    K = 131056
    say("int8 longest", K)
    x = torch.full((40, K), -128, dtype=torch.int8, device="cuda")
    x[:, ::3] = 127
    w = torch.full((24, K), -128, dtype=torch.int8, device="cuda")
    w[5, 1::2] = 127
    one = torch.ones(40, device="cuda")
    y = L.int8_linear(x, one, w, one[:24], out_dtype=F32)
    ref = (x.cpu().double() @ w.cpu().double().t()).float()
    assert torch.equal(y.cpu(), ref)
    few = L.int8_linear(x[:20].contiguous(), one[:20], w, one[:24], out_dtype=F32)
    assert torch.equal(few.cpu(), ref[:20])


def test_empty():
    z = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt, device="cuda")
    assert L.int8_linear(z(0, 32), z(0, dt=F32), z(8, 32), z(8, dt=F32)).shape == (0, 8)
    assert L.int8_gated_linear(z(4, 32), z(4, dt=F32), z(0, 32), z(0, dt=F32), z(0, 32), z(0, dt=F32)).shape == (4, 0)


@pytest.mark.parametrize("M", [1, 3, 4, 6, 1001])
@pytest.mark.parametrize("K", [16, 112, 1008, 1024, 1040])
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_short_rows(M, K, dt):
    """One wave a row, and the first length past it: also rows that are not finite."""
    say("int8 short rows", M, K, dt)
    x = (_rand(M + K, M, K) * torch.exp(_rand(1, M, 1))).to(dt)
    q, s = L.int8_quantize_rows(x)
    qr, sr = R.int8_rows(x)
    assert torch.equal(s, sr) and torch.equal(q, qr)
    if M > 2:
        x[0, K - 1], x[2, 0] = float("nan"), float("-inf")
        q2, s2 = L.int8_quantize_rows(x)
        assert bool(torch.isnan(s2[0])) and bool(torch.isinf(s2[2])) and not q2[0].any() and not q2[2].any()
        assert torch.equal(q2[1], qr[1]) and torch.equal(q2[3:], qr[3:]) and torch.equal(s2[3:], sr[3:])


@pytest.mark.parametrize("M,K", [((1 << 24) + 5, 16), ((1 << 26) + 3, 16), ((1 << 22) + 1, 1040)])
def test_many_rows(M, K):
    """More rows than one grid dimension has workgroups for, on both kernels."""
    say("int8 many rows", M, K)
    x = torch.randint(-100, 101, (M, K), device="cuda", dtype=torch.int8).to(BF16)
    q, s = L.int8_quantize_rows(x)
    for rows in (slice(0, 9), slice((1 << 22) - 5, (1 << 22) + 9), slice(M - 9, M)):
        qr, sr = R.int8_rows(x[rows])
        assert torch.equal(s[rows], sr) and torch.equal(q[rows], qr)
    assert bool((q.abs().amax(1)[:: 1 << 10] == 127).all())
