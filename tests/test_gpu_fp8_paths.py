"""GPU tests of every path of the 8-bit product -- each tile, with and without a
K split (and with a last split that is empty), 8-bit and widened sums, with and
without the LoRA fold -- against the definition in 64 bits on sampled rows,
which take in the edges of the tiles."""
import numpy as np
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import fp8_ref as R
from tests.gpu_cases import say
from tests.test_gpu_fp8_sums import _aligned

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

# rows, features, K, rank, activations' and factors' dtype (y is fp32 where one is)
CASES = [
    (4861, 2576, 848, 100, BF16, BF16), (4099, 4112, 1168, 5, F16, F16), (4861, 2576, 848, 256, F16, F16),
    (3301, 5568, 800, 24, BF16, F32), (3301, 5568, 800, 24, F32, F32), (2845, 1440, 5584, 130, BF16, F32),
    (777, 4112, 4112, 5, F16, F16), (777, 4112, 4112, 64, BF16, BF16), (1227, 1040, 6000, 16, F16, F16),
    (339, 2080, 5136, 33, BF16, BF16), (73, 2160, 5184, 7, F16, F16), (73, 2160, 5184, 200, BF16, BF16),
    (649, 2992, 3728, 40, F16, F32), (79, 6208, 7264, 9, BF16, F32), (73, 2160, 5184, 3, F32, F32),
    (33, 16, 512, 1, F16, F16), (1092, 192, 1040, 12, BF16, BF16), (35, 16, 912, 16, F16, F16),
    (155, 144, 3232, 20, BF16, BF16), (127, 1024, 8192, 65, F16, F16), (735, 608, 816, 128, F32, F32),
    (2229, 48, 1648, 18, BF16, F32), (122, 240, 2432, 70, F16, F32), (63, 64, 8192, 256, F32, F32),
]
# the product alone, features that are no multiple of anything (rows of y stored by element)
RAGGED = [(4861, 2573, 848, F16), (4095, 4097, 1040, BF16), (777, 4101, 4112, F16), (777, 4101, 4112, F32),
          (2501, 2500, 2512, BF16), (1227, 1037, 6000, BF16), (73, 2159, 5184, F16), (100, 203, 528, BF16),
          (155, 143, 3232, F16), (2845, 1437, 5584, F32), (122, 237, 2432, F32)]


def _rows(M):
    edges = [0, 1, 63, 64, 127, 128, 255, 256, M // 256 * 256 - 1, M // 256 * 256, M // 64 * 64, M - 2, M - 1]
    return np.unique([m for m in edges + list(np.linspace(0, M - 1, 24).astype(int)) if 0 <= m < M])


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std


def _round(v, dt):
    bits, low = (11, -14) if dt == F16 else (8, -126)
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, low) - (bits - 1))
    return np.round(v / step) * step


def _codes_at(q, s, rows):
    """The values that the sampled rows' codes stand for."""
    at = torch.from_numpy(rows).cuda()
    return R.rows_value(q.view(torch.uint8)[at].cpu().numpy(), s[:, at].cpu().numpy())


def _check(name, got, exact, mass, xv, wv, terms, slack=0.0):
    dt = got.dtype
    bound = R.product_bound(exact, mass, terms, dt) + slack
    if dt != F32:
        bound = bound + _aligned(xv, wv)
    err = np.abs(R.f64(got) - exact)
    assert np.all(err <= bound), (name, float((err / bound).max()))


@pytest.mark.parametrize("M,N,K,r,dt,adt", CASES)
def test_forward_and_product(M, N, K, r, dt, adt):
    out = F32 if F32 in (dt, adt) else dt
    plan = L.fp8_linear_plan(M, N, K, L.dtype_code(out))
    say("fp8 paths, forward and product", M, N, K, r, dt, adt, plan)
    scale, rows = 1.25, _rows(M)
    x, w = _rand(M, M, K).to(dt), _rand(N, N, K, std=K ** -0.5)
    down, up = _rand(1, r, K, std=K ** -0.5).to(adt), _rand(2, N, r, std=0.3).to(adt)
    bias = _rand(3, N).to(dt) if r % 2 else None
    wq, ws, _ = L.fp8_quantize_weight(w)
    y, work = L.fp8_lora_linear(x, wq, ws, down, up, scale, bias, return_workspace=True)
    assert y.dtype == out
    h = L.fp8_lora_saved_h(work, x, down, up, bias)
    q, s = L.fp8_quantize_rows(x)
    at = torch.from_numpy(rows).cuda()
    xv, wv = _codes_at(q, s, rows), R.tiles_value(wq.view(torch.uint8).cpu().numpy(), ws.cpu().numpy())
    xe, de, ue = R.f64(x[at]), R.f64(down.to(dt)), R.f64(up.to(dt))
    hr = R.f64(h[at])[:, :r]
    if dt != F32:
        assert np.array_equal(hr, _round(xe @ de.T, dt))
    base, mass = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    b = 0.0 if bias is None else R.f64(bias)
    terms = 128 + -(-K // 128) + 8
    _check("forward", y[at], base + scale * (hr @ ue.T) + b,
           mass + scale * (np.abs(hr) @ np.abs(ue).T) + np.abs(b), xv, wv, terms + r)
    p = L.fp8_linear(q, s, wq, ws, bias, out_dtype=out)
    _check("product", p[at], base + b, mass + np.abs(b), xv, wv, terms)


@pytest.mark.parametrize("M,N,K,r,dt,adt", CASES)
def test_dx(M, N, K, r, dt, adt):
    """dx [M][N] of a layer of K features out: the product over K as planned
    for an M x N output of x's dtype."""
    plan = L.fp8_linear_plan(M, N, K, L.dtype_code(dt))
    say("fp8 paths, dx", M, N, K, r, dt, adt, plan)
    scale, rows = 0.75, _rows(M)
    x, w = torch.zeros(M, N, dtype=dt, device="cuda"), _rand(N + 1, K, N, std=K ** -0.5)
    down, up = _rand(4, r, N, std=0.3).to(adt), _rand(5, K, r, std=K ** -0.5).to(adt)
    dy = _rand(M + 2, M, K).to(dt)
    _, ws, wqt = L.fp8_quantize_weight(w, transposed=True)
    dx, _, _ = L.fp8_lora_linear_backward(x, wqt, ws, down, up, scale, dy, want_ddown=False, want_dup=False)
    assert dx.dtype == dt
    q, s = L.fp8_quantize_rows(dy)
    at = torch.from_numpy(rows).cuda()
    gv = _codes_at(q, s, rows)
    wv = R.tiles_value(wqt.view(torch.uint8).cpu().numpy(), ws.t().contiguous().cpu().numpy())   # W^T [N][K]
    ge, de, ue = R.f64(dy[at]), R.f64(down.to(dt)), R.f64(up.to(dt))
    gh = scale * (ge @ ue)
    slack = 0.0
    if dt == F32:   # gh stays in fp32, its own sums' errors are part of the bound
        slack = (2.0 ** -23 * (K + 4) * scale * (np.abs(ge) @ np.abs(ue))) @ np.abs(de)
    else:
        gh = _round(gh, dt)
    _check("dx", dx[at], gv @ wv.T + gh @ de, np.abs(gv) @ np.abs(wv).T + np.abs(gh) @ np.abs(de), gv, wv,
           128 + -(-K // 128) + r + 8, slack)


@pytest.mark.parametrize("M,N,K,out", RAGGED)
def test_ragged_product(M, N, K, out):
    say("fp8 paths, ragged product", M, N, K, out, L.fp8_linear_plan(M, N, K, L.dtype_code(out)))
    rows = _rows(M)
    q, s = L.fp8_quantize_rows(_rand(M, M, K).to(BF16))
    wq, ws, _ = L.fp8_quantize_weight(_rand(N, N, K, std=K ** -0.5))
    bias = _rand(3, N).to(BF16 if out == F32 else out)
    room = torch.full((M + 2, N), 7.0, dtype=out, device="cuda")
    y = L.fp8_linear(q, s, wq, ws, bias, out=room[1:M + 1])
    at = torch.from_numpy(rows).cuda()
    xv, wv = _codes_at(q, s, rows), R.tiles_value(wq.view(torch.uint8).cpu().numpy(), ws.cpu().numpy())
    b = R.f64(bias)
    _check("product", y[at], xv @ wv.T + b, np.abs(xv) @ np.abs(wv).T + np.abs(b), xv, wv, 128 + -(-K // 128) + 8)
    assert (room[0] == 7).all() and (room[-1] == 7).all()


@pytest.mark.parametrize("M,N,K,out", [(4861, 2576, 848, BF16), (777, 4112, 4112, F16), (155, 144, 3232, F16),
                                       (73, 2160, 5184, BF16), (2845, 1440, 5584, F32)])
def test_repeats_itself(M, N, K, out):
    """The same bits from call to call, in a workspace full of NaN too."""
    say("fp8 paths, repeated", M, N, K, out)
    q, s = L.fp8_quantize_rows(_rand(M, M, K).to(BF16))
    wq, ws, _ = L.fp8_quantize_weight(_rand(N, N, K, std=K ** -0.5))
    first = L.fp8_linear(q, s, wq, ws, out_dtype=out)
    dirty = torch.full((max(256, L.fp8_linear_workspace_size(M, N, K)),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        assert torch.equal(L.fp8_linear(q, s, wq, ws, out_dtype=out, workspace=dirty), first)
