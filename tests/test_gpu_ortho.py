"""GPU tests of the orthogonalized update against the iteration in 64 bits.

Tolerance, of the result's norm: one rounding to the dtype (half a step of
each element), plus the products' own errors.  A step with p(0) = a amplifies
what is off in small singular directions by a, so after `steps` steps an
operand rounding of u is at most u * sqrt(n) * a^steps of the result; u is
2^-21 for 16-bit updates (two fp16 pieces, the dropped product, fp32 sums) and
2^-23 for fp32 ones (three bf16 pieces).  Norm-wise, not element by element:
the errors are the matrix's."""
import numpy as np
import pytest
import torch

import lora_bypass_linear_amd as L
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
COEF = (3.4445, -4.7750, 2.0315)


def _update(seed, R, C, dt, low=-1.0, std=1e-3):
    g = torch.Generator().manual_seed(seed)
    n, m = min(R, C), max(R, C)
    mix = torch.randn(n, n, generator=g, dtype=torch.float64) / n ** 0.5 * torch.logspace(0, low, n, dtype=torch.float64)
    u = (mix + 0.2 * torch.eye(n, dtype=torch.float64)) @ torch.randn(n, m, generator=g, dtype=torch.float64) * std
    return (u if R <= C else u.T).contiguous().to(dt)


def _exact(g, steps=5, coef=COEF, eps=1e-7):
    x = g.to(torch.float64).numpy()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    a, b, c = coef
    for _ in range(steps):
        t = x @ x.T
        x = a * x + (b * t + c * (t @ t)) @ x
    return x.T if tall else x


def _check(g, out, steps=5, coef=COEF, eps=1e-7):
    e = _exact(g, steps, coef, eps)
    n = min(g.shape)
    u = 2.0 ** -23 if g.dtype == F32 else 2.0 ** -21
    amp = max(abs(coef[0]), 1.0) ** steps
    off = np.linalg.norm(out.cpu().to(torch.float64).numpy() - e)
    tiny = 2.0 ** -25 * np.sqrt(e.size) if g.dtype == F16 else 0.0   # fp16's subnormal outputs
    bound = (torch.finfo(g.dtype).eps / 2 + u * np.sqrt(n) * amp) * np.linalg.norm(e) + tiny
    print(tuple(g.shape), g.dtype, "off", off / np.linalg.norm(e), "bound", bound / np.linalg.norm(e))
    assert off <= bound, (off, bound)


SHAPES = [(1, 1), (1, 16), (16, 1), (2, 3), (5, 33), (33, 5), (16, 4096), (17, 1000), (1000, 17), (64, 64), (100, 1030),
          (128, 520), (2056, 128), (129, 300), (200, 200), (257, 130), (300, 1100), (1100, 520)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_against_64_bits(R, C, dt):
    say("ortho", R, C, dt)
    g = _update(R * 3 + C, R, C, dt)
    _check(g, L.orthogonalize(g.cuda()))


@pytest.mark.parametrize("R,C", [(2048, 1024), (1030, 2100)])
def test_large(R, C):
    say("ortho large", R, C)
    g = _update(R, R, C, BF16)
    _check(g, L.orthogonalize(g.cuda()))


@pytest.mark.parametrize("dt,R,C", [(F32, 700, 1001), (F16, 1001, 700), (F32, 1501, 1290), (BF16, 1900, 2061)])
def test_halves_mirrored(dt, R, C):
    """Sizes whose two symmetric products are computed on and below the
    diagonal and mirrored, each tile with ragged edges."""
    say("ortho halves", R, C, dt)
    g = _update(R + C, R, C, dt)
    _check(g, L.orthogonalize(g.cuda()))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 9])
@pytest.mark.parametrize("dt,R,C", [(BF16, 24, 300), (F32, 300, 24), (F16, 150, 200)])
def test_steps(steps, dt, R, C):
    say("ortho steps", steps, dt)
    g = _update(steps, R, C, dt)
    _check(g, L.orthogonalize(g.cuda(), steps=steps), steps=min(steps, 9)) if steps < 9 else \
        _check_near_one(g, L.orthogonalize(g.cuda(), steps=steps))


def _check_near_one(g, out):
    """Many steps: the singular values lie in the coefficients' band about 1."""
    s = torch.linalg.svdvals(out.cpu().to(torch.float64))
    assert s.max() < 1.4 and s.min() > 0.3, (s.min(), s.max())


@pytest.mark.parametrize("coef,steps", [((1.5, -0.5, 0.0), 5), ((2.0, -1.5, 0.5), 4), ((0.25, 0.0, 0.0), 3)])
def test_other_coefficients(coef, steps):
    say("ortho coefficients", coef)
    for dt, R, C in ((BF16, 40, 200), (F32, 130, 60)):
        g = _update(7, R, C, dt)
        _check(g, L.orthogonalize(g.cuda(), steps=steps, coefficients=coef), steps, coef)


@pytest.mark.parametrize("dt,R,C", [(BF16, 32, 256), (F16, 300, 200), (F32, 64, 100)])
def test_spectra(dt, R, C):
    """One direction that outweighs the rest, a rank-deficient update, and
    scales near the dtype's ends."""
    say("ortho spectra", dt, R, C)
    g = torch.Generator().manual_seed(3)
    n = min(R, C)
    one = torch.outer(torch.randn(R, generator=g), torch.randn(C, generator=g)) * 3 + 0.01 * torch.randn(R, C, generator=g)
    low = torch.randn(R, n // 4, generator=g) @ torch.randn(n // 4, C, generator=g)
    for u in (one, low, _update(1, R, C, F32, low=-3.0, std=1.0)):
        u = u.to(dt)
        _check(u, L.orthogonalize(u.cuda()))
    if dt != F16:
        for f in (1e-30, 1e30):
            u = (torch.randn(R, C, generator=g) * f).to(dt)
            _check(u, L.orthogonalize(u.cuda(), eps=0.0), eps=0.0)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,C", [(8, 64), (300, 200), (64, 8)])
def test_zero_and_not_finite(dt, R, C):
    say("ortho zero and not finite", dt, R, C)
    z = torch.zeros(R, C, dtype=dt, device="cuda")
    assert torch.equal(L.orthogonalize(z), z)
    for bad in (float("nan"), float("inf")):
        g = torch.ones(R, C, dtype=dt, device="cuda")
        g[R // 2, C // 2] = bad
        assert torch.isnan(L.orthogonalize(g)).any()
    assert L.orthogonalize(torch.zeros(0, C, dtype=dt, device="cuda")).shape == (0, C)


def test_in_place_dirty_workspace_stream_and_graph():
    say("ortho in place, dirty workspace, stream, graph")
    for dt, R, C in ((BF16, 20, 300), (F32, 90, 37), (F16, 200, 150)):
        g = _update(5, R, C, dt).cuda()
        want = L.orthogonalize(g)
        ws = torch.full((L.orthogonalize_workspace_size(R, C, L.dtype_code(g)),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(L.orthogonalize(g, workspace=ws), want)   # (0xFF bytes: NaN in every type)
        mine = g.clone()
        assert L.orthogonalize(mine, out=mine) is mine and torch.equal(mine, want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = L.orthogonalize(g)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = L.orthogonalize(g)
        g0 = g.clone()
        for k in range(3):
            g.copy_(g0.roll(k, dims=1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, L.orthogonalize(g)), k


def test_neighbours_stay():
    say("ortho neighbours")
    room = torch.full((2 + 33 * 21,), 7.0, dtype=BF16, device="cuda")
    g = _update(9, 33, 21, BF16).cuda()
    out = room[1:-1].view(33, 21)   # element-aligned only
    L.orthogonalize(g, out=out)
    assert torch.equal(out, L.orthogonalize(g)) and room[0] == 7 and room[-1] == 7
