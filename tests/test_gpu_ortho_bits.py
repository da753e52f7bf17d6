"""GPU tests of the orthogonalized update to the bits its operands are held in:
every tile, side and split of the dense products, and thin updates whose long
side takes several chunks a workgroup."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import ortho_ref as O
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = O.F16, O.BF16, O.F32

DENSE2 = [(129, 129), (135, 129), (133, 399), (399, 133), (367, 370), (370, 367), (1097, 1140), (1217, 769),
          (769, 1217), (1413, 1457), (1457, 1413), (450, 5047), (5047, 450), (521, 7300), (7300, 521), (1040, 5555),
          (5555, 1040), (1948, 1999), (2041, 4090), (4090, 2041)]
DENSE3 = [(129, 129), (135, 129), (225, 267), (267, 225), (1097, 1140), (771, 1459), (1459, 771), (397, 4886),
          (4886, 397), (1948, 1999), (1999, 1948), (2200, 2315), (2315, 2200)]
DENSE = [(dt, R, C) for i, (R, C) in enumerate(DENSE2) for dt in ((F16, BF16) if R * C < 1e6 else (F16, BF16)[i % 2:][:1])]
DENSE += [(F32, R, C) for R, C in DENSE3]

# the long side past what one chunk for each of 32 or 128 workgroups covers
THIN = [(dt, R, C) for dt in (F16, BF16, F32)
        for R, C in ((1, 9000), (7, 20011), (20011, 7), (16, 8192), (19, 9001), (9001, 30), (33, 17000), (17000, 64),
                     (70, 20011), (20011, 128), (128, 8200), (3, 5), (128, 128), (17, 17))]


def _check(g, out, **kw):
    e = O.exact(g, **kw)
    tol = O.tolerance(g, e, **kw)
    off = float((out.to(O.F64) - e).norm())
    n = float(e.norm())
    print(tuple(g.shape), g.dtype, "off %.3g tolerance %.3g (rounding %.3g) of the norm" % (
        off / n, tol / n, O.rounding(e, g.dtype) / n))
    assert off <= tol, (off / n, tol / n)


@pytest.mark.parametrize("dt,R,C", DENSE)
def test_dense(dt, R, C):
    say("ortho bits, dense", dt, R, C)
    g = O.update(R + C, R, C, dt, device="cuda")
    _check(g, L.orthogonalize(g))


@pytest.mark.parametrize("dt,R,C", THIN)
def test_thin(dt, R, C):
    say("ortho bits, thin", dt, R, C)
    g = O.update(R + C, R, C, dt, device="cuda")
    _check(g, L.orthogonalize(g))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("n,m", [(9, 20011), (24, 9001), (60, 17000), (100, 17000)])
def test_thin_chunks_of_unlike_sizes(dt, n, m):
    """Chunks that a workgroup takes in turn: growing, shrinking and zero ones
    between others."""
    say("ortho bits, unlike chunks", dt, n, m)
    g = O.update(n + m, n, m, F32, std=1.0)
    at = torch.arange(m) // 64
    f = torch.exp2(((at * 7) % 11 - 5).float())
    f[at % 5 == 3] = 0.0
    f[(at >= 40) & (at < 60)] = 0.0
    for u in (g * f, (g * f).flip(1), (g * f).t().contiguous()):
        u = u.contiguous().to(dt).cuda()
        _check(u, L.orthogonalize(u))


@pytest.mark.parametrize("dt,R,C,steps", [(F16, 30, 500, 1), (F16, 100, 300, 4), (F32, 70, 900, 3), (F16, 200, 600, 2),
                                          (F32, 300, 200, 6), (F16, 12, 900, 6)])
def test_steps(dt, R, C, steps):
    say("ortho bits, steps", dt, R, C, steps)
    g = O.update(steps, R, C, dt, device="cuda")
    _check(g, L.orthogonalize(g, steps=steps), steps=steps)
