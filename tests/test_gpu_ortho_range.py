"""GPU tests of the orthogonalized update far from unit size: norms around and
far below eps, coefficients that shrink or grow the iterate, zero updates."""
import pytest
import torch

import lora_bypass_linear_amd as L
from tests import ortho_ref as O
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = O.F16, O.BF16, O.F32

# up to 16, 32, 64 and 128 (one and several chunks a workgroup), and dense
SHAPES = [(8, 200), (300, 24), (40, 170), (100, 9000), (150, 300), (520, 250)]


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-7, 1.0])
def test_zero(R, C, dt, eps):
    """A zero update gives zeros, whatever eps is."""
    say("ortho range, zero", R, C, dt, eps)
    z = torch.zeros(R, C, dtype=dt, device="cuda")
    for steps in (1, 5):
        assert torch.equal(L.orthogonalize(z, steps=steps, eps=eps), z)


def _check(g, **kw):
    e = O.exact(g, **kw)
    assert torch.isfinite(e).all() and float(e.abs().max()) < 2e38
    out = L.orthogonalize(g, steps=kw.get("steps", 5), coefficients=kw.get("coef", O.COEF), eps=kw.get("eps", 1e-7))
    tol, n = O.tolerance(g, e, **kw), float(e.norm())
    off = float((out.to(O.F64) - e).norm())
    print(tuple(g.shape), g.dtype, "off %.3g tolerance %.3g of the norm %.3g" % (off / n, tol / n, n))
    assert off <= tol, (off / n, tol / n)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("norm", [1e-7, 1e-9, 1e-12, 1e-14, 1e-16, 1e-20, 1e-28])
def test_norms_below_eps(R, C, dt, norm):
    """X0 = G / (|G| + eps) far below 1 with the usual eps: every bit of it is
    held, and the result is an ordinary number of the dtype."""
    say("ortho range, below eps", R, C, dt, norm)
    g = O.update(R + C, R, C, F32, device="cuda")
    _check((g * (norm / float(g.norm()))).to(dt))


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dt,eps", [(F16, 0.5), (F16, 10.0), (BF16, 1e3), (F32, 9e5)])
def test_large_eps(R, C, dt, eps):
    say("ortho range, large eps", R, C, dt, eps)
    g = O.update(R + C, R, C, F32, device="cuda")
    _check((g * (1.0 / float(g.norm()))).to(dt), eps=eps)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("coef,steps", [((0.25, 0.0, 0.0), 20), ((0.1, 0.02, -0.01), 9), ((-1e-4, 0.0, 0.0), 5),
                                        ((1e-12, 0.0, 0.0), 2), ((0.5, -0.3, 0.1), 32)])
def test_shrinking_coefficients(R, C, dt, coef, steps):
    say("ortho range, shrinking", R, C, dt, coef, steps)
    _check(O.update(R + C, R, C, dt, device="cuda"), coef=coef, steps=steps)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("coef,steps", [((10.0, 0.0, 0.0), 12), ((-100.0, 0.0, 0.0), 7), ((3.0, 1.0, 0.0), 4),
                                        ((1e6 * 0.99, 0.0, 0.0), 2), ((1.0, 0.5, 0.25), 3)])
def test_growing_coefficients(R, C, dt, coef, steps):
    """Iterates of up to about 1e18."""
    say("ortho range, growing", R, C, dt, coef, steps)
    _check(O.update(R + C, R, C, dt, device="cuda"), coef=coef, steps=steps)
