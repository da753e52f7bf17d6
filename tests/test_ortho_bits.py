"""The tolerance of the orthogonalized update's GPU tests tells operands held in
all their pieces from operands with one piece less (on the CPU, by emulation),
and the shapes of those tests reach every tile the planner picks."""
import random

import pytest
import torch

import lora_bypass_linear_amd as L
from tests import ortho_ref as O
from tests.test_gpu_ortho_bits import DENSE, THIN


@pytest.mark.parametrize("dt", [O.F16, O.BF16, O.F32])
@pytest.mark.parametrize("R,C", [(8, 700), (24, 600), (600, 24), (100, 530), (200, 333), (333, 200), (450, 701)])
def test_one_piece_less_is_seen(R, C, dt):
    g = O.update(R + C, R, C, dt)
    e = O.exact(g)
    tol = O.tolerance(g, e)
    held = (O.emulate(g, O.BITS[dt]).to(dt).to(O.F64) - e).norm()
    less = (O.emulate(g, O.FEWER[dt]).to(dt).to(O.F64) - e).norm()
    print(R, C, dt, "held", float(held / e.norm()), "tolerance", tol / float(e.norm()), "less", float(less / e.norm()))
    assert held <= tol
    assert less > tol


def _paths(R, C, dt):
    side = "tall" if R > C else "wide"
    return {(p, 3 if dt == L.F32 else 2, tn, tm, "" if p == 1 else side, ks > 1, halved)
            for p, (tn, tm, ks, halved) in enumerate(L.orthogonalize_plan(R, C, dt))}


def test_dense_shapes_reach_every_path():
    """Each (product, pieces, tile, side, split, halved) that 6000 shapes of up
    to 12 million elements pick is picked by a shape of the GPU tests too."""
    rng = random.Random(5)
    reached = set()
    for dt, R, C in DENSE:
        reached |= _paths(R, C, L.dtype_code(dt))
    for _ in range(3000):
        a = int(129 * 2 ** rng.uniform(0, 4.2))
        b = int(a * 2 ** rng.uniform(0, 4))
        if a * b <= 12e6:
            for R, C in ((a, b), (b, a)):
                for dt in (L.BF16, L.F32):
                    assert _paths(R, C, dt) <= reached, (R, C, dt, _paths(R, C, dt) - reached)


def test_thin_shapes_are_thin():
    for dt, R, C in THIN:
        assert L.orthogonalize_plan(R, C, L.dtype_code(dt)) == []


def test_plan_refusals():
    with pytest.raises(L.LycError):
        L.orthogonalize_plan(1 << 21, 4, L.BF16)
    with pytest.raises(L.LycError):
        L.orthogonalize_plan(200, 300, 0)
    assert L.lib().lyc_orthogonalize_plan(200, 300, 2, 3, None, None, None, None) == L.ERR_INVALID_ARG
    assert L.lib().lyc_orthogonalize_plan(200, 300, 2, 2, None, None, None, None) == L.OK
    assert torch.finfo(torch.bfloat16).eps / 2 == 2.0 ** -8
