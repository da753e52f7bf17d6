"""Refusals of the 8-bit integer calls, before any GPU work (fake pointers), their
plans, and the paths that the GPU tests' sizes reach."""
import ctypes

import pytest
import torch

import lora_bypass_linear_amd as L
from tests.test_gpu_int8 import SHAPES

V = ctypes.c_void_p
P = lambda n: V(n << 32)
INV, UNS, WSP = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE


def _rows(x=P(1), dt=2, q=P(2), s=P(3), M=70, K=64):
    return L.lib().lyc_int8_quantize_rows(x, dt, q, s, M, K, None)


@pytest.mark.parametrize("kw,st", [
    (dict(x=None), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(dt=4), INV), (dict(M=-1), INV), (dict(K=-16), INV),
    (dict(K=72), UNS), (dict(K=131072), UNS), (dict(M=(1 << 30) + 1), UNS), (dict(x=V((1 << 32) + 8)), UNS),
    (dict(q=V((2 << 32) + 8)), UNS), (dict(s=V((3 << 32) + 2)), UNS), (dict(q=P(1)), INV), (dict(s=P(2)), INV)])
def test_rows_refusals(kw, st):
    assert _rows(**kw) == st


def _linear(q=P(1), s=P(2), w=P(3), ws=P(4), b=P(5), b_dt=2, y=P(6), y_dt=2, M=64, N=512, K=8192, wsp=P(7), nws=1 << 30):
    return L.lib().lyc_int8_linear_fwd(q, s, w, ws, b, b_dt, y, y_dt, M, N, K, wsp, nws, None)


def _gated(q=P(1), s=P(2), g=P(3), gs=P(4), v=P(5), vs=P(6), bg=P(7), bv=P(8), b_dt=2, act=0, y=P(9), y_dt=2, M=64, N=512,
           K=8192, wsp=P(10), nws=1 << 30):
    return L.lib().lyc_int8_gated_fwd(q, s, g, gs, v, vs, bg, bv, b_dt, act, y, y_dt, M, N, K, wsp, nws, None)


@pytest.mark.parametrize("kw,st", [
    (dict(q=None), INV), (dict(s=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(b=None), INV),
    (dict(b_dt=0), INV), (dict(b_dt=9), INV), (dict(y=None), INV), (dict(y_dt=4), INV), (dict(M=-1), INV), (dict(K=8200), UNS),
    (dict(K=131072), UNS), (dict(M=1 << 21, N=1 << 20), UNS), (dict(q=V((1 << 32) + 8)), UNS), (dict(w=V((3 << 32) + 8)), UNS),
    (dict(s=V((2 << 32) + 2)), UNS), (dict(ws=V((4 << 32) + 1)), UNS), (dict(y=V((6 << 32) + 1)), UNS),
    (dict(b=V((5 << 32) + 1)), UNS), (dict(wsp=None), WSP), (dict(nws=128), WSP), (dict(wsp=V((7 << 32) + 8)), WSP),
    (dict(y=P(1)), INV), (dict(y=P(3)), INV), (dict(y=P(4)), INV), (dict(wsp=P(6)), INV), (dict(wsp=P(3)), INV),
    (dict(y=P(5)), INV)])
def test_linear_refusals(kw, st):
    assert L.int8_linear_plan(64, 512, 8192)[2] > 1   # (the workspace is needed)
    assert _linear(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(q=None), INV), (dict(s=None), INV), (dict(g=None), INV), (dict(v=None), INV), (dict(gs=None), INV),
    (dict(vs=None), INV), (dict(bg=None), INV), (dict(bv=None), INV), (dict(act=3), INV), (dict(act=-1), INV),
    (dict(y=None), INV), (dict(y_dt=0), INV), (dict(K=8200), UNS), (dict(v=V((5 << 32) + 8)), UNS),
    (dict(vs=V((6 << 32) + 1)), UNS), (dict(bv=V((8 << 32) + 1)), UNS), (dict(wsp=None), WSP), (dict(nws=128), WSP),
    (dict(y=P(5)), INV), (dict(y=P(8)), INV), (dict(wsp=P(9)), INV), (dict(y=P(6)), INV)])
def test_gated_refusals(kw, st):
    assert L.int8_gated_plan(64, 512, 8192)[2] > 1
    assert _gated(**kw) == st


def test_empty():
    assert _rows(M=0) == L.OK
    assert _linear(M=0) == L.OK and _linear(N=0) == L.OK and _gated(M=0) == L.OK and _gated(N=0) == L.OK


def test_binding_checks():
    q, s, w, ws = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        L.int8_quantize_rows(torch.zeros(4, 32))
    with pytest.raises(ValueError, match="2-D"):
        L.int8_quantize_rows(torch.zeros(32))
    with pytest.raises(ValueError, match="GPU"):
        L.int8_linear(q, s, w, ws)
    for bad, what in (((q.float(), s, w, ws), "dtype"), ((q, s[:3], w, ws), "scales has shape"),
                      ((q, s, w[:, :16], ws), "w_q has shape"), ((q, s.half(), w, ws), "scales has dtype"),
                      ((q, s, w.to(torch.uint8), ws), "dtype")):
        with pytest.raises(ValueError, match=what):
            L.int8_linear(*bad)
    with pytest.raises(ValueError, match="bias has shape"):
        L.int8_linear(q, s, w, ws, torch.zeros(7))
    with pytest.raises(ValueError, match="activation"):
        L.int8_gated_linear(q, s, w, ws, w, ws, activation="tanh")
    with pytest.raises(ValueError, match="both or neither"):
        L.int8_gated_linear(q, s, w, ws, w, ws, torch.zeros(8))
    with pytest.raises(L.LycError):
        L.int8_linear_workspace_size(4, 4, 24)
    with pytest.raises(L.LycError):
        L.int8_gated_workspace_size(4, 4, 131072)


def test_shapes_reach_every_path():
    for plan in (L.int8_linear_plan, L.int8_gated_plan):
        seen = {(plan(*s)[1], plan(*s)[2] > 1) for s in SHAPES if s[0] and s[1]}
        assert {(16, False), (32, False), (64, False), (64, True), (128, False), (256, False)} <= seen, seen
    assert {L.int8_linear_plan(*s)[0] for s in SHAPES if 0 < s[0] <= 32 and s[2]} == {16, 32}


def test_sizes_that_one_launch_covers():
    assert L.int8_linear_workspace_size(1, (1 << 28) - 64, 16) == 0
    for size, plan in ((L.int8_linear_workspace_size, L.int8_linear_plan), (L.int8_gated_workspace_size, L.int8_gated_plan)):
        for f in (size, plan):
            with pytest.raises(L.LycError):
                f(1, 1 << 29, 16)
            with pytest.raises(L.LycError):
                f(1 << 30, 1 << 20, 16)
