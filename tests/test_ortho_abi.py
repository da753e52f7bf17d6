"""Refusals of the orthogonalized update, before any GPU work (fake pointers)."""
import ctypes

import pytest
import torch

import lora_bypass_linear_amd as L

V = ctypes.c_void_p
INV, UNS, WSP = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE


def _call(g=V(1 << 20), dt=2, out=V(2 << 20), R=16, C=64, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7,
          ws=V(1 << 30), nws=1 << 40):
    return L.lib().lyc_orthogonalize(g, dt, out, R, C, steps, a, b, c, eps, ws, nws, None)


@pytest.mark.parametrize("kw,st", [
    (dict(g=None), INV), (dict(out=None), INV), (dict(dt=0), INV), (dict(R=-1), INV), (dict(steps=0), INV),
    (dict(steps=33), INV), (dict(a=float("nan")), INV), (dict(c=float("inf")), INV), (dict(eps=-1e-9), INV),
    (dict(R=(1 << 20) + 1), UNS), (dict(R=20000, C=20000), UNS), (dict(R=1 << 14, C=1 << 18), UNS), (dict(g=V(1)), UNS),
    (dict(dt=3, out=V((2 << 20) + 2)), UNS), (dict(out=V((1 << 20) + 2)), INV), (dict(ws=None), WSP),
    (dict(ws=V(64)), WSP), (dict(nws=100), WSP), (dict(ws=V(1 << 20)), INV), (dict(ws=V(2 << 20)), INV)])
def test_refusals(kw, st):
    assert _call(**kw) == st


def test_empty():
    assert _call(R=0) == L.OK and _call(C=0) == L.OK


def test_binding_checks():
    with pytest.raises(ValueError, match="GPU"):
        L.orthogonalize(torch.zeros(4, 16))
    with pytest.raises(ValueError, match="2-D"):
        L.orthogonalize(torch.zeros(16))
    with pytest.raises(ValueError, match="out has shape"):
        L.orthogonalize(torch.zeros(4, 16), out=torch.zeros(16, 4))
    with pytest.raises(ValueError, match="dtype"):
        L.orthogonalize(torch.zeros(4, 16), out=torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(L.LycError):
        L.orthogonalize_workspace_size(1 << 21, 4, 2)
