"""Refusals of the 8-bit calls, before any GPU work (fake pointers that nothing
dereferences), and the shape checks of their Python binding."""
import ctypes

import pytest
import torch

import lora_bypass_linear_amd as L

V = ctypes.c_void_p
P, P2, P3, P4 = V(1 << 20), V(2 << 20), V(3 << 20), V(4 << 20)
W = V(1 << 30)
BIG = 1 << 40
NULL = None


def _rows(x=P, dt=2, q=P2, s=P3, M=4, K=16):
    return L.lib().lyc_fp8_quantize_rows(x, dt, q, s, M, K, NULL)


def _weight(w=P, dt=2, q=P2, qt=NULL, s=P3, N=16, K=16):
    return L.lib().lyc_fp8_quantize_weight(w, dt, q, qt, s, N, K, NULL)


def _product(qx=P, sx=P2, qw=P3, sw=P4, b=NULL, b_dt=0, y=V(5 << 20), y_dt=2, M=4, N=16, K=16, ws=W, nws=BIG):
    return L.lib().lyc_fp8_linear_fwd(qx, sx, qw, sw, b, b_dt, y, y_dt, M, N, K, ws, nws, NULL)


def _fwd(x=P, x_dt=2, qw=P2, sw=P3, b=NULL, b_dt=0, d=P4, d_dt=2, u=V(5 << 20), u_dt=2, r=4, scale=1.0,
         y=V(6 << 20), y_dt=2, M=4, N=16, K=16, ws=W, nws=BIG):
    return L.lib().lyc_fp8_lora_linear_fwd(x, x_dt, qw, sw, b, b_dt, d, d_dt, u, u_dt, r, scale, y, y_dt, M, N, K, ws,
                                           nws, NULL)


def _bwd(x=P, x_dt=2, qwt=P2, sw=P3, b_dt=0, d=P4, d_dt=2, u=V(5 << 20), u_dt=2, h=NULL, r=4, scale=1.0,
         dy=V(6 << 20), g_dt=2, dx=V(7 << 20), dd=V(8 << 20), du=V(9 << 20), M=4, N=16, K=16, ws=W, nws=BIG):
    return L.lib().lyc_fp8_lora_linear_bwd(x, x_dt, qwt, sw, b_dt, d, d_dt, u, u_dt, h, r, scale, dy, g_dt, dx, dd,
                                           du, M, N, K, ws, nws, NULL)


INV, UNS, WSP = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE


@pytest.mark.parametrize("kw,st", [
    (dict(x=NULL), INV), (dict(q=NULL), INV), (dict(s=NULL), INV), (dict(dt=0), INV), (dict(M=-1), INV),
    (dict(K=24), UNS), (dict(K=(1 << 20) + 16), UNS), (dict(M=(1 << 28) + 1), UNS), (dict(x=V(8)), UNS),
    (dict(q=V(8)), UNS), (dict(s=V(2)), UNS), (dict(q=P), INV), (dict(s=P), INV), (dict(s=P2), INV)])
def test_rows_refusals(kw, st):
    assert _rows(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(w=NULL), INV), (dict(q=NULL), INV), (dict(s=NULL), INV), (dict(dt=9), INV), (dict(N=-1), INV),
    (dict(K=8), UNS), (dict(qt=P4, N=24), UNS), (dict(N=1 << 30, K=1 << 10), UNS), (dict(w=V(4)), UNS),
    (dict(q=P), INV), (dict(qt=P2), INV), (dict(qt=P), INV), (dict(qt=P3), INV)])
def test_weight_refusals(kw, st):
    assert _weight(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(qx=NULL), INV), (dict(sx=NULL), INV), (dict(qw=NULL), INV), (dict(sw=NULL), INV), (dict(y=NULL), INV),
    (dict(b=P, b_dt=0), INV), (dict(b_dt=2), INV), (dict(y_dt=4), INV), (dict(K=40), UNS), (dict(M=-3), INV),
    (dict(qx=V(8)), UNS), (dict(qw=V(24)), UNS), (dict(sx=V(2)), UNS), (dict(y=V(1)), UNS), (dict(y=P), INV),
    (dict(y=P3), INV), (dict(y=P2), INV), (dict(M=64, N=64, K=8192, ws=NULL), WSP),
    (dict(M=64, N=64, K=8192, ws=V(64)), WSP), (dict(M=64, N=64, K=8192, nws=16), WSP)])
def test_product_refusals(kw, st):
    assert _product(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(x=NULL), INV), (dict(qw=NULL), INV), (dict(sw=NULL), INV), (dict(d=NULL), INV), (dict(u=NULL), INV),
    (dict(y=NULL), INV), (dict(x_dt=1), L.ERR_MIXED_HALF), (dict(y_dt=3), L.ERR_DTYPE_MISMATCH), (dict(K=24), UNS),
    (dict(r=257), UNS), (dict(sw=V(2)), UNS), (dict(x=V(8)), UNS), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(ws=NULL), WSP), (dict(nws=8), WSP), (dict(b_dt=2), INV)])
def test_forward_refusals(kw, st):
    assert _fwd(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(x=NULL), INV), (dict(qwt=NULL), INV), (dict(sw=NULL), INV), (dict(d=NULL), INV), (dict(dy=NULL), INV),
    (dict(g_dt=1), L.ERR_MIXED_HALF), (dict(K=24), UNS), (dict(N=24), UNS), (dict(qwt=V(8)), UNS), (dict(sw=V(2)), UNS),
    (dict(dy=V(8)), UNS), (dict(h=V(8)), UNS), (dict(dx=P2), INV), (dict(dx=P3), INV), (dict(dd=V(7 << 20)), INV),
    (dict(ws=NULL), WSP), (dict(scale=float("nan")), INV)])
def test_backward_refusals(kw, st):
    assert _bwd(**kw) == st


def test_empty_calls_launch_nothing():
    assert _rows(M=0) == L.OK and _rows(K=0) == L.OK and _weight(N=0) == L.OK
    assert _product(M=0) == L.OK and _product(N=0) == L.OK and _fwd(M=0) == L.OK


def test_sizes():
    assert L.fp8_linear_workspace_size(0, 16, 16) == 0
    a = L.fp8_lora_workspace_size(64, 256, 512, 8, 2, 0, 2, 2)
    assert a >= 64 * 512 + 4 * 64 * 4
    for want in range(1, 8):
        assert L.fp8_lora_bwd_workspace_size(64, 256, 512, 8, 2, 0, 2, 2, 2, want) > 0
    with pytest.raises(L.LycError):
        L.fp8_lora_workspace_size(64, 256, 520, 8, 2, 0, 2, 2)
    with pytest.raises(L.MixedHalfError):
        L.fp8_lora_workspace_size(64, 256, 512, 8, 2, 0, 1, 2)


def test_binding_checks():
    z = torch.zeros
    e = lambda *s: z(*s, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="GPU"):
        L.fp8_quantize_rows(z(4, 16))
    with pytest.raises(ValueError, match="2-D"):
        L.fp8_quantize_weight(z(16))
    with pytest.raises(ValueError, match="w_q has dtype"):
        L.fp8_linear(e(4, 16), z(1, 4), z(16, 16), z(1, 1))
    with pytest.raises(ValueError, match="scales has shape"):
        L.fp8_linear(e(4, 16), z(4, 1), e(16, 16), z(1, 1))
    with pytest.raises(ValueError, match="scales has dtype"):
        L.fp8_linear(e(4, 16), z(1, 4), e(16, 16), z(1, 1, dtype=torch.float64))
    with pytest.raises(ValueError, match="down has shape"):
        L.fp8_lora_linear(z(4, 32), e(16, 32), z(1, 1), z(2, 16), z(16, 2), 1.0)
    with pytest.raises(ValueError, match="w_qt has shape"):
        L.fp8_lora_linear_backward(z(4, 32), e(16, 32), z(1, 1), z(2, 32), z(16, 2), 1.0, z(4, 16))
