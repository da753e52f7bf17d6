"""Refusals of the gated block's calls, before any GPU work (fake pointers), its
plans, and the paths that the GPU tests' sizes reach."""
import ctypes

import pytest
import torch

import lora_bypass_linear_amd as L
from tests.test_gpu_gated import BACKWARD, FORWARD

V = ctypes.c_void_p
P = lambda n: V(n << 32)
INV, UNS, WSP, MIX, DTY = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE, L.ERR_MIXED_HALF, L.ERR_DTYPE_MISMATCH


def _fwd(x=P(1), x_dt=2, wg=P(2), wv=P(3), w_dt=2, bg=P(4), bv=P(5), b_dt=2, dg=P(6), dv=P(7), d_dt=2, ug=P(8), uv=P(9),
         u_dt=2, r=16, scale=1.0, act=0, y=P(10), y_dt=2, gate=P(11), value=P(12), h=P(13), M=70, N=72, K=64, ws=P(14),
         nws=1 << 30):
    return L.lib().lyc_lora_gated_fwd(x, x_dt, wg, wv, w_dt, bg, bv, b_dt, dg, dv, d_dt, ug, uv, u_dt, r, scale, act, y,
                                      y_dt, gate, value, h, M, N, K, ws, nws, None)


@pytest.mark.parametrize("kw,st", [
    (dict(x=None), INV), (dict(wg=None), INV), (dict(wv=None), INV), (dict(bg=None), INV), (dict(bv=None), INV),
    (dict(b_dt=0), INV), (dict(dg=None), INV), (dict(uv=None), INV), (dict(y=None), INV), (dict(gate=None), INV),
    (dict(value=None), INV), (dict(act=-1), INV), (dict(act=3), INV), (dict(x_dt=0), INV), (dict(y_dt=7), INV),
    (dict(M=-1), INV), (dict(r=-1), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(x_dt=1), MIX), (dict(u_dt=1), MIX), (dict(y_dt=3), DTY), (dict(d_dt=3), DTY),
    (dict(K=60), UNS), (dict(r=257), UNS), (dict(K=(1 << 20) + 8), UNS), (dict(M=1 << 21, N=1 << 20), UNS),
    (dict(x=V((1 << 32) + 8)), UNS), (dict(wv=V((3 << 32) + 8)), UNS), (dict(dg=V((6 << 32) + 1)), UNS),
    (dict(y=V((10 << 32) + 1)), UNS), (dict(gate=V((11 << 32) + 1)), UNS), (dict(h=V((13 << 32) + 8)), UNS),
    (dict(bv=V((5 << 32) + 1)), UNS), (dict(ws=None), WSP), (dict(ws=V((14 << 32) + 16)), WSP), (dict(nws=64), WSP),
    (dict(y=P(1)), INV), (dict(y=P(3)), INV), (dict(gate=P(10)), INV), (dict(value=P(11)), INV), (dict(h=P(12)), INV),
    (dict(h=P(7)), INV), (dict(ws=P(8)), INV), (dict(ws=P(10)), INV), (dict(y=P(5)), INV)])
def test_forward_refusals(kw, st):
    assert _fwd(**kw) == st


def test_forward_empty():
    assert _fwd(M=0) == L.OK and _fwd(N=0) == L.OK


def _bwd(x=P(1), x_dt=2, wg=None, wv=None, gt=P(2), vt=P(3), w_dt=2, b_dt=0, dg=P(4), dv=P(5), d_dt=2, ug=P(6), uv=P(7),
         u_dt=2, gate=P(8), value=P(9), h=P(10), r=16, scale=1.0, act=0, dy=P(11), dy_dt=2, dx=P(12), ddg=P(13), ddv=P(14),
         dug=P(15), duv=P(16), M=70, N=72, K=64, ws=P(17), nws=1 << 30):
    return L.lib().lyc_lora_gated_bwd(x, x_dt, wg, wv, gt, vt, w_dt, b_dt, dg, dv, d_dt, ug, uv, u_dt, gate, value, h, r,
                                      scale, act, dy, dy_dt, dx, ddg, ddv, dug, duv, M, N, K, ws, nws, None)


@pytest.mark.parametrize("kw,st", [
    (dict(x=None), INV), (dict(gt=None), INV), (dict(wg=P(2)), INV), (dict(gt=None, vt=None), INV), (dict(dg=None), INV),
    (dict(ug=None), INV), (dict(gate=None), INV), (dict(value=None), INV), (dict(dy=None), INV), (dict(ddg=None), INV),
    (dict(dug=None), INV), (dict(act=3), INV), (dict(scale=float("nan")), INV), (dict(dy_dt=0), INV),
    (dict(dy_dt=1), MIX), (dict(N=76), UNS), (dict(K=60), UNS), (dict(M=(1 << 20) + 1), UNS), (dict(r=300), UNS),
    (dict(x=V((1 << 32) + 8)), UNS), (dict(gt=V((2 << 32) + 8)), UNS), (dict(gate=V((8 << 32) + 8)), UNS),
    (dict(dy=V((11 << 32) + 8)), UNS), (dict(h=V((10 << 32) + 8)), UNS), (dict(dx=V((12 << 32) + 1)), UNS),
    (dict(ddv=V((14 << 32) + 1)), UNS), (dict(ws=None), WSP), (dict(nws=64), WSP), (dict(ws=V((17 << 32) + 8)), WSP),
    (dict(dx=P(1)), INV), (dict(dx=P(11)), INV), (dict(ddg=P(8)), INV), (dict(duv=P(15)), INV), (dict(ws=P(9)), INV),
    (dict(dug=P(10)), INV), (dict(ws=P(12)), INV)])
def test_backward_refusals(kw, st):
    assert _bwd(**kw) == st


def test_what_is_not_read_may_be_absent():
    """(the call then gets as far as the workspace check)"""
    assert _bwd(dx=None, gt=None, vt=None, nws=0) == WSP
    assert _bwd(dx=None, ddg=None, ddv=None, x=None, ug=None, uv=None, dg=None, dv=None, gt=None, vt=None, nws=0) == WSP
    assert _bwd(dug=None, duv=None, h=None, nws=0) == WSP


def test_sizes_are_checked_by_the_queries():
    for args in ((-1, 8, 8, 1), (8, 8, 12, 1), (8, 8, 8, 257)):
        with pytest.raises(L.LycError):
            L.lora_gated_workspace_size(*args, 2, 2, 0, 2, 2)
    with pytest.raises(L.LycError):
        L.lora_gated_bwd_workspace_size(8, 12, 8, 1, 2, 2, 0, 2, 2, 2)
    with pytest.raises(L.LycError):
        L.lora_gated_plan(8, 8, 12, 2)
    # a kept h, given back, needs none of the recomputation's room
    a = L.lora_gated_bwd_workspace_size(300, 264, 136, 16, 2, 2, 0, 2, 2, 2, 7)
    b = L.lora_gated_bwd_workspace_size(300, 264, 136, 16, 2, 2, 0, 2, 2, 2, 7 | L.BWD_H | L.BWD_WT)
    assert b < a


def test_binding_checks():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    ok = dict(x=z(4, 16), w_gate=z(8, 16), w_value=z(8, 16), down_gate=z(2, 16), up_gate=z(8, 2), down_value=z(2, 16),
              up_value=z(8, 2))

    def call(**kw):
        a = {**ok, **kw}
        act = a.pop("activation", "silu")
        extra = {k: a.pop(k) for k in ("bias_gate", "bias_value", "out") if k in a}
        return L.lora_gated_linear(*a.values(), 1.0, activation=act, **extra)

    for kw, what in ((dict(), "GPU"), (dict(activation="relu"), "activation"), (dict(w_value=z(8, 24)), "w_value has shape"),
                     (dict(up_value=z(8, 3)), "up_value has shape"), (dict(down_value=z(3, 16)), "down_value has shape"),
                     (dict(w_value=z(8, 16, dt=torch.float32)), "w_gate and w_value have dtypes"),
                     (dict(bias_gate=z(8)), "both or neither"), (dict(bias_gate=z(8), bias_value=z(7)), "bias_value has shape"),
                     (dict(out=z(4, 9)), "out has shape")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
    with pytest.raises(ValueError, match="both or neither"):
        L.lora_gated_linear_backward(*ok.values(), 1.0, z(4, 8), z(4, 8), z(4, 8), w_gate_t=z(16, 8))
    with pytest.raises(ValueError, match="gate has shape"):
        L.lora_gated_linear_backward(*ok.values(), 1.0, z(4, 8), z(4, 7), z(4, 8))


def test_cases_reach_every_path():
    """(tile features, tile rows, whether K is split, whether compute is fp32) of the GPU tests' sizes"""
    def seen(cases, backward):
        out = set()
        for M, N, K, r, *dts in cases:
            c, _ = L.resolve_dtypes([L._CODE[t] for t in dts if isinstance(t, torch.dtype)])
            tn, tm, ks = L.lora_gated_plan(M, N, K, c, backward)
            out.add((tn, tm, ks > 1, c == L.F32))
        return out
    f, b = seen(FORWARD, False), seen(BACKWARD, True)
    for w in (1, 2):   # features of a forward tile are half its weight rows
        every = {(64 // w, 64, False, False), (64 // w, 64, True, False), (128 // w, 128, False, False),
                 (256 // w, 256, False, False), (64 // w, 64, False, True), (64 // w, 64, True, True),
                 (96 // w, 128, False, True), (128 // w, 128, False, True), (16, 16, False, False), (16, 32, False, False),
                 (16, 16, False, True), (16, 32, False, True)}
        have = f if w == 2 else b
        assert every <= have, (w, every - have)
    assert {(32, 16, False, False), (32, 32, False, False)} <= b


def test_sizes_that_one_launch_covers():
    assert L.lora_gated_workspace_size(1 << 26, 8, 8, 4, 2, 2, 0, 2, 2) > 0
    assert L.lora_gated_workspace_size((1 << 26) + 1, 8, 8, 0, 2, 2, 0, 2, 2) == 0
    for args in (((1 << 26) + 1, 8, 8, 4), (1, 1 << 29, 8, 0), (1 << 30, 1 << 20, 8, 0)):
        with pytest.raises(L.LycError):
            L.lora_gated_workspace_size(*args, 2, 2, 0, 2, 2)
    with pytest.raises(L.LycError):
        L.lora_gated_plan(1, 1 << 29, 8, 2)


def test_calls_run_with_the_operands_device_current(monkeypatch):
    """A default stream (0) belongs to the current device, so another device's operands make theirs current."""
    import contextlib
    import inspect
    import torch
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d.index)
        yield
        entered.append("left")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(L, "_stream", lambda d: 70 + d.index)
    got = []
    fn = lambda *a: got.append((a, list(entered))) or 0
    L._launch(torch.device("cuda", 0), fn, 5)
    L._launch(torch.device("cuda", 1), fn, 6)
    assert got == [((5, 70), []), ((6, 71), [1])] and entered == [1, "left"]
    with pytest.raises(L.LycError):
        L._launch(torch.device("cuda", 0), lambda *a: 1)
    for f in (L.lora_gated_linear, L.lora_gated_linear_backward, L.int8_quantize_rows, L.int8_linear, L.int8_gated_linear):
        assert "_launch(dev" in inspect.getsource(f)
