"""The gated block and the 8-bit integer operators as a program uses them: a
training step of an adapted block, its merge, and the merged block served in
8-bit integers; on other streams, in captured graphs, over workspaces in any
state."""
import math

import pytest
import torch

import lora_bypass_linear_amd as L
from tests import block_ref as R
from tests.gpu_cases import say
from tests.test_gpu_gated import _args, _inputs, _rand

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _serve(q, s, block, down, act, **kw):
    """The served block: int8 gate and value, activations quantized again, int8 down projection."""
    y = L.int8_gated_linear(q, s, *block, activation=act, out_dtype=BF16)
    yq, ys = L.int8_quantize_rows(y)
    return L.int8_linear(yq, ys, *down, out_dtype=F32, **kw), y, yq, ys


@pytest.mark.parametrize("M", [1, 37, 300])
def test_train_merge_serve(M):
    """Each stage against its definition on what the stage before it gave; and the served block against the
    unquantized one, within what the roundings of the codes allow."""
    say("train, merge, serve", M)
    N, K, r, act, scale = 528, 272, 12, "silu", 2.0
    t = _inputs(M, N, K, r, BF16, BF16, BF16)
    y, gate, value, h = L.lora_gated_linear(*_args(t), scale, activation=act, keep=True)
    dy = (_rand(3, M, N) * 1e-2).to(BF16)
    dx, ddg, dug, ddv, duv = L.lora_gated_linear_backward(*_args(t), scale, dy, gate, value, activation=act, h=h)
    for k, g in (("down_gate", ddg), ("up_gate", dug), ("down_value", ddv), ("up_value", duv)):
        t[k] = (t[k].float() - 0.1 * L.orthogonalize(g).float()).to(BF16)
    merged = {n: L.lora_merge(t["w_" + n], t["down_" + n], t["up_" + n], scale) for n in ("gate", "value")}
    w_down = (_rand(50, K, N) / math.sqrt(N)).to(BF16)
    block = L.int8_quantize_rows(merged["gate"]) + L.int8_quantize_rows(merged["value"])
    down = L.int8_quantize_rows(w_down)
    q, s = L.int8_quantize_rows(t["x"])
    out, y8, yq, ys = _serve(q, s, block, down, act)

    g, eg = R.int8_project(q, s, block[0], block[1], None)
    v, ev = R.int8_project(q, s, block[2], block[3], None)
    ref = R.act(act, g)[0] * v
    assert ((y8.double() - ref).abs() <= R.block_bound(act, g, eg, v, ev, ref, BF16)).all()
    qr, sr = R.int8_rows(y8)
    assert torch.equal(yq, qr) and torch.equal(ys, sr)
    o, eo = R.int8_project(yq, ys, *down, None)
    assert ((out.double() - o).abs() <= eo + R.U[F32] * o.abs()).all()

    # what every code stands for is within half a step of the value: |a b - a' b'| <= |a - a'| |b| + |a'| |b - b'|
    def off(a, aq, as_):
        d = aq.double() * as_.double()[:, None]
        assert ((a.double() - d).abs() <= 0.5001 * as_.double()[:, None]).all()
        return (a.double() - d).abs(), d.abs()

    ex, xd = off(t["x"], q, s)
    eg_w, _ = off(merged["gate"], *block[:2])
    ev_w, _ = off(merged["value"], *block[2:])
    full_g, full_v = (t["x"].double() @ merged[n].double().t() for n in ("gate", "value"))
    dg = ex @ merged["gate"].double().abs().t() + xd @ eg_w.t() + eg
    dv = ex @ merged["value"].double().abs().t() + xd @ ev_w.t() + ev
    full = R.act(act, full_g)[0] * full_v
    d_y = 1.13 * dg * (full_v.abs() + dv) + R.act(act, full_g)[0].abs() * dv + 2 * (R.U[BF16] + R.ACT) * (full.abs() + 1.0)
    d_y = d_y + 2 * (R.U[BF16] + R.ACT) * (1.13 * dg * dv)
    assert ((y8.double() - full).abs() <= d_y).all()


def _ops(M=70, N=136, K=72, r=8):
    """(name, call) of each operator on fixed operands, with a workspace of its own where it takes one."""
    t = _inputs(M, N, K, r, BF16, BF16, BF16)
    q, s = L.int8_quantize_rows(_rand(1, M, 4096))
    a, b = L.int8_quantize_rows(_rand(2, N, 4096)), L.int8_quantize_rows(_rand(4, N, 4096))
    _, gate, value, h = L.lora_gated_linear(*_args(t), 1.0, keep=True)
    dy = _rand(5, M, N).to(BF16)
    big = lambda: torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return [
        ("rows", lambda ws: L.int8_quantize_rows(t["x"][:, :64].contiguous()), None),
        ("int8", lambda ws: (L.int8_linear(q, s, *a, out_dtype=F32, workspace=ws),), big()),
        ("int8 gated", lambda ws: (L.int8_gated_linear(q, s, *a, *b, workspace=ws),), big()),
        ("forward", lambda ws: L.lora_gated_linear(*_args(t), 1.0, keep=True, workspace=ws), big()),
        ("backward", lambda ws: L.lora_gated_linear_backward(*_args(t), 1.0, dy, gate, value, workspace=ws), big()),
        ("backward with h", lambda ws: L.lora_gated_linear_backward(*_args(t), 1.0, dy, gate, value, h=h, workspace=ws),
         big()),
    ], (t, q, s, gate, value, h, dy)


def test_workspace_contents_do_not_matter():
    assert L.int8_linear_plan(70, 136, 4096)[2] > 1 and L.int8_gated_plan(70, 136, 4096)[2] > 1
    ops, keep = _ops()
    for name, call, ws in ops:
        say("workspace", name)
        if ws is not None:
            ws.zero_()
        want = [v.clone() for v in call(ws)]
        for fill in (0xFF, 0x7F):
            if ws is not None:
                ws.fill_(fill)
            for v, w in zip(call(ws), want):
                assert torch.equal(v, w), name


def test_other_streams():
    """Each call on a stream of its own, all at once."""
    ops, keep = _ops()
    want = [[v.clone() for v in call(ws)] for _, call, ws in ops]
    torch.cuda.synchronize()
    say("streams")
    got, streams = [], [torch.cuda.Stream() for _ in ops]
    for _ in range(3):
        got = []
        for (name, call, ws), st in zip(ops, streams):
            with torch.cuda.stream(st):
                got.append(call(ws))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_captured_and_replayed():
    """A graph of all of them, replayed over new inputs with eager work between, against eager calls."""
    ops, (t, q, s, gate, value, h, dy) = _ops()
    for _, call, ws in ops:
        call(ws)
    torch.cuda.synchronize()
    say("capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call(ws) for _, call, ws in ops]
    for i in range(4):
        t["x"].copy_(_rand(100 + i, *t["x"].shape))
        dy.copy_(_rand(200 + i, *dy.shape))
        s.copy_(torch.rand_like(s) + 0.5)
        want = [[v.clone() for v in call(ws)] for _, call, ws in ops]
        torch.cuda.synchronize()
        say("replay", i)
        graph.replay()
        torch.cuda.synchronize()
        for (name, _, _), g, w in zip(ops, outs, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w)), (i, name)


def test_operands_in_place_of_strided_ones():
    """What is not contiguous is refused, not read as if it were."""
    ops, (t, q, s, gate, value, h, dy) = _ops()
    wide = torch.zeros(136, 144, dtype=BF16, device="cuda")[:, :72]
    with pytest.raises(ValueError, match="contiguous"):
        L.lora_gated_linear(t["x"], wide, t["w_value"], *_args(t)[3:], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        L.lora_gated_linear_backward(*_args(t), 1.0, dy.t().contiguous().t(), gate, value)
    with pytest.raises(ValueError, match="contiguous"):
        L.int8_quantize_rows(torch.zeros(64, 8, device="cuda").t())
    with pytest.raises(ValueError, match="contiguous"):
        L.int8_linear(q, s, torch.zeros(4096, 136, dtype=torch.int8, device="cuda").t(), torch.ones(136, device="cuda"))


def test_far_rows():
    """Outputs and operands past 2 and 4 GiB: the last rows of a long batch."""
    M, N, K = 2_200_000, 520, 16
    say("far rows", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(M, generator=g, device="cuda") + 0.5
    a = (torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8), torch.rand(N, device="cuda") * 1e-3)
    b = (torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8), torch.rand(N, device="cuda") * 1e-3)
    rows = torch.tensor([0, 255, 256, 1 << 20, 2_064_888, M - 257, M - 1], device="cuda")
    y = L.int8_linear(q, s, *a, out_dtype=F32)
    assert y.numel() * 4 > 1 << 32
    p, e = R.int8_project(q[rows], s[rows], *a, None)
    assert ((y[rows].double() - p).abs() <= e + R.U[F32] * p.abs()).all()
    del y
    y = L.int8_gated_linear(q, s, *a, *b)
    v, ev = R.int8_project(q[rows], s[rows], *b, None)
    ref = R.act("silu", p)[0] * v
    assert ((y[rows].double() - ref).abs() <= R.block_bound("silu", p, e, v, ev, ref, BF16)).all()


def test_backward_past_one_gibibyte():
    """Token-major operands of 1 GiB and more take the transposed copies: the same definition, the same bounds."""
    M, N, K, r, scale = 131080, 4104, 16, 3, 1.5
    say("backward past 1 GiB", M, N, K)
    assert M * N * 2 >= 1 << 30
    t = _inputs(M, N, K, r, BF16, BF16, BF16)
    _, gate, value, h = L.lora_gated_linear(*_args(t), scale, keep=True)
    dy = _rand(9, M, N).to(BF16)
    got = L.lora_gated_linear_backward(*_args(t), scale, dy, gate, value, h=h)
    rp = R.r_pad(r, BF16)
    for i, n in enumerate(("gate", "value")):
        a, slope = R.act("silu", gate.double())
        d = R.nearest(dy.double() * (value.double() * slope if i == 0 else a), BF16)
        del a, slope
        off = d.abs() * 2.0 ** -7   # (a step the other way, at most; far less in all)
        hp = h[:, i * rp:i * rp + r].double()
        ref = scale * (d.t() @ hp)
        du = got[2 + 2 * i].double()
        assert ((du - ref).abs() <= scale * (off.t() @ hp.abs()) + (R.U[BF16] + M * 2.0 ** -24) * scale * (d.abs().t() @ hp.abs())).all()
        assert torch.linalg.norm(du - ref) <= 1.5 * R.U[BF16] * torch.linalg.norm(ref)
        gh = R.nearest(scale * (d @ t["up_" + n].double()), BF16)
        ref = gh.t() @ t["x"].double()
        assert torch.linalg.norm(got[1 + 2 * i].double() - ref) <= 1.5 * R.U[BF16] * torch.linalg.norm(ref)
        part = d @ t["w_" + n].double() + gh @ t["down_" + n].double()
        dx = part if i == 0 else dx + part
    assert torch.linalg.norm(got[0].double() - dx) <= 1.5 * R.U[BF16] * torch.linalg.norm(dx)


def test_factor_gradients_of_the_longest_batch():
    """2^20 tokens at the largest rank: the kept h is then 1 GiB, its rows the farthest apart."""
    M, N, K, r, scale = 1 << 20, 16, 8, 255, 1.5
    say("longest batch", M, N, K, r)
    t = _inputs(M, N, K, r, BF16, BF16, BF16)
    _, gate, value, h = L.lora_gated_linear(*_args(t), scale, keep=True)
    assert h.numel() * 2 == 1 << 30
    dy = _rand(9, M, N).to(BF16)
    got = L.lora_gated_linear_backward(*_args(t), scale, dy, gate, value, h=h, want_dx=False)
    rp = R.r_pad(r, BF16)
    for i, n in enumerate(("gate", "value")):
        a, slope = R.act("silu", gate.double())
        d = R.nearest(dy.double() * (value.double() * slope if i == 0 else a), BF16)
        ref = scale * (d.t() @ h[:, i * rp:i * rp + r].double())
        assert torch.linalg.norm(got[2 + 2 * i].double() - ref) <= 1.5 * R.U[BF16] * torch.linalg.norm(ref)
        gh = R.nearest(scale * (d @ t["up_" + n].double()), BF16)
        ref = gh.t() @ t["x"].double()
        assert torch.linalg.norm(got[1 + 2 * i].double() - ref) <= 1.5 * R.U[BF16] * torch.linalg.norm(ref)
