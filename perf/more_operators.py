"""The gated feed-forward block and the 8-bit integer operators of the library,
as a program that fine-tunes adapted layers and serves the merged ones calls
them, with their plain forms.

  quantize   rows to int8 codes with one fp32 scale each (tokens of x, output channels of a weight)
  product    y = round( s_x s_w (q_x . q_w) + b )                  both sides in hand as int8
  igated     y = round( act(g) * v ), g and v such products         the block over int8 weights
  gated      y = round( act(g) * v ), g and v LoRA-bypass projections of one x
  backward   dx and the four factors' gradients from dy and the kept g and v

Sizes are those of the library's LoRA workloads (tokens x features x features,
rank) or generic ones between a single token and those.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FLOOR = 2.0 ** -100   # a row's largest magnitude counts as at least this
LARGEST = 2.0 * 16384 * 8192 * 8192   # operations of the largest listed product


def listed():
    return [
        # the activations of the largest workload, quantized before its product
        {"name": "rows_bf16_16384x8192", "op": "quantize", "R": 16384, "C": 8192, "dt": "bf16"},
        # a merged fp32 weight quantized once per model
        {"name": "rows_f32_4096x4096", "op": "quantize", "R": 4096, "C": 4096, "dt": "f32"},
        # decoding: sixteen sequences, one token each, a large projection
        {"name": "product_16x8192x8192", "op": "product", "M": 16, "N": 8192, "K": 8192, "dt": "bf16", "bias": False},
        # a ragged prompt through a projection that fills no tile evenly
        {"name": "product_777x4104x4112", "op": "product", "M": 777, "N": 4104, "K": 4112, "dt": "f16", "bias": True},
        # the prompts of the largest workload
        {"name": "product_16384x8192x8192", "op": "product", "M": 16384, "N": 8192, "K": 8192, "dt": "bf16",
         "bias": True},
        # one token through the served block: latency
        {"name": "igated_1x8192x4096", "op": "igated", "M": 1, "N": 8192, "K": 4096, "dt": "bf16", "act": "silu",
         "bias": False},
        # a batch of prompts through the served block
        {"name": "igated_2048x8192x4096", "op": "igated", "M": 2048, "N": 8192, "K": 4096, "dt": "bf16",
         "act": "silu", "bias": False},
        # one token through the adapted block: latency
        {"name": "gated_1x8192x4096_r16", "op": "gated", "M": 1, "N": 8192, "K": 4096, "r": 16, "dt": "f16",
         "adt": "f16", "act": "silu", "bias": False, "keep": False},
        # a short ragged batch in fp32 at an odd rank, biased, the other activation
        {"name": "gated_517x2056x1032_r5_f32", "op": "gated", "M": 517, "N": 2056, "K": 1032, "r": 5, "dt": "f32",
         "adt": "f32", "act": "gelu_tanh", "bias": True, "keep": True},
        # the training forward, with what its backward reads
        {"name": "gated_8192x8192x4096_r64", "op": "gated", "M": 8192, "N": 8192, "K": 4096, "r": 64, "dt": "bf16",
         "adt": "bf16", "act": "silu", "bias": False, "keep": True},
        # a short ragged batch at an odd rank
        {"name": "backward_300x2064x1040_r5", "op": "backward", "M": 300, "N": 2064, "K": 1040, "r": 5, "dt": "f16",
         "adt": "f16", "act": "silu"},
        # the training backward with fp32 master factors
        {"name": "backward_8192x8192x4096_r64", "op": "backward", "M": 8192, "N": 8192, "K": 4096, "r": 64,
         "dt": "bf16", "adt": "f32", "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, m, lo, hi):
    return m * _log(rng, lo // m, hi // m)


def draw(rng):
    op = rng.choice(["quantize", "product", "igated", "gated", "backward"])
    while True:
        if op == "quantize":
            return {"op": op, "R": _log(rng, 1, 16384), "C": _mult(rng, 16, 64, 8192),
                    "dt": rng.choice(["f16", "bf16", "f32"])}
        M = _log(rng, 1, 16384)
        if op in ("product", "igated"):
            c = {"op": op, "M": M, "N": _log(rng, 256, 8192), "K": _mult(rng, 16, 256, 8192),
                 "dt": rng.choice(["f16", "bf16", "f32"]), "bias": rng.random() < 0.5}
            if op == "igated":
                c["act"] = rng.choice(["silu", "gelu_tanh", "gelu"])
            if 2.0 * c["M"] * c["N"] * c["K"] <= LARGEST / 8:
                return c
            continue
        dt = rng.choice(["f16", "bf16", "f32"])
        c = {"op": op, "M": M, "N": _mult(rng, 8, 256, 8192), "K": _mult(rng, 8, 256, 8192), "r": _log(rng, 1, 256),
             "dt": dt, "adt": rng.choice([dt, "f32"]), "act": rng.choice(["silu", "gelu_tanh", "gelu"])}
        if op == "gated":
            c["bias"] = rng.random() < 0.5
            c["keep"] = rng.random() < 0.5
        if 2.0 * c["M"] * c["N"] * c["K"] <= LARGEST / (64 if dt == "f32" else 8):
            return c


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, M, K):
    """Token rows of unlike sizes, and features of which a few stand out."""
    rows = torch.exp(0.5 * _randn(g, M, 1))
    cols = 1.0 + 8.0 * (torch.rand(1, K, generator=g, device="cuda") < 0.01)
    return _randn(g, M, K) * rows * cols


def _int8_of(v):
    """Codes and row scales, for inputs only."""
    s = v.abs().amax(dim=1) / 127.0
    return torch.round(v / s[:, None]).clamp(-127, 127).to(torch.int8), s


def _rank_pad(r, dt):
    return next(p for p in ((32, 64, 128, 256) if dt == torch.float32 else (16, 32, 64, 128, 256)) if r <= p)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    dt = DT[case["dt"]]
    if op == "quantize":
        st["x"] = _activations(g, case["R"], case["C"]).to(dt)
        return st
    M, N, K = case["M"], case["N"], case["K"]
    bdt = dt if op in ("product", "igated") else DT[case["adt"]]
    names = ("",) if op == "product" else ("_gate", "_value")
    if case.get("bias"):
        for n in names:
            st["bias" + n] = _randn(g, N, std=0.1).to(bdt)
    # (feature spread of the few large ones: the projections stay of order one)
    x = _activations(g, M, K)
    if op in ("product", "igated"):
        st["q"], st["s"] = _int8_of(x)
        for n in names:
            st["wq" + n], st["ws" + n] = _int8_of(_randn(g, N, K, std=1.0 / math.sqrt(K)))
        return st
    adt, r = DT[case["adt"]], case["r"]
    st["x"] = x.to(dt)
    st["scale"] = 2.0
    w = {}
    for n in names:
        w[n] = _randn(g, N, K, std=1.0 / math.sqrt(K)).to(dt)
        st["down" + n] = _randn(g, r, K, std=1.0 / math.sqrt(K)).to(adt)
        st["up" + n] = _randn(g, N, r, std=0.05).to(adt)
    if op == "gated":
        for n in names:
            st["w" + n] = w[n]
        return st
    st["dy"] = (_activations(g, M, N) * 1e-2).to(dt)
    # what the forward kept: g, v and round(x.down^T) of both, the rank padded as the library pads it
    rp = _rank_pad(r, dt)
    st["h"] = torch.zeros(M, 2 * rp, dtype=dt, device="cuda")
    for i, n in enumerate(names):
        h = (st["x"].float() @ st["down" + n].to(dt).float().t()).to(dt)
        st["h"][:, i * rp:i * rp + r] = h
        st[n[1:]] = (st["x"].float() @ w[n].float().t() +
                     st["scale"] * (h.float() @ st["up" + n].to(dt).float().t())).to(dt)
        # the frozen weight as its program keeps it for the backward
        st["w" + n] = w[n]
        st["wt" + n] = w[n].t().contiguous()
    return st


# ---- the plain forms --------------------------------------------------------------

def _round16(v, dt):
    """v (64 bits) to the nearest value of dt, ties to even, in one rounding."""
    if dt == torch.float32:
        return v.to(dt)
    bits, low, top = (11, -14, 65504.0) if dt == torch.float16 else (8, -126, 3.3895313892515355e38)
    e = (torch.frexp(v.abs())[1] - 1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(v), e - (bits - 1))
    return (torch.round(v / step) * step).clamp(-top, top).to(dt)


def _plain_act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-2.0 * z))


def _plain_slope(name, g):
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    if name == "gelu":
        return 0.5 * torch.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    p = 1.0 / (1.0 + torch.exp(-2.0 * c * (g + 0.044715 * g * g * g)))
    return p + g * p * (1.0 - p) * 2.0 * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_quantize(st):
    x = st["x"]
    # one rounding to 32 bits of the scale; quotients in 64: values next to a border between codes
    s = (x.float().abs().amax(dim=1).clamp(min=FLOOR).double() / 127.0).float()
    q = torch.round(x.double() / s.double()[:, None])
    return {"q": q.to(torch.int8), "s": s}


def _plain_projection(st, n):
    t = (st["q"].float() @ st["wq" + n].float().t()) * st["ws" + n] * st["s"][:, None]
    return t + st["bias" + n].float() if "bias" + n in st else t


def _plain_product(st):
    return _plain_projection(st, "").to(DT[st["case"]["dt"]])


def _plain_igated(st):
    g, v = _plain_projection(st, "_gate"), _plain_projection(st, "_value")
    return (_plain_act(st["case"]["act"], g) * v).to(DT[st["case"]["dt"]])


def _plain_gated(st):
    case = st["case"]
    c = DT[case["dt"]]
    x, r = st["x"], case["r"]
    rp = _rank_pad(r, c)
    hs = torch.zeros(x.shape[0], 2 * rp, dtype=c, device=x.device)
    p = []
    for i, n in enumerate(("_gate", "_value")):
        # in 64 bits: h is rounded before its second product
        h = _round16(x.double() @ st["down" + n].to(c).double().t(), c)
        hs[:, i * rp:i * rp + r] = h
        t = x.float() @ st["w" + n].float().t() + st["scale"] * (h.float() @ st["up" + n].to(c).float().t())
        p.append(t + st["bias" + n].float() if "bias" + n in st else t)
    y = (_plain_act(case["act"], p[0]) * p[1]).to(torch.float32 if case["adt"] == "f32" else c)
    if not case["keep"]:
        return {"y": y}
    return {"y": y, "gate": p[0].to(c), "value": p[1].to(c), "h": hs}


def _plain_backward(st):
    case = st["case"]
    c = DT[case["dt"]]
    x, r = st["x"], case["r"]
    rp = _rank_pad(r, c)
    # in 64 bits up to the rounding of what the products read
    g, v, dy = st["gate"].double(), st["value"].double(), st["dy"].double()
    d = {"_gate": _round16(dy * v * _plain_slope(case["act"], g), c),
         "_value": _round16(dy * _plain_act(case["act"], g), c)}
    out, dx = {}, 0.0
    for i, n in enumerate(("_gate", "_value")):
        down, up = st["down" + n].to(c).float(), st["up" + n].to(c).float()
        h = st["h"][:, i * rp:i * rp + r].float()
        gh = _round16(st["scale"] * (d[n].double() @ up.double()), c).float()
        dx = dx + d[n].float() @ st["w" + n].float() + gh @ down
        out["d_down" + n] = (gh.t() @ x.float()).to(st["down" + n].dtype)
        out["d_up" + n] = (st["scale"] * (d[n].float().t() @ h)).to(st["up" + n].dtype)
    return {"dx": dx.to(x.dtype), **out}


_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "igated": _plain_igated, "gated": _plain_gated,
          "backward": _plain_backward}


# ---- the library's calls ------------------------------------------------------------

def _own_run(st):
    import lora_bypass_linear_amd as lyc

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        q, s = lyc.int8_quantize_rows(st["x"])
        return {"q": q, "s": s}
    if op == "product":
        return lyc.int8_linear(st["q"], st["s"], st["wq"], st["ws"], st.get("bias"), out_dtype=DT[case["dt"]])
    if op == "igated":
        return lyc.int8_gated_linear(st["q"], st["s"], st["wq_gate"], st["ws_gate"], st["wq_value"], st["ws_value"],
                                     st.get("bias_gate"), st.get("bias_value"), activation=case["act"],
                                     out_dtype=DT[case["dt"]])
    factors = (st["down_gate"], st["up_gate"], st["down_value"], st["up_value"])
    if op == "gated":
        out = lyc.lora_gated_linear(st["x"], st["w_gate"], st["w_value"], *factors, st["scale"], st.get("bias_gate"),
                                    st.get("bias_value"), activation=case["act"], keep=case["keep"])
        return {"y": out[0], "gate": out[1], "value": out[2], "h": out[3]} if case["keep"] else {"y": out}
    dx, ddg, dug, ddv, duv = lyc.lora_gated_linear_backward(
        st["x"], st["w_gate"], st["w_value"], *factors, st["scale"], st["dy"], st["gate"], st["value"],
        activation=case["act"], w_gate_t=st["wt_gate"], w_value_t=st["wt_value"], h=st["h"])
    return {"dx": dx, "d_down_gate": ddg, "d_up_gate": dug, "d_down_value": ddv, "d_up_value": duv}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    op = case["op"]
    es = 4 if case["dt"] == "f32" else 2
    if op == "quantize":
        R, C = case["R"], case["C"]
        return {"bytes": R * C * (es + 1) + 4 * R, "flops": 2 * R * C}
    M, N, K = case["M"], case["N"], case["K"]
    if op in ("product", "igated"):
        p = 1 if op == "product" else 2
        return {"bytes": M * K + 4 * M + p * N * (K + 4 + (es if case["bias"] else 0)) + M * N * es,
                "flops": p * 2.0 * M * N * K}
    r, aes = case["r"], 4 if case["adt"] == "f32" else 2
    weights = 2 * N * K * es
    factors = 2 * (r * K + N * r) * aes
    rp = _rank_pad(r, DT[case["dt"]])
    if op == "gated":
        kept = (2 * M * N + 2 * M * rp) * es if case["keep"] else 0
        return {"bytes": M * K * es + weights + factors + M * N * aes + kept + (2 * N * aes if case["bias"] else 0),
                "flops": 4.0 * M * N * K + 4.0 * M * r * (K + N)}
    return {"bytes": (2 * M * K + 3 * M * N + 2 * M * rp) * es + weights + 2 * factors,
            "flops": 4.0 * M * N * K + 8.0 * M * r * (K + N)}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _nearest(v, dt):
    """v to the nearest of the values of a 16-bit type around its torch conversion (which rounds through 32 bits)."""
    if dt == torch.float32:
        return v.float().double()
    mid = v.to(dt).view(torch.int16)
    best = mid.view(dt).double()
    for d in (-1, 1):
        near = (mid + d).view(dt).double()
        off, was = (near - v).abs(), (best - v).abs()
        best = torch.where((off < was) | ((off == was) & (mid % 2 != 0)), near, best)
    return best


def _act64(name, g):
    """(act, its derivative) of g in 64 bits."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(g * -math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-g.square() / 2) * math.sqrt(0.5 / math.pi)
    a, b = math.sqrt(8.0 / math.pi), 0.044715 * math.sqrt(8.0 / math.pi)
    u = g * (a + b * g.square())          # act = g sigmoid(u)
    p = torch.sigmoid(u)
    return g * p, p + g * p * torch.sigmoid(-u) * (a + 3.0 * b * g.square())


def _scaled64(st, n):
    acc = torch.mm(st["q"].double(), st["wq" + n].double().t())   # whole numbers, exact
    v = acc * torch.outer(st["s"].double(), st["ws" + n].double())
    return v + st["bias" + n].double()[None, :] if "bias" + n in st else v


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        s = (torch.clamp(x.abs().max(dim=1).values, min=FLOOR) / 127.0).float().double()
        low = torch.floor(x / s[:, None])
        past = x - (low + 0.5) * s[:, None]              # (low + 0.5) s is exact in 64 bits
        up = (past > 0) | ((past == 0) & (low % 2 != 0))
        return {"q": (low + up).to(torch.int8), "s": s}
    if op == "product":
        return _scaled64(st, "")
    if op == "igated":
        return _act64(case["act"], _scaled64(st, "_gate"))[0] * _scaled64(st, "_value")
    c, r = DT[case["dt"]], case["r"]
    rp = _rank_pad(r, c)
    x = st["x"].double()
    if op == "gated":
        h = torch.zeros(x.shape[0], 2 * rp, dtype=torch.float64, device=x.device)
        p = []
        for i, n in enumerate(("_gate", "_value")):
            h[:, i * rp:i * rp + r] = _nearest(torch.mm(x, st["down" + n].to(c).double().t()), c)
            t = torch.addmm(torch.mm(x, st["w" + n].double().t()), h[:, i * rp:i * rp + r],
                            st["up" + n].to(c).double().t(), alpha=st["scale"])
            p.append(t + st["bias" + n].double() if case["bias"] else t)
        y = _act64(case["act"], p[0])[0] * p[1]
        return {"y": y, "gate": p[0], "value": p[1], "h": h} if case["keep"] else {"y": y}
    a, slope = _act64(case["act"], st["gate"].double())
    dy = st["dy"].double()
    grads = {"_gate": _nearest(dy * st["value"].double() * slope, c), "_value": _nearest(dy * a, c)}
    out = {"dx": torch.zeros_like(x)}
    for i, n in enumerate(("_gate", "_value")):
        d = grads[n]
        down, up = st["down" + n].to(c).double(), st["up" + n].to(c).double()
        gh = _nearest(st["scale"] * torch.mm(d, up), c)
        out["dx"].addmm_(d, st["w" + n].double()).addmm_(gh, down)
        out["d_down" + n] = torch.mm(gh.t(), x)
        out["d_up" + n] = st["scale"] * torch.mm(d.t(), st["h"][:, i * rp:i * rp + r].double())
    return out
