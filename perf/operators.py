"""The 8-bit and update operators of the library, as a LoRA fine-tuning program
over a frozen 8-bit base weight calls them, with their plain forms.

  quantize   rows (1 x 128 groups) or tiles (128 x 128, a weight) to e4m3 with fp32 scales
  product    y = round( sum_b s_x s_w (q_x . q_w) + b )          both sides in hand as e4m3
  forward    the same with x quantized in the call, plus scale * round(x.down^T) . up^T
  backward   dx over W^T in e4m3 (dy quantized in the call), dDown, dUp
  orthogonalize   Newton-Schulz steps on a factor's (or a dense matrix's) update

Sizes are those of the library's LoRA workloads (tokens x features x features,
rank) or generic ones between a single token and those.
"""
import math

import torch

own = False

STEPS, COEF, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100   # a group's largest magnitude counts as at least this
LARGEST = 2.0 * 16384 * 8192 * 8192   # flops of the largest listed product


def listed():
    return [
        # the activations of the largest workload, quantized before its product
        {"name": "rows_bf16_16384x8192", "op": "quantize", "form": "rows", "R": 16384, "C": 8192, "dt": "bf16"},
        # a master weight quantized once per model, with the transposed codes the backward reads
        {"name": "tiles_f32_4096x4096", "op": "quantize", "form": "tiles", "R": 4096, "C": 4096, "dt": "f32"},
        # decoding: sixteen sequences, one token each, a large projection
        {"name": "product_16x8192x8192", "op": "product", "M": 16, "N": 8192, "K": 8192, "dt": "bf16", "bias": False},
        # a ragged prompt through a projection that fills no tile evenly
        {"name": "product_777x4104x4112", "op": "product", "M": 777, "N": 4104, "K": 4112, "dt": "f16", "bias": True},
        # one token through an adapted layer: latency
        {"name": "forward_1x4096x4096_r16", "op": "forward", "M": 1, "N": 4096, "K": 4096, "r": 16, "dt": "f16",
         "adt": "f16", "bias": False},
        # the training forward of the largest workload
        {"name": "forward_16384x8192x8192_r128", "op": "forward", "M": 16384, "N": 8192, "K": 8192, "r": 128,
         "dt": "bf16", "adt": "bf16", "bias": True},
        # a short ragged batch at an odd rank
        {"name": "backward_300x1040x2064_r5", "op": "backward", "M": 300, "N": 1040, "K": 2064, "r": 5, "dt": "f16",
         "adt": "f16"},
        # the training backward of the workload with fp32 master factors
        {"name": "backward_8192x4096x4096_r64", "op": "backward", "M": 8192, "N": 4096, "K": 4096, "r": 64,
         "dt": "bf16", "adt": "f32"},
        # the updates of LoRA factors: a small down, a large up, an fp32 master down
        {"name": "ortho_bf16_16x4096", "op": "ortho", "R": 16, "C": 4096, "dt": "bf16"},
        {"name": "ortho_bf16_8192x128", "op": "ortho", "R": 8192, "C": 128, "dt": "bf16"},
        {"name": "ortho_f32_64x4096", "op": "ortho", "R": 64, "C": 4096, "dt": "f32"},
        # the update of a dense projection that is trained whole
        {"name": "ortho_bf16_2048x4096", "op": "ortho", "R": 2048, "C": 4096, "dt": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of16(rng, lo, hi):
    return 16 * _log(rng, lo // 16, hi // 16)


def draw(rng):
    op = rng.choice(["quantize", "product", "forward", "backward", "ortho"])
    while True:
        if op == "quantize":
            form = rng.choice(["rows", "tiles"])
            c = {"op": op, "form": form, "R": _log(rng, 1, 16384) if form == "rows" else _of16(rng, 64, 8192),
                 "C": _of16(rng, 64, 8192), "dt": rng.choice(["f16", "bf16", "f32"])}
            return c
        if op == "ortho":
            c = {"op": op, "R": _log(rng, 2, 8192), "C": _log(rng, 16, 8192), "dt": rng.choice(["f16", "bf16", "f32"])}
            if rng.random() < 0.5:
                c["R"], c["C"] = c["C"], c["R"]
            if min(c["R"], c["C"]) <= 2048 and c["R"] * c["C"] <= 2048 * 4096:
                return c
            continue
        c = {"op": op, "M": _log(rng, 1, 16384), "N": _of16(rng, 256, 8192), "K": _of16(rng, 256, 8192),
             "dt": rng.choice(["f16", "bf16"])}
        if op != "product":
            c["r"] = _log(rng, 1, 256)
            c["adt"] = rng.choice([c["dt"], "f32"])
        if op != "backward":
            c["bias"] = rng.random() < 0.5
        if 2.0 * c["M"] * c["N"] * c["K"] <= LARGEST / 4:
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


def _e4m3_of(v, s):
    """Codes of v for given scales, for inputs only."""
    return (v / s).clamp(-448, 448).to(E4M3)


def _weight_codes(g, N, K):
    """A frozen weight as its codes, transposed codes and tile scales."""
    w = _randn(g, N, K, std=1.0 / math.sqrt(K))
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.zeros(nb * 128, kb * 128, device="cuda")
    p[:N, :K] = w
    s = p.view(nb, 128, kb, 128).abs().amax(dim=(1, 3)) / 448.0
    q = _e4m3_of(w, _spread(s, N, K))
    return q, q.t().contiguous(), s


def _rank_pad(r):
    return next(p for p in (16, 32, 64, 128, 256) if r <= p)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    dt = DT[case["dt"]]
    if op == "quantize":
        x = _activations(g, case["R"], case["C"]) if case["form"] == "rows" else \
            _randn(g, case["R"], case["C"], std=1.0 / math.sqrt(case["C"]))
        st["x"] = x.to(dt)
        return st
    if op == "ortho":
        R, C = case["R"], case["C"]
        n, m = min(R, C), max(R, C)
        # an update of uneven spectrum, as sums of correlated tokens give
        mix = _randn(g, n, n, std=1.0 / math.sqrt(n)) * torch.logspace(0, -1, n, device="cuda")
        u = (mix + 0.2 * torch.eye(n, device="cuda")) @ _randn(g, n, m, std=1e-3)
        st["g"] = (u if R <= C else u.t()).contiguous().to(dt)
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["wq"], st["wqt"], st["ws"] = _weight_codes(g, N, K)
    if case.get("bias"):
        st["bias"] = _randn(g, N, std=0.1).to(dt)
    x = _activations(g, M, K)
    if op == "product":
        kb = -(-K // 128)
        p = torch.zeros(M, kb * 128, device="cuda")
        p[:, :K] = x
        s = p.view(M, kb, 128).abs().amax(dim=2) / 448.0
        st["xq"] = _e4m3_of(x, s.repeat_interleave(128, dim=1)[:, :K])
        st["xs"] = s.t().contiguous()
        return st
    adt, r = DT[case["adt"]], case["r"]
    st["x"] = x.to(dt)
    st["down"] = _randn(g, r, K, std=1.0 / math.sqrt(K)).to(adt)
    st["up"] = _randn(g, N, r, std=0.05).to(adt)
    st["scale"] = 2.0
    if op == "backward":
        st["dy"] = (_activations(g, M, N) * 1e-2).to(dt)
        # what the forward kept: round(x.down^T), the rank padded as the library pads it
        h = _round16(st["x"].double() @ st["down"].to(dt).double().t(), dt)
        st["h"] = torch.zeros(M, _rank_pad(r), dtype=dt, device="cuda")
        st["h"][:, :r] = h
        del st["wq"]
    return st


# ---- the plain forms --------------------------------------------------------------

def _spread(s, R, C):
    """Tile scales [ceil(R/128), ceil(C/128)], one for each element."""
    return s.repeat_interleave(128, dim=0)[:R].repeat_interleave(128, dim=1)[:, :C]


def _round_e4m3(v):
    """v (64 bits, |v| < 464) to the nearest e4m3 value, ties to even."""
    e = (torch.frexp(v.abs())[1] - 1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _round16(v, dt):
    """v (64 bits) to the nearest value of a 16-bit type, ties to even, in one rounding."""
    bits, low = (11, -14) if dt == torch.float16 else (8, -126)
    e = (torch.frexp(v.abs())[1] - 1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(v), e - (bits - 1))
    return (torch.round(v / step) * step).to(dt)


def _padded(x, R, C):
    p = torch.zeros(R, C, dtype=x.dtype, device=x.device)
    p[:x.shape[0], :x.shape[1]] = x
    return p


def _scale(amax):
    """amax / 448 rounded once to 32 bits (the quotients x / s often lie on a border between codes)."""
    return (amax.clamp(min=FLOOR).double() / 448.0).float()


def _row_quantized(x):
    """(values of the codes [M, K] in fp32, scales [ceil(K/128), M])."""
    M, K = x.shape
    kb = -(-K // 128)
    amax = _padded(x.float(), M, kb * 128).view(M, kb, 128).abs().amax(dim=2)
    s = _scale(amax)
    # quotients in 64 bits: values next to a border between codes
    v = x.double() / s.double().repeat_interleave(128, dim=1)[:, :K]
    return _round_e4m3(v).float(), s.t().contiguous()


def _plain_quantize(st):
    x = st["x"]
    if st["case"]["form"] == "rows":
        v, s = _row_quantized(x)
        return {"q": v.to(E4M3), "s": s}
    R, C = x.shape
    nb, kb = -(-R // 128), -(-C // 128)
    p = _padded(x.float(), nb * 128, kb * 128).view(nb, 128, kb, 128)
    s = _scale(p.abs().amax(dim=(1, 3)))
    v = x.double() / _spread(s.double(), R, C)
    q = _round_e4m3(v).float().to(E4M3)
    return {"q": q, "s": s, "qt": q.t().contiguous()}


def _rows_value(q, s):
    return q.float() * s.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _plain_product(st):
    x = _rows_value(st["xq"], st["xs"])
    w = st["wq"].float() * _spread(st["ws"], *st["wq"].shape)
    y = x @ w.t()
    if "bias" in st:
        y = y + st["bias"].float()
    return y.to(DT[st["case"]["dt"]])


def _out_dtype(st):
    return torch.float32 if st["case"]["adt"] == "f32" else DT[st["case"]["dt"]]


def _plain_forward(st):
    c = DT[st["case"]["dt"]]
    x = st["x"]
    v, s = _row_quantized(x)
    w = st["wq"].float() * _spread(st["ws"], *st["wq"].shape)
    # in 64 bits: h is rounded to 16 bits before its second product
    h = _round16(x.double() @ st["down"].to(c).double().t(), c).float()
    y = _rows_value(v, s) @ w.t() + st["scale"] * (h @ st["up"].to(c).float().t())
    if "bias" in st:
        y = y + st["bias"].float()
    return y.to(_out_dtype(st))


def _plain_backward(st):
    c = DT[st["case"]["dt"]]
    x, dy, r = st["x"], st["dy"], st["case"]["r"]
    down, up = st["down"].to(c).float(), st["up"].to(c).float()
    v, s = _row_quantized(dy)
    w = st["wqt"].float().t() * _spread(st["ws"], dy.shape[1], x.shape[1])
    gh = _round16(st["scale"] * (dy.double() @ up.double()), c).float()
    dx = _rows_value(v, s) @ w + gh @ down
    dd = gh.t() @ x.float()
    du = st["scale"] * (dy.float().t() @ st["h"][:, :r].float())
    return {"dx": dx.to(c), "d_down": dd.to(st["down"].dtype), "d_up": du.to(st["up"].dtype)}


def _plain_ortho(st):
    g = st["g"].float()
    tall = g.shape[0] > g.shape[1]
    x = g.t() if tall else g
    x = x / (x.square().sum().sqrt() + EPS)
    a, b, c = COEF
    for _ in range(STEPS):
        t = x @ x.t()
        x = a * x + (b * t + c * (t @ t)) @ x
    return (x.t() if tall else x).contiguous().to(st["g"].dtype)


_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "forward": _plain_forward,
          "backward": _plain_backward, "ortho": _plain_ortho}


# ---- the library's calls ------------------------------------------------------------

def _own_run(st):
    import lora_bypass_linear_amd as lyc

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        if case["form"] == "rows":
            q, s = lyc.fp8_quantize_rows(st["x"])
            return {"q": q, "s": s}
        q, s, qt = lyc.fp8_quantize_weight(st["x"], transposed=True)
        return {"q": q, "s": s, "qt": qt}
    if op == "product":
        return lyc.fp8_linear(st["xq"], st["xs"], st["wq"], st["ws"], st.get("bias"), out_dtype=DT[case["dt"]])
    if op == "forward":
        return lyc.fp8_lora_linear(st["x"], st["wq"], st["ws"], st["down"], st["up"], st["scale"], st.get("bias"))
    if op == "backward":
        dx, dd, du = lyc.fp8_lora_linear_backward(st["x"], st["wqt"], st["ws"], st["down"], st["up"], st["scale"],
                                                  st["dy"], h=st["h"])
        return {"dx": dx, "d_down": dd, "d_up": du}
    return lyc.orthogonalize(st["g"], steps=STEPS, coefficients=COEF, eps=EPS)


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
        if case["form"] == "rows":
            return {"bytes": R * C * (es + 1) + 4 * R * -(-C // 128), "flops": 2 * R * C}
        return {"bytes": R * C * (es + 2) + 4 * -(-R // 128) * -(-C // 128), "flops": 2 * R * C}
    if op == "ortho":
        n, m = min(case["R"], case["C"]), max(case["R"], case["C"])
        # the Gram matrix once, four n x n products a step, one application
        thin = 4.0 * n * n * m + STEPS * 4 * 2.0 * n ** 3
        direct = STEPS * (4.0 * n * n * m + 2.0 * n ** 3)
        return {"bytes": 2 * n * m * es, "flops": min(thin, direct)}
    M, N, K = case["M"], case["N"], case["K"]
    wbytes = N * K + 4 * -(-N // 128) * -(-K // 128)
    if op == "product":
        return {"bytes": M * K + 4 * M * -(-K // 128) + wbytes + M * N * 2 + (2 * N if case["bias"] else 0),
                "flops": 2.0 * M * N * K}
    r, aes = case["r"], 4 if case["adt"] == "f32" else 2
    factors = (r * K + N * r) * aes
    if op == "forward":
        return {"bytes": M * K * 2 + wbytes + factors + M * N * aes + (2 * N if case["bias"] else 0),
                "flops": 2.0 * M * N * K + 2.0 * M * r * (K + N)}
    return {"bytes": M * K * 2 + M * N * 2 + M * r * 2 + wbytes + factors + M * K * 2 + factors,
            "flops": 2.0 * M * N * K + 4.0 * M * r * (K + N)}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _codes64(v):
    """Nearest e4m3 value of v through the ordered list of its values and their midpoints."""
    k = torch.arange(127, device=v.device)
    e, f = k // 8, (k % 8).double()
    val = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.pow(torch.tensor(2.0, dtype=torch.float64,
                                                                              device=v.device), (e - 10).double()))
    mid = (val[1:] + val[:-1]) / 2
    a = v.abs().contiguous()
    lo = torch.searchsorted(mid, a)               # midpoints below a
    hi = torch.searchsorted(mid, a, right=True)   # midpoints up to a
    code = torch.where(lo == hi, lo, lo + lo % 2)   # on a midpoint: the even one of lo, lo + 1
    return torch.copysign(val[code], v)


def _nearest16(v, dt):
    """v to the nearest of the 16-bit values around its torch conversion (which rounds through 32 bits)."""
    mid = v.to(dt).view(torch.int16)
    best = mid.view(dt).double()
    for d in (-1, 1):
        near = (mid + d).view(dt).double()
        off, was = (near - v).abs(), (best - v).abs()
        best = torch.where((off < was) | ((off == was) & (mid % 2 != 0)), near, best)
    return best


def _exact_rows(x):
    """(dequantized values, code values, scales [kb, M]) of rows in groups of 128."""
    M, K = x.shape
    full = x.double()
    vals, codes, scales = [], [], []
    for k0 in range(0, K, 128):
        part = full[:, k0:k0 + 128]
        top = part.abs().max(dim=1).values
        s = (torch.clamp(top, min=FLOOR) / 448.0).float().double()
        q = _codes64(part / s[:, None])
        codes.append(q)
        vals.append(q * s[:, None])
        scales.append(s)
    return torch.cat(vals, 1), torch.cat(codes, 1), torch.stack(scales)


def _exact_weight(q, s):
    w = q.float().double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] *= s[i, j].double()
    return w


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"]
        if case["form"] == "rows":
            _, q, s = _exact_rows(x)
            return {"q": q, "s": s}
        R, C = x.shape
        q = torch.empty(R, C, dtype=torch.float64, device="cuda")
        s = torch.empty(-(-R // 128), -(-C // 128), dtype=torch.float64, device="cuda")
        for i in range(s.shape[0]):
            band = x[i * 128:(i + 1) * 128].double()
            for j in range(s.shape[1]):
                t = band[:, j * 128:(j + 1) * 128]
                s[i, j] = (torch.clamp(t.abs().max(), min=FLOOR) / 448.0).float().double()
            per = s[i].repeat_interleave(128)[:C]
            q[i * 128:(i + 1) * 128] = _codes64(band / per)
        return {"q": q, "s": s, "qt": q.t().contiguous()}
    if op == "ortho":
        # through the singular values: each step maps s to a s + b s^3 + c s^5
        g = st["g"].double()
        u, sv, vt = torch.linalg.svd(g.cpu() if min(g.shape) > 512 else g, full_matrices=False) \
            if min(g.shape) <= 512 else (None, None, None)
        if u is None:
            x = g if g.shape[0] <= g.shape[1] else g.t()
            x = x / (torch.linalg.norm(x) + EPS)
            a, b, c = COEF
            for _ in range(STEPS):
                t = torch.mm(x, x.t())
                x = torch.addmm(torch.addmm(a * x, t, x, alpha=b), torch.mm(t, t), x, alpha=c)
            return (x if g.shape[0] <= g.shape[1] else x.t()).contiguous()
        sv = sv / (torch.sqrt((sv * sv).sum()) + EPS)
        for _ in range(STEPS):
            sv = COEF[0] * sv + COEF[1] * sv ** 3 + COEF[2] * sv ** 5
        return (u * sv) @ vt
    if op == "product":
        w = _exact_weight(st["wq"], st["ws"])
        x = st["xq"].float().double()
        for j in range(st["xs"].shape[0]):
            x[:, j * 128:(j + 1) * 128] *= st["xs"][j].double()[:, None]
        y = torch.mm(x, w.t())
        return y + st["bias"].double() if "bias" in st else y
    c = DT[case["dt"]]
    down, up = st["down"].to(c).double(), st["up"].to(c).double()
    if op == "forward":
        xv, _, _ = _exact_rows(st["x"])
        y = torch.mm(xv, _exact_weight(st["wq"], st["ws"]).t())
        h = _nearest16(torch.mm(st["x"].double(), down.t()), c)
        y = torch.addmm(y, h, up.t(), alpha=st["scale"])
        return y + st["bias"].double() if "bias" in st else y
    w = _exact_weight(st["wqt"].t().contiguous(), st["ws"])
    gv, _, _ = _exact_rows(st["dy"])
    gh = _nearest16(st["scale"] * torch.mm(st["dy"].double(), up), c)
    dx = torch.addmm(torch.mm(gv, w), gh, down)
    dd = torch.mm(gh.t(), st["x"].double())
    du = st["scale"] * torch.mm(st["dy"].double().t(), st["h"][:, :case["r"]].double())
    return {"dx": dx, "d_down": dd, "d_up": du}
