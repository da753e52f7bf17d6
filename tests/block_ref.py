"""The gated feed-forward block and the int8 operators by their definitions in 64
bits (plain torch, on any device), and the error bounds of their tests.

A bound adds up, per element: every fp32 addition of a sum of n products at
2^-24 of the sum of their magnitudes (whatever the order), the activation's own
2^-20, the output's rounding at half a step, and one step for the smallest
subnormals."""
import math

import torch

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -126}   # (fp32 results below 2^-126 may be flushed)
ACT = 2.0 ** -20   # relative error of act, absolute of its slope in units of 1 + |g|


def nearest(v, dt):
    """v (64 bits) to dt in one rounding, ties to even, as 64 bits."""
    if dt == F32:
        return v.float().double()
    bits, low = (11, -14) if dt == F16 else (8, -126)
    e = (torch.frexp(v.abs())[1] - 1).clamp(min=low)
    step = ((e - (bits - 1) + 1023).to(torch.int64) << 52).view(torch.float64)   # 2^(e - bits + 1), exactly
    return torch.round(v / step) * step


def r_pad(r, c):
    return 0 if r == 0 else next(p for p in ((32, 64, 128, 256) if c == F32 else (16, 32, 64, 128, 256)) if r <= p)


def act(name, g):
    """(act(g), act'(g)) in 64 bits."""
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "silu":
        u, du = g, torch.ones_like(g)
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        u, du = c * (g + 0.044715 * g ** 3), c * (1.0 + 3.0 * 0.044715 * g * g)
    p, q = torch.sigmoid(u), torch.sigmoid(-u)
    return g * p, p + g * p * q * du


def act_error(name, g):
    """Bound of the library's error of act(g).  The tanh form's logistic argument u is an fp32 value of three
    roundings (under 2^-22 |u|), which its exponential turns into that relative error of p(u) (d ln p / du is 1 - p,
    at most 1): it counts where act is near 0, for negative u."""
    a = act(name, g)[0].abs()
    if name != "gelu_tanh":
        return ACT * a
    u = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    return a * (ACT + 2.0 ** -22 * u.clamp(-100.0, 0.0).abs())


def project(x, w, down, up, scale, bias, c):
    """(g, the bound of its fp32 error, h_r, the bound of h_r's): one projection, operands rounded to c."""
    xc, wc = x.to(c).double(), w.to(c).double()
    g, mass = xc @ wc.t(), xc.abs() @ wc.abs().t()
    h, eh, past = None, None, 0.0
    if down.shape[0]:
        uc = up.to(c).double()
        h, eh = low_rank(xc, down.to(c).double().t(), c)
        g, mass = g + scale * (h @ uc.t()), mass + abs(scale) * (h.abs() @ uc.abs().t())
        past = abs(scale) * (eh @ uc.abs().t())
    if bias is not None:
        g, mass = g + bias.double(), mass + bias.double().abs()
    return g, (x.shape[1] + down.shape[0] + 4) * 2.0 ** -24 * mass + past, h, eh


def low_rank(a, b, c):
    """(round_c(a b), the bound of the library's error): none in 16 bits, where the rounding is decided as the exact
    value decides it; in fp32 each of the sum's n products and n - 1 additions may be off by 2^-24 of the magnitudes
    added up so far, which n 2^-24 (|a| |b|) covers (the rounding of the product and of its addition are one fused
    step), and the result is rounded once."""
    h = a @ b
    if c != F32:
        return nearest(h, c), torch.zeros_like(h)
    return h, a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs()) + 2.0 ** -24 * h.abs()


def block_bound(name, g, eg, v, ev, y, out_dt):
    """Bound of |y - act(g) v| where g and v are off by up to eg and ev."""
    a, _ = act(name, g)
    ea = 1.13 * eg + act_error(name, g)   # |act'| <= 1.13 for every form
    return ea * (v.abs() + ev) + a.abs() * ev + (U[out_dt] + 2.0 ** -23) * y.abs() + TINY[out_dt]


def int8_rows(x):
    """(codes, scales) of rows."""
    s = (x.double().abs().amax(dim=1).clamp(min=2.0 ** -100) / 127.0).float()
    return torch.round(x.double() / s.double()[:, None]).to(torch.int8), s


def int8_project(q, s, wq, ws, bias):
    """(g, the bound of its fp32 error): three roundings (the sum, times s_w, the fused multiply-add)."""
    acc = q.double() @ wq.double().t()
    p = acc * torch.outer(s.double(), ws.double())
    g = p + bias.double() if bias is not None else p
    return g, 2.1 * 2.0 ** -24 * p.abs() + 1.1 * 2.0 ** -24 * g.abs()
