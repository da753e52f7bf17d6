"""The orthogonalized update for its tests: the iteration in 64 bits, and the
same iteration with every operand rounded to a given number of bits and its
products summed in fp32, which says how far a kernel that holds its operands in
so many bits is from the 64-bit result."""
import torch

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
COEF = (3.4445, -4.7750, 2.0315)
BITS = {F16: 22, BF16: 22, F32: 24}     # two fp16 pieces, three bf16 pieces
FEWER = {F16: 11, BF16: 11, F32: 16}    # one piece less


def update(seed, R, C, dt, low=-1.0, std=1e-3, device="cpu"):
    """An update of uneven spectrum, as sums of correlated tokens give."""
    g = torch.Generator().manual_seed(seed)
    n, m = min(R, C), max(R, C)
    mix = torch.randn(n, n, generator=g, dtype=F64) / n ** 0.5 * torch.logspace(0, low, n, dtype=F64)
    x = torch.randn(n, m, generator=g, dtype=F64).to(device)
    u = torch.mm((mix + 0.2 * torch.eye(n, dtype=F64)).to(device), x) * std
    return (u if R <= C else u.t()).contiguous().to(dt)


def start(g, eps):
    """X0 in 64 bits, the short side first."""
    x = g.to(F64)
    x = x if x.shape[0] <= x.shape[1] else x.t()
    norm = x.square().sum().sqrt() + eps
    return x / norm if norm != 0 else x


def exact(g, steps=5, coef=COEF, eps=1e-7):
    a, b, c = coef
    x = start(g, eps)
    for _ in range(steps):
        t = torch.mm(x, x.t().contiguous())
        x = a * x + torch.mm(b * t + c * torch.mm(t, t), x)
    return (x if g.shape[0] <= g.shape[1] else x.t()).contiguous()


def _rounded(v, bits):
    """v to `bits` significand bits (a 64-bit split: exact, ties aside)."""
    t = v * (2.0 ** (53 - bits) + 1)
    return t - (t - v)


def _sum32(u, v):
    # (sizes by powers of two inside fp32's range: the sums' relative errors stay)
    su, sv = (2.0 ** -torch.frexp(t.abs().max())[1].item() for t in (u, v))
    return torch.mm((u * su).to(F32), (v * sv).to(F32).contiguous()).to(F64) / su / sv


def emulate(g, bits, steps=5, coef=COEF, eps=1e-7):
    """The iteration with operands of `bits` bits, unrounded at its end: on X
    for a short side past 128, else in segments on the n x n side."""
    a, b, c = coef
    x = start(g, eps)
    n = x.shape[0]
    one = torch.eye(n, dtype=F64, device=g.device)
    r = lambda v: _rounded(v, bits)
    if n > 128:
        for _ in range(steps):
            x = r(x)
            t = r(_sum32(x, x.t()))
            x = _sum32(r(a * one + b * t + c * _sum32(t, t)), x)
    else:
        wide = n <= 16 and g.dtype != F32   # the n x n side in 64 bits
        seg = 5 if wide else 3 if g.dtype != F32 else 1
        segs = -(-steps // seg)
        done = 0
        for k in range(segs):
            count = -(-(steps - done) // (segs - k))
            done += count
            t = _sum32(r(x), r(x).t())
            mm, p = (torch.mm, lambda v: v) if wide else (_sum32, r)
            for i in range(count):
                t = p(t)
                f = a * one + b * t + c * mm(t, t)
                q = f if i == 0 else mm(p(q), p(f))
                t = mm(p(mm(t, p(f))), p(f))
            x = _sum32(r(q), r(x))
    return (x if g.shape[0] <= g.shape[1] else x.t()).contiguous()


def rounding(e, dt):
    """How far rounding the matrix e to dt is from it (2-norm): what it is for e
    itself, with 2 % for the elements that a small error rounds otherwise; half a
    step of each element where there are too few of them for that."""
    half = torch.finfo(dt).eps / 2 * float(e.norm()) + (2.0 ** -25 * e.numel() ** 0.5 if dt == F16 else 0.0)
    return min(half, 1.02 * float((e.to(dt).to(F64) - e).norm())) if e.numel() >= 1000 else half


def tolerance(g, e, bits=None, **kw):
    """Four times what the operands' bits alone give (the kernels' sums run in
    another order), and the result's rounding to its dtype."""
    own = float((emulate(g, bits or BITS[g.dtype], **kw) - e).norm())
    return 4 * own + 2.0 ** -22 * float(e.norm()) + rounding(e, g.dtype)
