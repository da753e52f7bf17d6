"""LoRA fine-tuning of one projection over a frozen 8-bit base weight.

    python examples/finetune_8bit.py [--steps 30] [--tokens 256] [--features 512] [--rank 16]

A teacher layer with weight W + dW (dW of low rank) gives the targets.  The
student keeps W as e4m3 codes and learns the two factors: each step is the
LoRA forward over the codes, the backward with the forward's h, and an update
of the factors by their orthogonalized momentum.  All of it runs in the
library's kernels except the loss and the two in-place updates.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import lora_bypass_linear_amd as lyc  # noqa: E402


def finetune(steps: int = 30, tokens: int = 256, features: int = 512, rank: int = 16, lr: float = 0.1, seed: int = 0):
    """The loss (mean squared error, relative to the targets') before each step and after the last."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    k = n = features
    w = rand(n, k) / k ** 0.5
    teacher = w + 0.5 * (rand(n, 4) @ rand(4, k)) / k ** 0.5 / 4 ** 0.5

    # once: the frozen weight as codes, scales and transposed codes
    w_q, w_s, w_qt = lyc.fp8_quantize_weight(w, transposed=True)
    down = (rand(rank, k) / k ** 0.5)          # fp32 master factors
    up = torch.zeros(n, rank, device="cuda")
    m_down, m_up = torch.zeros_like(down), torch.zeros_like(up)
    scale, momentum = 1.0, 0.9

    losses = []
    for step in range(steps + 1):
        x = rand(tokens, k).to(torch.bfloat16)
        target = x.float() @ teacher.t()
        y, ws = lyc.fp8_lora_linear(x, w_q, w_s, down, up, scale, return_workspace=True)
        diff = y.float() - target
        losses.append((diff.square().mean() / target.square().mean()).item())
        if step == steps:
            break
        dy = (2.0 / diff.numel() * diff * tokens).to(torch.bfloat16)
        h = lyc.fp8_lora_saved_h(ws, x, down, up)
        _, d_down, d_up = lyc.fp8_lora_linear_backward(x, w_qt, w_s, down, up, scale, dy, want_dx=False, h=h)
        for p, m, d in ((down, m_down, d_down), (up, m_up, d_up)):
            m.mul_(momentum).add_(d)
            # an orthogonal update has unit singular values: scale it to the
            # matrix's shape, and fade it out
            o = lyc.orthogonalize(m)
            p.add_(o, alpha=-lr * (1 - step / steps) * max(1.0, p.shape[0] / p.shape[1]) ** 0.5)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 30), ("tokens", 256), ("features", 512), ("rank", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    got = finetune(a.steps, a.tokens, a.features, a.rank)
    for i, v in enumerate(got):
        if i % 5 == 0 or i == len(got) - 1:
            print(f"step {i:3d}  loss {v:.4f}")
