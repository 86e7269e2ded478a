"""A layer of experts from training to serving in 4 or 8 bits, on one MI355X:

    python examples/expert_ffn.py [--steps 20] [--form mx4|fp8]

Trains a small ExpertFFN to imitate a dense feed-forward layer on random tokens (--form fp8: with products in 8 bits), then holds its
experts in microscaled 4-bit or in 8-bit form and serves a prompt and single tokens with it (--form fp8: those in one call each)."""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_gemm_amd import ExpertFFN  # noqa: E402


def main(steps: int, form: str = "mx4") -> dict:
    torch.manual_seed(0)
    dev = torch.device("cuda", 0)
    dim, hidden, tokens = 256, 512, 2048
    teacher = nn.Sequential(nn.Linear(dim, hidden), nn.GELU(), nn.Linear(hidden, dim)).to(dev)
    layer = ExpertFFN(dim, hidden, num_experts=8, k=2, device=dev, fp8=form == "fp8", decode_tokens=16 if form == "fp8" else 0)
    opt = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, dim, device=dev)
        with torch.no_grad():
            want = teacher(x)
        loss = nn.functional.mse_loss(layer(x).float(), want)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step}: loss {losses[-1]:.5f}", flush=True)

    prompt = torch.randn(tokens, dim, device=dev)
    with torch.no_grad():
        before = layer(prompt).float(), layer(prompt[:1]).float()
        layer.quantize_(form)
        after = layer(prompt).float(), layer(prompt[:1]).float()
    rel = [float((a - b).norm() / b.norm()) for a, b in zip(after, before)]
    print(f"{layer.form} experts: prompt differs by {rel[0]:.3f}, one token by {rel[1]:.3f}", flush=True)
    return {"losses": losses, "prompt": rel[0], "token": rel[1]}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--form", choices=("mx4", "fp8"), default="mx4")
    args = ap.parse_args()
    main(args.steps, args.form)
