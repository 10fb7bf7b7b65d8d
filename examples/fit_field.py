#!/usr/bin/env python3
"""Fits a field of density and colour with the hash-grid encoder and a residual head, and renders it in 8 bits.

    python examples/fit_field.py [--steps 300] [--points 65536] [--width 256] [--blocks 2] [--state-bits 8]

The encoder, the head's linear layers and norms, and the AdamW step over the tables and the head's weights all run in
the library's kernels; PyTorch holds the loss.  The tables get 10 times the head's rate and no weight decay.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import multiresolution_hash_grid_amd as hg  # noqa: E402


def field(x: torch.Tensor) -> torch.Tensor:
    """Density of two soft balls and a colour that varies between them: [n, 4] of points in [0, 1)^3."""
    balls = [((0.35, 0.4, 0.5), 0.18), ((0.65, 0.6, 0.45), 0.14)]
    d = sum(torch.sigmoid((r - (x - torch.tensor(c, device=x.device)).norm(dim=1)) * 60) for c, r in balls)
    rgb = 0.5 + 0.5 * torch.sin(x * torch.tensor([9.0, 13.0, 7.0], device=x.device))
    return torch.cat([d[:, None], rgb * d[:, None].clamp_max(1)], 1)


def fit(steps=300, points=1 << 16, width=256, blocks=2, state_bits=8, seed=0, report=None):
    """(encoder, head, losses) after ``steps`` steps on uniform points."""
    torch.manual_seed(seed)
    enc = hg.HashGridEncoder(n_levels=16, n_features_per_level=2, log2_hashmap_size=17)
    head = hg.HashGridResidualHead(enc.cfg.out_features, width, blocks, 4)
    matrices = [p for p in head.parameters() if p.dim() == 2]
    vectors = [p for p in head.parameters() if p.dim() == 1]
    opt = hg.HashGridAdamW([dict(params=[enc.embeddings], lr=1e-2), dict(params=matrices, lr=1e-3, weight_decay=1e-2),
                            dict(params=vectors, lr=1e-3)], state_bits=state_bits, seed=seed)
    losses = []
    for step in range(steps):
        x = torch.rand(points, 3, device="cuda")
        loss = (head(enc(x)) - field(x)).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and step % report == 0:
            print(f"step {step}: loss {losses[-1].item():.3e}", flush=True)
    return enc, head, torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--points", type=int, default=1 << 16)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    enc, head, losses = fit(a.steps, a.points, a.width, a.blocks, a.state_bits, report=50)
    print(f"loss {losses[0].item():.3e} -> {losses[-10:].mean().item():.3e}")
    with torch.no_grad():
        x = torch.rand(1 << 18, 3, device="cuda")
        features = enc(x)
        y, y8, want = head(features), head.quantized()(features), field(x)
    psnr = lambda a, b: float(-10 * torch.log10((a - b).square().mean()))  # noqa: E731
    print(f"held-out points: {psnr(y, want):.1f} dB in 16 bits, {psnr(y8, want):.1f} dB in 8 bits")


if __name__ == "__main__":
    main()
