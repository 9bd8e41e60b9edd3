"""Inputs and the bound that tell two-part weights of the paged attention from
weights rounded once."""
import numpy as np
import torch

from paged import Step


def cancelling(kv, Hq, Hkv, d, k):
    """Caches whose values are +-v0 in turn, read with nearly equal weights: outputs are small beside sum p |v|, so that
    their own rounding (2^-8 of the output) does not hide an error of the weights."""
    step = Step([17, 64, 200], [1, 1, 1], Hq, Hkv, d, kv, page=32, seed=Hq + d, k=k, spread=0.05)
    v0 = torch.ones(d, device=step.V.device) if kv == "e4m3" else 1.0 + torch.arange(d, device=step.V.device) / 256
    for b, n in enumerate(step.lens):
        pos = torch.arange(n, device=step.V.device)
        at = (step.table[b].long()[pos // 32], pos % 32)
        x = ((1 - 2 * (pos % 2)).float()[:, None, None] * v0).expand(n, Hkv, d).to(torch.bfloat16).to(step.V.dtype)
        if kv == "e4m3":
            step.V.view(torch.uint8)[at] = x.view(torch.uint8)
            step.scales[1][at] = 1.5
        else:
            step.V[at] = x
    return step


def two_parts_exceeded(step, out):
    """Where outputs are off by more than paged.check's bound with the weights' own error in two bf16 parts: each leaves
    2^-8 of what it rounds, 2^-16 of the weight in all."""
    ref, _, mag, top, count = step.oracle()
    dw = 2 * (step.d + 8) * 2.0 ** -23 * top + 2.0 ** -21 + count[:, None] * 2.0 ** -23 + 2.0 ** -16
    return ~(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + dw[..., None] * (1 + 2.0 ** -8) * mag)


TWO_PARTS = [("bf16", 8, 1, 128), ("bf16", 16, 1, 64), ("bf16", 32, 1, 128), ("bf16", 20, 1, 64), ("e4m3", 16, 1, 128),
             ("e4m3", 32, 1, 64), ("e4m3", 64, 1, 128), ("e4m3", 48, 1, 64), ("e4m3", 128, 1, 128), ("e4m3", 100, 1, 64),
             ("bf16", 8, 2, 136), ("e4m3", 8, 2, 24)]
