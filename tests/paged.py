"""Builders and tolerances of the paged-cache GPU tests."""
import random

import numpy as np
import torch

from oracle import paged_oracle as P

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


class Step:
    """Caches of the given lengths in shuffled pages, and one step's queries.

    Slots that hold no token are NaN (bf16, fp32) or the e4m3 NaN byte with a
    NaN scale, so that whatever reads one shows it.  ``pad`` rows behind the
    last request stand for a padded batch."""

    def __init__(self, lens, news, Hq, Hkv, d, kv="bf16", page=16, pad=0, joint=False, k=None, seed=0, spread=1.5,
                 width=None):
        gen = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        self.lens, self.news, self.page, self.Hq, self.Hkv, self.d, self.kv = lens, news, page, Hq, Hkv, d, kv
        held = [-(-n // page) for n in lens]
        n_pages = sum(held) + 3
        ids = list(range(n_pages))
        rng.shuffle(ids)
        width = max(held + [1]) + 1 if width is None else width
        table = np.full((len(lens), width), -1, np.int32)
        at = 0
        dead = torch.ones((n_pages, page), dtype=torch.bool)
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
            for c in range(h):
                dead[table[b, c], :min(page, lens[b] - c * page)] = False
        shape = (n_pages, page, Hkv, d)
        self.scales = [None, None]
        pages = []
        for i in range(2):
            x = torch.randn(shape, generator=gen)
            if kv == "e4m3":
                x = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                x.view(torch.uint8)[dead] = 0x7f
                s = (torch.rand(shape[:3], generator=gen) + 0.5) / 100
                s[dead] = float("nan")
                self.scales[i] = s.to(DEV)
            else:
                x = x.to(TYPES[kv])
                x[dead] = float("nan")
            pages.append(x)
        if joint:
            both = torch.stack(pages, 1).to(DEV)
            self.K, self.V = both[:, 0], both[:, 1]
        else:
            self.K, self.V = pages[0].to(DEV), pages[1].to(DEV)
        rows = sum(news) + pad
        qt = torch.float32 if kv == "fp32" else torch.bfloat16
        self.Q = (torch.randn((rows, Hq, d), generator=gen) * spread).to(qt).to(DEV)
        self.table = torch.from_numpy(table).to(DEV)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.q_off = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
        self.idx = None
        if k is not None:  # lists as the indexer answers them, with extra entries that must be skipped
            idx = np.full((rows, k), -1, np.int32)
            r = 0
            for n, m in zip(lens, news):
                for j in range(m):
                    pos = n - m + j
                    if pos >= 0:
                        got = rng.sample(range(pos + 1), min(k, pos + 1))
                        idx[r, :len(got)] = got
                    r += 1
            idx[r:] = 0
            self.idx = torch.from_numpy(idx).to(DEV)
        self.max_q = max(news + [1])

    @property
    def shared(self):
        """Query rows that read the same tokens, at most."""
        return self.Hq // self.Hkv * (self.max_q if self.idx is None else 1)

    def args(self):
        return (self.Q, self.K, self.V, self.table, self.lens_t, self.q_off)

    def scale_args(self):
        return {"K_scale": self.scales[0], "V_scale": self.scales[1]}

    def oracle(self, scale=None):
        return P.attend(f64(self.Q), f64(self.K), f64(self.V), self.table.cpu().numpy(), self.lens,
                        self.q_off.cpu().numpy(), scale, f64(self.scales[0]), f64(self.scales[1]),
                        None if self.idx is None else self.idx.cpu().numpy())


def check(step, out, lse, scale=None, what=""):
    """Compares with the oracle.  A score is an fp32 sum of d products (and one
    or two more roundings: the scale), each step off by at most 2^-23 of the
    largest magnitude S = max |scale q| . |k| (accumulation may truncate), so
    a weight is off by the relative 2 (d + 8) 2^-23 S, plus 2^-21 for the
    exponential.  Sums over n tokens add n 2^-23.  The tensor-core kernel
    rounds each weight to bf16 (half a step: 2^-8), and bf16 outputs round
    once more.  All of it acts on sum p |v|; the log-sum-exp sees the scores'
    error and the sum's only.  Where 33 to 64 bf16 query rows share their
    tokens the output is N / D with N = sum p^ v, D = sum p^ of the rounded
    weights p^ = p (1 + e), |e| <= 2^-8: N / D - ref = (N - ref - ref (D - 1)) / D,
    so |N / D - ref| <= (2^-8 sum p |v| + 2^-8 |ref|) / (1 - 2^-8): the
    denominator's rounding adds 2^-8 |ref|, and 1 / D the factor 1 + 2^-7."""
    ref, rlse, mag, top, count = step.oracle(scale)
    live = ~np.isnan(rlse[:, 0])
    o, l = f64(out)[live], lse.double().cpu().numpy()[live]
    ref, rlse, mag, top, count = ref[live], rlse[live], mag[live], top[live], count[live][:, None]
    ds = (step.d + 8) * 2.0 ** -23 * top
    dw = 2 * ds + 2.0 ** -21 + count * 2.0 ** -23
    half = 2.0 ** -24 if step.kv == "fp32" else 2.0 ** -8
    weights = 0.0 if step.kv == "fp32" else 2.0 ** -8
    tol = half * np.abs(ref) + (dw[..., None] * (1 + half) + weights * (1 + half)) * mag
    if step.kv == "bf16" and 32 < getattr(step, "shared", 0) <= 64:
        tol = half * np.abs(ref) + (dw[..., None] * (1 + half) * mag + weights * (1 + half) * (mag + np.abs(ref))) * (1 + 2.0 ** -7)
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(o - ref)[bad])), np.argwhere(bad)[:4].tolist())
    none = count[:, 0] == 0
    assert np.all(o[none] == 0) and np.all(l[none] == -np.inf), what
    dl = ds + 2.0 ** -20 + count * 2.0 ** -23 + 2.0 ** -23 * np.abs(np.where(none[:, None], 0, rlse))
    off = np.abs(l[~none] - rlse[~none]) - dl[~none]
    assert not off.size or float(off.max()) <= 0, (what, "lse", float(off.max()))
