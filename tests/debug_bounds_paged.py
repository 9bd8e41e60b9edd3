"""Calls run by test_gpu_debug_bounds_paged.py in a child process whose DSA_LIB
is the bounds-checking debug build: the four paged-cache calls on shapes that
reach the kernels' edges (empty and one-token requests, tiles cut at both ends,
several blocks of rows, padded batches, lists longer than their prefix, pages
of one token and larger than a tile, rows of any alignment, every element
type).  Every call is checked through the status word, where a failed bounds
check reads as an invalid internal state, and against the oracle."""
import os
import sys

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import sparse_attention_token_index_b200 as dsa  # noqa: E402
from oracle import paged_oracle as P  # noqa: E402
from paged import DEV, TYPES, Step, check  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def attend(step, what):
    kw = dict(return_lse=True, check=True, **step.scale_args())
    if step.idx is None:
        check(step, *dsa.dsa_attend_paged(*step.args(), step.max_q, **kw), what=what)
    else:
        check(step, *dsa.dsa_attend_selected(*step.args(), step.idx, **kw), what=what)


def plan(B, longest, new, page, in_place):
    rng = np.random.default_rng(B)
    lens, news = rng.integers(0, longest + 1, B), rng.integers(0, new + 1, B)
    held, want = -(-lens // page), -(-(lens + news) // page)
    n_pages, mt = int(want.sum()) + 1, int(news.sum()) + 3
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, max(1, int(want.max()))), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:]
    ref = P.page_plan(lens, news, table, free, 0, page, mt)
    t, ln, used = i32(table), i32(lens), i32([0])
    out = (torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(mt, dtype=torch.int64, device=DEV),
           torch.empty(mt, dtype=torch.int32, device=DEV), ln, used) if in_place else None
    got = dsa.dsa_page_plan(ln, i32(news), t, i32(free), used, page, n_pages, mt, out=out, check=True)
    for x, y in zip((t, *got), (ref["table"], ref["q_offsets"], ref["slots"], ref["positions"], ref["lens"], [ref["used"]])):
        assert np.array_equal(x.cpu().numpy(), np.asarray(y)), (B, page)


def append(src, kv, T, Hkv, d, page):
    x = torch.randn((T, Hkv, d), device=DEV).to(TYPES[src])
    n = -(-T // page)
    pages = [torch.zeros((n, page, Hkv, d), dtype=TYPES[kv], device=DEV) for _ in range(2)]
    sc = [torch.ones((n, page, Hkv), device=DEV) if kv == "e4m3" else None for _ in range(2)]
    slots = torch.arange(n * page, device=DEV).flip(0)[:T].contiguous()  # the pool's last slot among them
    dsa.dsa_page_append(x, pages[0], slots, v=x, V_pages=pages[1], K_scale=sc[0], V_scale=sc[1], check=True)
    got = pages[1].float().view(-1, Hkv, d)[slots]
    if kv == "e4m3":
        s = sc[1].view(-1, Hkv)[slots][..., None]
        assert torch.all((got * s - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + s * 2.0 ** -9)
    else:
        assert torch.equal(got, x.float())


def main():
    assert os.path.basename(dsa.lib_path) == "libdsa_index_debug.so", dsa.lib_path
    for B, longest, new, page in ((1, 0, 1, 1), (8, 300, 3, 16), (700, 90, 40, 7), (2500, 9, 2, 8)):
        for in_place in (False, True):
            plan(B, longest, new, page, in_place)
    for src, kv in (("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp32", "e4m3")):
        for T, Hkv, d, page in ((1, 1, 128, 16), (33, 3, 80, 16), (9, 5, 1, 4), (40, 2, 24, 1), (300, 4, 256, 64)):
            append(src, kv, T, Hkv, d, page)
    lens, news = [0, 1, 2, 127, 128, 129, 300, 513, 40], [1, 1, 3, 1, 2, 4, 1, 2, 0]
    for kv, d in (("bf16", 128), ("bf16", 64), ("bf16", 80), ("bf16", 136), ("e4m3", 128), ("e4m3", 64), ("e4m3", 24), ("fp32", 64)):
        for Hq, Hkv in ((32, 8), (6, 2), (20, 1), (64, 1), (128, 1)):
            for page, k in ((16, None), (1, 70), (300, 300)):
                attend(Step(lens, news, Hq, Hkv, d, kv, page=page, pad=2, k=k, seed=Hq + d), (kv, d, Hq, Hkv, page, k))
    for kv in ("bf16", "e4m3", "fp32"):
        attend(Step([9000, 1, 0, 333], [2, 1, 1, 1], 16, 2, 128, kv, page=64, seed=1), "long")
        attend(Step([9000, 333], [2, 1], 64, 1, 128, kv, page=64, seed=2, k=3000), "long lists")
        attend(Step([300, 130], [130, 17], 4, 1, 64, kv, page=32, seed=3), "many rows")
    print("debug-bounds cases ok")


if __name__ == "__main__":
    main()
