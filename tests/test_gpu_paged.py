"""Paged-cache calls on the GPU against the float64 oracle: page plan, cache
write, attention over all cached tokens and over chosen positions."""
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from oracle import paged_oracle as P
from paged import DEV, TYPES, Step, check, f64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# page plan
# ---------------------------------------------------------------------------
def _plan_case(B, longest, new, page, seed, room=5, spare=3):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, B)
    news = rng.integers(0, new + 1, B)
    held, want = -(-lens // page), -(-(lens + news) // page)
    n_pages = int(want.sum()) + 2 * spare + 1
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, int(want.max()) + 2), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return lens, news, table, ids[at:], spare, n_pages, int(news.sum()) + room


def _run_plan(lens, news, table, free, used, page, n_pages, max_tokens, **kw):
    t = i32(table)
    got = dsa.dsa_page_plan(i32(lens), i32(news), t, i32(free), i32([used]), page, n_pages, max_tokens, **kw)
    return [t.cpu().numpy()] + [x.cpu().numpy() for x in got]


def _same_plan(got, ref):
    table, q_off, slots, pos, lens, used = got
    assert np.array_equal(table, ref["table"]) and np.array_equal(q_off, ref["q_offsets"])
    assert np.array_equal(slots, ref["slots"]) and np.array_equal(pos, ref["positions"])
    assert np.array_equal(lens, ref["lens"]) and int(used[0]) == ref["used"]


@pytest.mark.parametrize("B,longest,new,page", [(1, 0, 1, 16), (1, 5, 0, 4), (8, 300, 3, 16), (33, 100, 1, 1),
                                                (257, 900, 5, 7), (1024, 64, 4, 64), (1025, 64, 40, 100),
                                                (3000, 20, 2, 8), (5, 4000, 3000, 128)])
def test_plan(B, longest, new, page):
    c = _plan_case(B, longest, new, page, B + page)
    lens, news, table, free, used, n_pages, mt = c
    _same_plan(_run_plan(lens, news, table, free, used, page, n_pages, mt, check=True),
               P.page_plan(lens, news, table, free, used, page, mt))


def test_plan_of_no_requests():
    q_off, slots, pos, lens, used = dsa.dsa_page_plan(i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32, device=DEV),
                                                      i32([1]), i32([1]), 16, 4, 3)
    assert q_off.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3
    assert lens.numel() == 0 and used.tolist() == [1]


@pytest.mark.parametrize("B,lens,new,used,mt,status", [(1, 3, 90, 0, 200, -1), (1, -1, 1, 0, 9, -1), (1, 1, -2, 0, 9, -1),
                                                       (2, 1, 5, 0, 9, -1), (1, 1, 1, 5, 9, -1), (1, 1, 1, -1, 9, -1),
                                                       (2, 1, 8, 1, 20, -8), (1500, 1, 8, 0, 20000, -8)])
def test_plan_that_fails_changes_nothing(B, lens, new, used, mt, status):
    lens, news = [lens] * B, [new] * B
    table, free = np.full((B, 3), 2, np.int32), [1, 2, 3, 4]
    ws = torch.zeros(1 << 14, dtype=torch.uint8, device=DEV)
    got = _run_plan(lens, news, table, free, used, 4, 5, mt, workspace=ws)
    ref = P.page_plan(lens, news, table, free, used, 4, mt)
    assert ref["status"] == status
    _same_plan(got, ref)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_status(ws)
    assert e.value.status == status
    # the workspace serves the next step
    _run_plan([1], [1], [[0, 0]], [1], 0, 4, 5, 2, workspace=ws, check=True)


def test_plan_reports_page_ids_outside_the_pool():
    ws = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    table, q_off, slots, *_ = _run_plan([2, 4], [3, 1], [[9, -1], [1, -1]], [7, 0], 0, 4, 5, 4, workspace=ws)
    assert slots.tolist() == [-1, -1, -1, 0] and q_off.tolist() == [0, 3, 4]
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_status(ws)
    assert e.value.status == -1


@pytest.mark.parametrize("B", [7, 1500])
def test_plan_in_place_steps(B):
    # lens and used updated in place, step after step, as a captured step does
    page, width, rng = 8, 12, np.random.default_rng(B)
    n_pages = B * width
    lens, used = i32([0] * B), i32([0])
    table, free = torch.full((B, width), -1, dtype=torch.int32, device=DEV), i32(rng.permutation(n_pages))
    hl, hu, ht = np.zeros(B, int), 0, table.cpu().numpy()
    mt = 6 * B
    out = (torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(mt, dtype=torch.int64, device=DEV),
           torch.empty(mt, dtype=torch.int32, device=DEV), lens, used)
    for _ in range(5):
        new = rng.integers(0, 7, B)
        got = dsa.dsa_page_plan(lens, i32(new), table, free, used, page, n_pages, mt, out=out, check=True)
        ref = P.page_plan(hl, new, ht, free.cpu().numpy(), hu, page, mt)
        _same_plan([table.cpu().numpy()] + [x.cpu().numpy() for x in got], ref)
        hl, hu, ht = ref["lens"], ref["used"], ref["table"]


# ---------------------------------------------------------------------------
# cache write
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("src,kv", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "e4m3"), ("fp32", "e4m3")])
@pytest.mark.parametrize("T,Hkv,d,page,joint", [(1, 1, 128, 16, False), (5, 8, 64, 7, True), (64, 2, 128, 1, False),
                                                (33, 3, 80, 16, True), (9, 5, 1, 4, False), (7, 1, 3, 4, True),
                                                (300, 4, 256, 64, False), (1000, 8, 96, 32, False)])
def test_append(src, kv, T, Hkv, d, page, joint):
    gen = torch.Generator().manual_seed(T + d)
    n_pages = -(-T // page) + 2
    k, v = (torch.randn((T, Hkv, d), generator=gen).to(TYPES[src]).to(DEV) for _ in range(2))
    k[T // 2] = 0  # a row of zeros: the smallest scale
    dt = torch.uint8 if kv == "e4m3" else TYPES[kv]
    both = torch.randint(1, 100, (n_pages, 2, page, Hkv, d), generator=gen).to(dt).to(DEV)
    K, V = (both[:, 0], both[:, 1]) if joint else (both[:, 0].contiguous(), both[:, 1].contiguous())
    sc = [torch.full((n_pages, page, Hkv), 3.0, device=DEV) for _ in range(2)] if kv == "e4m3" else [None, None]
    before = [f64(x) for x in (K, V)]
    slots = torch.randperm(n_pages * page, generator=gen)[:T]
    slots[T // 3] = -1 if T > 2 else slots[T // 3]
    dsa.dsa_page_append(k, K, slots.to(DEV), v=v, V_pages=V, K_scale=sc[0], V_scale=sc[1], check=True)
    rows, keep = slots.numpy(), slots.numpy() >= 0
    for x, pages, s, old in ((k, K, sc[0], before[0]), (v, V, sc[1], before[1])):
        x = f64(x)[keep]
        at = (rows[keep] // page, rows[keep] % page)
        if kv != "e4m3":
            old[at] = x
            assert np.array_equal(f64(pages), old)
            continue
        scale = P.e4m3_scale(x)
        got_s = s.cpu().double().numpy()
        assert np.all(np.abs(got_s[at] - scale) <= 2.0 ** -24 * scale)  # one fp32 rounding
        vals = pages.contiguous().view(torch.float8_e4m3fn).float().cpu().double().numpy()
        # the quotient: the scale's and the division's roundings (fp32), then e4m3's half step:
        # 2^-4 of the value, or half of the smallest e4m3 value (2^-9)
        exact = x / scale[..., None]
        assert np.all(np.abs(vals[at] - exact) <= np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10) + 2.0 ** -22 * np.abs(exact))
        mask = np.ones(got_s.shape[:2], bool)
        mask[at] = False
        assert np.all(got_s[mask] == 3.0)
        assert np.array_equal(pages.cpu().numpy()[mask].astype(np.float64), old[mask])


def test_append_keys_alone_feed_the_indexer():
    # the indexer's fp8 key cache: one head of 128, keys alone
    x = torch.randn((200, 1, 128), device=DEV, dtype=torch.bfloat16)
    K = torch.zeros((1, 256, 1, 128), dtype=torch.uint8, device=DEV)
    s = torch.ones((1, 256, 1), device=DEV)
    dsa.dsa_page_append(x, K, torch.arange(200, device=DEV), K_scale=s, check=True)
    got = K.view(torch.float8_e4m3fn).float()[0, :200, 0] * s[0, :200]
    assert torch.all((got - x[:, 0].float()).abs() <= 2.0 ** -4 * x[:, 0].float().abs() + s[0, :200] * 2.0 ** -9)
    q, w = torch.randn((2, 64, 128), device=DEV).bfloat16(), torch.rand((2, 64), device=DEV)
    idx, _ = dsa.dsa_index_decode(q, w, K[0, :200, 0], 16, torch.tensor([0, 200]), torch.tensor([0, 2]),
                                  K_scale=s[0, :200, 0].contiguous(), check=True)
    assert int(idx.min()) >= 0 and int(idx.max()) < 200


def test_append_skips_and_reports_slots_beyond_the_pool():
    k = torch.ones((3, 2, 64), device=DEV, dtype=torch.bfloat16)
    K = torch.zeros((4, 8, 2, 64), device=DEV, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    dsa.dsa_page_append(k, K, torch.tensor([0, 32, 1 << 40], device=DEV), workspace=ws)
    assert float(K.float().sum()) == 2 * 64
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_status(ws)
    assert e.value.status == -1
    dsa.dsa_page_append(k[:0], K, torch.empty(0, dtype=torch.int64, device=DEV), check=True)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _both(step, scale=None, what="", **kw):
    """Runs the step's form into sentinel-filled outputs, compares, and checks that padding stayed."""
    out = torch.full_like(step.Q, 7.0)
    lse = torch.full(step.Q.shape[:2], 7.0, device=DEV)
    kw = dict(scale=scale, out=out, lse=lse, check=True, **step.scale_args(), **kw)
    if step.idx is None:
        dsa.dsa_attend_paged(*step.args(), step.max_q, **kw)
    else:
        dsa.dsa_attend_selected(*step.args(), step.idx, **kw)
    check(step, out, lse, scale, what)
    n = sum(step.news)
    assert torch.all(out[n:] == 7) and torch.all(lse[n:] == 7), what
    return out, lse


HEADS = [(8, 8), (32, 8), (40, 8), (64, 1), (6, 2), (128, 1), (1, 1)]


@pytest.mark.parametrize("k", [None, 1, 70, 300])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64), ("fp32", 64), ("bf16", 80),
                                  ("fp32", 256), ("e4m3", 24)])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_attend_layouts(kv, d, Hq, Hkv, k):
    # ragged batch: none, one, a tile's edges, several tiles; a request without rows, one with more rows than tokens
    lens, news = [0, 1, 2, 127, 128, 129, 300, 513, 40, 64], [1, 1, 3, 1, 2, 4, 1, 2, 0, 4]
    _both(Step(lens, news, Hq, Hkv, d, kv, page=16, pad=3, k=k, seed=Hq + d))


@pytest.mark.parametrize("k", [None, 150])
@pytest.mark.parametrize("page,joint", [(1, False), (3, True), (8, False), (24, True), (64, True), (100, False),
                                        (128, False), (256, True), (1000, False)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp32"])
def test_attend_pages(kv, page, joint, k):
    _both(Step([257, 130, 999, 5], [2, 1, 1, 3], 16, 2, 128, kv, page=page, joint=joint and kv != "e4m3", k=k, seed=page))


@pytest.mark.parametrize("kv,d,Hq,Hkv,m", [("bf16", 128, 32, 8, 1), ("bf16", 128, 64, 1, 2), ("e4m3", 128, 64, 8, 1),
                                           ("bf16", 64, 8, 1, 4), ("fp32", 64, 4, 2, 1)])
def test_attend_long_split_and_joined(kv, d, Hq, Hkv, m):
    # one long cache over all multiprocessors, alone and beside short ones
    _both(Step([40000], [m], Hq, Hkv, d, kv, page=64, seed=1))
    _both(Step([1, 20011, 0, 333], [1, m, 1, 1], Hq, Hkv, d, kv, page=64, seed=2))
    _both(Step([40000], [m], Hq, Hkv, d, kv, page=64, seed=3, k=5000))


@pytest.mark.parametrize("m,Hq,Hkv", [(5, 32, 1), (9, 64, 2), (130, 4, 1), (17, 128, 1)])
def test_attend_many_rows(m, Hq, Hkv):
    # more query rows than one tile holds: several blocks of rows, each with its own causal end
    _both(Step([300, m, 700], [m, m, 3], Hq, Hkv, 128, page=32, seed=m))
    _both(Step([300, m, 700], [m, m, 3], Hq, Hkv, 128, page=32, seed=m, k=64))


def test_attend_many_requests():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 700, 1500)]
    _both(Step(lens, [int(x) for x in rng.integers(0, 3, 1500)], 4, 2, 64, page=32, seed=9))


@pytest.mark.parametrize("scale", [0.0, -0.7, 5.0])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp32"])
def test_attend_scale(scale, kv):
    _both(Step([300, 64], [1, 2], 8, 2, 64, kv, seed=3, spread=1.0), scale=scale)
    _both(Step([300, 64], [1, 2], 8, 2, 64, kv, seed=3, spread=1.0, k=90), scale=scale)


@pytest.mark.parametrize("kv", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [None, 1000])
def test_attend_rising_and_falling_scores(kv, k):
    # the running maximum grows at every tile, then never again; the last key outweighs all before it
    for sign in (1.0, -1.0):
        s = Step([1000], [1], 8, 1, 128, kv, page=16, seed=4, k=k)
        ramp = torch.linspace(0.1, 30.0, 1000) * sign
        u = torch.ones(128) / 128 ** 0.5
        s.Q.copy_((u * 12).expand_as(s.Q))
        for pos in range(1000):
            pg, off = int(s.table[0, pos // 16]), pos % 16
            s.K[pg, off, 0] = (u * ramp[pos]).to(s.K.dtype)
        _both(s, what=str(sign))


def test_selected_skips_and_repeats():
    s = Step([50, 60], [2, 2], 8, 2, 128, page=16, k=200, seed=6)
    idx = s.idx
    idx[0] = -1                                   # nothing chosen
    idx[1, :8] = torch.tensor([49, 49, 3, -5, 50, 1 << 30, -(1 << 31), 3], device=DEV, dtype=torch.int32)
    idx[1, 8:] = -1
    idx[2, :150] = 58                             # one key many times
    idx[3, :60] = torch.arange(60, device=DEV, dtype=torch.int32).flip(0)
    _both(s)
    # a list of every position gives what attention over all tokens gives
    full = torch.arange(60, device=DEV, dtype=torch.int32).expand(4, 60).contiguous()
    a = dsa.dsa_attend_selected(*s.args(), full, return_lse=True, check=True)
    b = dsa.dsa_attend_paged(*s.args(), 2, return_lse=True, check=True)
    assert torch.allclose(a[1], b[1], atol=1e-5, rtol=0) and torch.allclose(a[0].float(), b[0].float(), atol=0.03)


@pytest.mark.parametrize("k", [None, 64])
def test_attend_reports_bad_requests(k):
    def bad(change, **kw):
        s = Step([50, 60, 70], [1, 1, 1], 8, 2, 128, page=16, k=k, seed=8)
        ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
        change(s)
        if k is None:
            dsa.dsa_attend_paged(*s.args(), s.max_q, workspace=ws, **kw)
        else:
            dsa.dsa_attend_selected(*s.args(), s.idx, workspace=ws, **kw)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_check_status(ws)
        assert e.value.status == -1
        # the same workspace serves a good call
        s = Step([50, 60, 70], [1, 1, 1], 8, 2, 128, page=16, k=k, seed=8)
        _both(s, workspace=ws)
    bad(lambda s: s.lens_t.fill_(-3))
    bad(lambda s: s.lens_t.fill_(1 << 30))
    bad(lambda s: s.table.fill_(1 << 29))
    bad(lambda s: s.table.fill_(-1))
    bad(lambda s: s.q_off.copy_(torch.tensor([0, 5, 1, 3])))
    bad(lambda s: s.q_off.copy_(torch.tensor([-4, 1, 2, 3])))
    bad(lambda s: s.q_off.copy_(torch.tensor([0, 1, 2, 9])))


def test_attend_reports_more_rows_than_max_q():
    s = Step([50, 60], [1, 3], 8, 2, 128, page=16)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    dsa.dsa_attend_paged(*s.args(), 2, workspace=ws)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_check_status(ws)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("k", [None, 300])
def test_attend_repeats_bitwise(kv, k):
    s = Step([9000, 3, 500], [1, 1, 2], 32, 8, 128, kv, page=32, k=k, seed=11)
    a, la = _both(s)
    for _ in range(3):
        b, lb = _both(s)
        assert torch.equal(a, b) and torch.equal(la, lb)


# ---------------------------------------------------------------------------
# streams, graphs, and a run of all calls together
# ---------------------------------------------------------------------------
def test_other_stream_and_two_at_once():
    one, two = Step([5000], [1], 32, 8, 128, seed=1), Step([300, 4000], [2, 1], 32, 8, 128, seed=2, k=200)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((dsa.dsa_attend_paged(*one.args(), 1, return_lse=True, stream=s1),
                    dsa.dsa_attend_selected(*two.args(), two.idx, return_lse=True, stream=s2)))
    torch.cuda.synchronize()
    for a, b in got:
        check(one, *a)
        check(two, *b)


class Serve:
    """One decode step as a server keeps it: all buffers its own, nothing allocated."""

    def __init__(self, B, Hq, Hkv, d, kv, page, width, pad=0, seed=0):
        gen = torch.Generator().manual_seed(seed)
        n_pages = B * width
        dt = torch.uint8 if kv == "e4m3" else TYPES[kv]
        self.page, self.n_pages, self.B, self.rows = page, n_pages, B, 2 * B + pad
        self.K, self.V = (torch.zeros((n_pages, page, Hkv, d), dtype=dt, device=DEV) for _ in range(2))
        self.s = [torch.ones((n_pages, page, Hkv), device=DEV) for _ in range(2)] if kv == "e4m3" else [None, None]
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(n_pages, generator=gen).to(torch.int32).to(DEV)
        self.lens, self.used, self.new = i32([0] * B), i32([0]), i32([0] * B)
        e = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
        self.plan = (e(B + 1), e(self.rows, torch.int64), e(self.rows), self.lens, self.used)
        self.k, self.v = (torch.zeros((self.rows, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.q = torch.zeros((self.rows, Hq, d), dtype=torch.bfloat16, device=DEV)
        self.idx = torch.full((self.rows, 32), -1, dtype=torch.int32, device=DEV)
        self.out, self.sel = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.lse, self.sel_lse = (torch.zeros((self.rows, Hq), device=DEV) for _ in range(2))
        self.ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)

    def step(self):
        dsa.dsa_page_plan(self.lens, self.new, self.table, self.free, self.used, self.page, self.n_pages, self.rows,
                          out=self.plan, workspace=self.ws)
        dsa.dsa_page_append(self.k, self.K, self.plan[1], v=self.v, V_pages=self.V, K_scale=self.s[0], V_scale=self.s[1],
                            workspace=self.ws)
        kw = dict(K_scale=self.s[0], V_scale=self.s[1], workspace=self.ws)
        dsa.dsa_attend_paged(self.q, self.K, self.V, self.table, self.lens, self.plan[0], 2, out=self.out, lse=self.lse, **kw)
        dsa.dsa_attend_selected(self.q, self.K, self.V, self.table, self.lens, self.plan[0], self.idx, out=self.sel,
                                lse=self.sel_lse, **kw)


class View:
    """What check() reads of a step, from a server's buffers."""

    def __init__(self, s, idx):
        self.s, self.d, self.kv = s, s.q.shape[2], "bf16"
        self.idx = idx

    def oracle(self, scale):
        s = self.s
        K, V = ((x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x) for x in (s.K, s.V))
        return P.attend(f64(s.q), f64(K), f64(V), s.table.cpu().numpy(), s.lens.cpu().numpy(), s.plan[0].cpu().numpy(),
                        scale, f64(s.s[0]), f64(s.s[1]), self.idx)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_run_of_steps(kv, captured):
    # plan -> append -> attend over all tokens and over chosen ones, for some steps, eager or replayed
    B, rng = 5, np.random.default_rng(3)
    s = Serve(B, 16, 2, 128, kv, 16, 8, pad=4, seed=1)
    s.step()  # nothing new: also the warm-up before a capture
    g = None
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        torch.cuda.synchronize()
        assert s.lens.tolist() == [0] * B  # capturing runs nothing
    for _ in range(12):
        new = rng.integers(0, 3, B)
        s.new.copy_(torch.from_numpy(new))
        s.q.normal_()
        s.k.normal_()
        s.v.normal_()
        lens = s.lens.cpu().numpy() + new
        s.idx.fill_(-1)
        r = 0
        for b in range(B):
            for j in range(new[b]):
                pos = int(lens[b] - new[b] + j)
                pick = rng.permutation(pos + 1)[:32]
                s.idx[r, :len(pick)] = torch.from_numpy(pick.astype(np.int32))
                r += 1
        g.replay() if captured else s.step()
        dsa.dsa_check_status(s.ws)
        assert s.lens.tolist() == lens.tolist()
        check(View(s, None), s.out, s.lse)
        check(View(s, s.idx.cpu().numpy()), s.sel, s.sel_lse)


def test_two_graphs_share_a_workspace():
    a, b = Step([3000, 5], [1, 1], 32, 8, 128, seed=1), Step([70, 9000], [1, 2], 16, 2, 64, seed=2)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    runs = []
    for s in (a, b):
        out, lse = torch.zeros_like(s.Q), torch.zeros(s.Q.shape[:2], device=DEV)
        call = lambda s=s, out=out, lse=lse: dsa.dsa_attend_paged(*s.args(), s.max_q, out=out, lse=lse, workspace=ws)  # noqa: E731
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((s, g, out, lse))
    for _ in range(3):
        for s, g, out, lse in runs:
            out.zero_()
            g.replay()
        for s, _, out, lse in runs:
            check(s, out, lse)
    dsa.dsa_check_status(ws)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_indexer_then_selected_attention(kv):
    # decode: the indexer's answer over its own keys is the list that attention reads
    lens, news = [700, 64, 1500], [2, 1, 2]
    s = Step(lens, news, 64, 8, 128, kv, page=64, seed=5, k=8)
    q, w = torch.randn((5, 64, 128), device=DEV).bfloat16(), torch.rand((5, 64), device=DEV)
    keys = torch.randn((sum(lens), 128), device=DEV).bfloat16()
    ko = torch.tensor(np.concatenate([[0], np.cumsum(lens)]))
    s.idx, _ = dsa.dsa_index_decode(q, w, keys, 256, ko, s.q_off.cpu(), check=True)
    _both(s)
    # prefill: the dense indexer's rows, 256 positions each
    s = Step([512], [512], 16, 2, 128, kv, page=64, seed=6, k=8)
    q, w = torch.randn((512, 64, 128), device=DEV).bfloat16(), torch.rand((512, 64), device=DEV)
    s.idx, _ = dsa.dsa_index_dense(q, w, keys[:512], 256, q_pos0=0, check=True)
    _both(s)


# ---------------------------------------------------------------------------
# where the kernels change form
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,longest,new,page", [(2047, 40, 3, 16), (2048, 9, 1, 1), (2049, 40, 3, 16), (5000, 20, 2, 8)])
def test_plan_of_many_requests(B, longest, new, page):
    # one launch up to 2048 requests, two beyond; outputs apart from their inputs
    lens, news, table, free, used, n_pages, mt = _plan_case(B, longest, new, page, seed=B)
    got = _run_plan(lens, news, table, free, used, page, n_pages, mt)
    _same_plan(got, P.page_plan(lens, news, table, free, used, page, mt))


@pytest.mark.parametrize("src", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [128, 24, 7])  # 16, 8 and one element a lane
def test_append_e4m3_rounds_as_the_division_does(src, d):
    """The stored bytes are those of rn_e4m3(rn_fp32(x / scale)), at the borders between e4m3 values too: scales that
    are powers of two, have a fraction of all ones, lie near the smallest normal number or are large."""
    gen = torch.Generator().manual_seed(d)
    half = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (half[1:] + half[:-1]) / 2  # the borders
    scales = [1.0, 2.0 ** -20, 2.0 - 2.0 ** -23, (2.0 - 2.0 ** -23) * 2.0 ** -40, 1.17549435e-38, 2.0 ** -119, 3e35, 0.3]
    rows = []
    for s in scales:
        for _ in range(8):
            pick = mid[torch.randint(0, len(mid), (d,), generator=gen)]
            x = pick * s * (1 + torch.randint(-2, 3, (d,), generator=gen).double() * 2.0 ** -23)
            x *= torch.randint(0, 2, (d,), generator=gen).double() * 2 - 1
            x[0] = 448.0 * s
            rows.append(x)
    x = torch.stack(rows).to(TYPES[src])[:, None].to(DEV)
    T = x.shape[0]
    K = torch.zeros((T, 1, 1, d), dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.zeros((T, 1, 1), device=DEV)
    dsa.dsa_page_append(x, K, torch.arange(T, device=DEV), K_scale=sc, check=True)
    xf = x.cpu().float()[:, 0]
    want_s = (xf.abs().amax(-1) / np.float32(448)).clamp(min=2.0 ** -126)
    assert torch.equal(sc.cpu().view(-1), want_s)
    want = (xf / want_s[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(K.cpu().view(T, d).view(torch.uint8), want.view(torch.uint8))


def _baselines(step, per_head, per_query):
    """Gives every (query, head) row a baseline score of its own: keys share a direction that queries have more or less
    of.  ``per_head`` and ``per_query`` are the amounts."""
    d = step.d
    k0 = torch.zeros(d)
    k0[: d // 2] = 1.0
    K = step.K.float()
    K = torch.where(K.isnan(), K, K * 0.25 + k0.to(DEV)).to(step.K.dtype)
    step.K.copy_(K)
    rows, Hq = step.Q.shape[:2]
    amount = torch.tensor([[per_head[h % len(per_head)] + per_query[r % len(per_query)] for h in range(Hq)]
                           for r in range(rows)])
    step.Q.copy_((step.Q.float().cpu() * 0.5 + amount[..., None] * k0).to(step.Q.dtype))


@pytest.mark.parametrize("k", [None, 300])
@pytest.mark.parametrize("Hq,Hkv,m", [(2, 1, 8), (8, 1, 4), (64, 1, 1), (64, 1, 2), (32, 8, 1)])
def test_attend_rows_far_apart(Hq, Hkv, m, k):
    # rows that share a tile have baselines hundreds of powers of two apart, and the last tile of a cut cache holds
    # tokens that only the later queries see
    step = Step([128 * 2 + m - 3, 128 * 6 + 1, 700], [m, m, m], Hq, Hkv, 128, "bf16", page=16, pad=2, k=k, seed=m + Hq)
    _baselines(step, [0.0, 40.0, -40.0, 3.0], [0.0] * (m // 2) + [60.0] * (m - m // 2))
    _both(step)


@pytest.mark.parametrize("kv", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [None, 100])
def test_attend_pages_off_16_bytes(kv, k):
    step = Step([300, 129], [2, 1], 8, 2, 128, kv, page=16, k=k)
    for name in ("K", "V"):
        x = getattr(step, name)
        buf = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)
        buf[1:] = x.reshape(-1)
        setattr(step, name, buf[1:].view(x.shape))
    _both(step)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_cache_of_more_than_2_to_the_32_bytes(kv):
    # 2^20 + 64 pages of 16 tokens, 2 heads of 128: the last pages lie beyond 2^32 elements
    n_pages, page, Hkv, d, Hq = (1 << 20) + 64, 16, 2, 128, 8
    small = Step([500, 40], [1, 2], Hq, Hkv, d, kv, page=page, k=64)
    dt = TYPES[kv]
    big = [torch.empty((n_pages, page, Hkv, d), dtype=dt, device=DEV) for _ in range(2)]
    scales = [torch.empty((n_pages, page, Hkv), device=DEV) if kv == "e4m3" else None for _ in range(2)]
    have = small.K.shape[0]
    for x, b, s, bs in zip((small.K, small.V), big, small.scales, scales):
        b.view(torch.uint8)[-have:] = x.view(torch.uint8)
        if s is not None:
            bs[-have:] = s
    want = [dsa.dsa_attend_paged(*small.args(), small.max_q, **small.scale_args()),
            dsa.dsa_attend_selected(*small.args(), small.idx, **small.scale_args())]
    table = torch.where(small.table >= 0, small.table + (n_pages - have), small.table)
    args = (small.Q, big[0], big[1], table, small.lens_t, small.q_off)
    sc = {"K_scale": scales[0], "V_scale": scales[1]}
    assert torch.equal(dsa.dsa_attend_paged(*args, small.max_q, check=True, **sc), want[0])
    assert torch.equal(dsa.dsa_attend_selected(*args, small.idx, check=True, **sc), want[1])
    # and written there
    rows = torch.randn((3, Hkv, d), device=DEV).to(torch.bfloat16)
    slots = torch.tensor([n_pages * page - 1, 5, n_pages * page - 17], device=DEV)
    dsa.dsa_page_append(rows, big[0], slots, v=rows, V_pages=big[1], check=True, **sc)
    at = (slots // page, slots % page)
    got = big[0].view(torch.uint8)[at[0], at[1]].view(dt).float()
    if kv == "e4m3":
        got = got * scales[0][at[0], at[1]][..., None]
        assert torch.all((got - rows.float()).abs() <= 2.0 ** -4 * rows.float().abs() + scales[0][at[0], at[1]][..., None] * 2.0 ** -9)
    else:
        assert torch.equal(got, rows.float())


# ---------------------------------------------------------------------------
# the two ways into the library
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp32"])
def test_plain_calls_and_detailed_ones_agree(kv):
    # with a workspace and nothing else of the caller's the extension makes the call; with `out` _paged.py does
    ext = dsa._paged._ext()
    step = Step([300, 7, 129], [2, 1, 3], 8, 2, 64, kv, k=50)
    sc = step.scale_args()
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    for idx, f in ((None, lambda **kw: dsa.dsa_attend_paged(*step.args(), step.max_q, scale=0.1, workspace=ws, **sc, **kw)),
                   (step.idx, lambda **kw: dsa.dsa_attend_selected(*step.args(), step.idx, scale=0.1, workspace=ws, **sc, **kw))):
        assert ext.attend(*step.args(), idx, sc["K_scale"], sc["V_scale"], ws, step.max_q, 0.1, False) is not None
        o, l = f(return_lse=True)
        o2, l2 = f(out=torch.empty_like(step.Q), lse=torch.empty_like(l))
        assert torch.equal(o, o2) and torch.equal(l, l2) and torch.equal(f(), o)
    rows = torch.randn((5, 2, 64), device=DEV).to(step.Q.dtype)
    slots = torch.tensor([3, 1, -1, 40, 17], device=DEV)
    pages = [[x.clone() for x in (step.K, step.V)] + [None if s is None else s.clone() for s in step.scales] for _ in range(2)]
    for (K, V, ks, vs), kw in zip(pages, ({"workspace": ws}, {"check": True})):
        dsa.dsa_page_append(rows, K, slots, v=rows, V_pages=V, K_scale=ks, V_scale=vs, **kw)
    for x, y in zip(*pages):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    lens, news, table, free, used, n_pages, mt = _plan_case(9, 300, 5, 16, seed=2)
    _same_plan(_run_plan(lens, news, table, free, used, 16, n_pages, mt, workspace=ws),
               P.page_plan(lens, news, table, free, used, 16, mt))
    dsa.dsa_check_status(ws)


def test_the_extension_leaves_what_it_does_not_take():
    ext = dsa._paged._ext()
    step = Step([40, 9], [1, 2], 4, 2, 64, "bf16", k=8)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    good = [*step.args(), step.idx, None, None, ws, step.max_q, None, False]
    assert ext.attend(*good) is not None
    for i, bad in ((0, step.Q.half()), (0, step.Q[:, :, ::2]), (0, step.Q.cpu()), (1, step.K.float()), (1, step.K[:, :, :1]),
                   (2, step.V[:, :5]), (3, step.table.long()), (3, step.table.t()), (4, step.lens_t[:1]), (5, step.lens_t),
                   (6, step.idx.long()), (6, step.idx[:, ::2]), (7, torch.ones(3, device=DEV)), (9, ws[:16]), (9, None),
                   (10, 1.5), (11, "1")):
        assert ext.attend(*good[:i], bad, *good[i + 1:]) is None, i
    with pytest.raises(TypeError):
        dsa.dsa_attend_selected(step.Q.half(), *step.args()[1:], step.idx, workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        dsa.dsa_attend_selected(*step.args(), step.idx, workspace=ws[:16])
    with pytest.raises(dsa.DsaError):  # the library's own refusal
        dsa.dsa_attend_paged(*step.args(), 0, workspace=ws)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_page_plan(step.lens_t, step.lens_t, step.table, step.lens_t, step.lens_t[:1], 0, 4, 8, workspace=ws)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(6))
def test_attend_random_shapes(kv, seed):
    """Group sizes, head sizes, pages and lengths as they fall, short rows and padded batches among them."""
    rng = random.Random(seed * 2 + (kv == "e4m3"))
    for _ in range(12):
        Hkv, g = rng.choice([(1, 1), (2, 3), (1, 5), (3, 7), (8, 8), (1, 17), (2, 33), (1, 48), (1, 64), (1, 65), (1, 100)])
        d = rng.choice([8, 48, 64, 80, 112, 128]) if kv == "bf16" else rng.choice([16, 64, 80, 128])
        lens = [rng.randint(0, rng.choice([3, 130, 600])) for _ in range(rng.randint(1, 8))]
        news = [rng.randint(0, rng.choice([1, 2, 4])) for _ in lens]
        k = rng.choice([None, 1, 63, 129, 300])
        step = Step(lens, news, Hkv * g, Hkv, d, kv, page=rng.choice([1, 5, 16, 64, 300]), pad=rng.randint(1, 3),
                    joint=rng.random() < 0.3, k=k, seed=rng.randint(0, 1 << 30), spread=rng.choice([0.1, 1.5, 8.0]))
        _both(step, what=(Hkv, g, d, lens, news, k))


def test_first_calls_in_a_capture():
    # a process whose first attention calls are captured: nothing of theirs may need the host
    code = """
import torch
import sparse_attention_token_index_b200 as dsa
from tests.paged import Step, check
step = Step([300, 7, 129], [2, 1, 3], 8, 2, 64, "bf16", k=50)
ws = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
    a = dsa.dsa_attend_paged(*step.args(), step.max_q, return_lse=True, workspace=ws)
    b = dsa.dsa_attend_selected(*step.args(), step.idx, return_lse=True, workspace=ws)
g.replay()
torch.cuda.synchronize()
check(step, *b)
step.idx = None
check(step, *a)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
