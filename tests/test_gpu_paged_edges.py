"""Paged-cache calls on the GPU at their edges: references that move while
other outputs wait, weights in two parts, empty steps, rows of no request,
tensors that want a gradient, pages outside the pool, values that are not
finite, waits that run out."""
import numpy as np
import pytest
import torch

import sparse_attention_token_index_b200 as dsa
from paged import DEV, TYPES, Step, check, f64
from paged_weights import TWO_PARTS, cancelling, two_parts_exceeded

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(step, out=None, lse=None, **kw):
    kw = {"return_lse": True, "check": True, **step.scale_args(), **kw}
    if out is not None:
        kw.update(out=out, lse=lse)
    if step.idx is None:
        return dsa.dsa_attend_paged(*step.args(), step.max_q, **kw)
    return dsa.dsa_attend_selected(*step.args(), step.idx, **kw)


def loud_tokens(step, loud, jumps):
    """Raises the scores of the positions `loud` (a function of the position) by jumps[h % len] natural units in head h:
    keys and queries get a direction of their own on top of what they hold."""
    u = torch.zeros(step.d, device=DEV)
    u[:16] = 0.25  # |u| = 1
    K = step.K.float()
    K[..., :16] = torch.where(K[..., :16].isnan(), K[..., :16], 0.0)
    for b, n in enumerate(step.lens):
        pos = torch.tensor([p for p in range(n) if loud(p)], device=DEV, dtype=torch.int64)
        if len(pos):
            at = (step.table[b].long()[pos // step.page], pos % step.page)
            K[at[0], at[1]] += 8.0 * u
    step.K.copy_(K.to(step.K.dtype))
    j = torch.tensor([jumps[h % len(jumps)] for h in range(step.Hq)], device=DEV) * step.d ** 0.5 / 8.0
    Q = step.Q.float()
    Q[..., :16] = 0.0
    step.Q.copy_((Q + j[:, None] * u).to(step.Q.dtype))


# ---------------------------------------------------------------------------
# references that move
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("k", [None, 256])
@pytest.mark.parametrize("Hq,m", [(5, 8), (40, 1), (16, 2), (70, 1)])
def test_a_moving_reference_leaves_the_other_outputs(Hq, m, k):
    """Many short caches a multiprocessor, each of two tiles, the second far above the first: every cache's second tile
    scales its own output, while the output of the cache before it still waits to be stored."""
    units = 148 * 3
    if k is None:
        step = Step([256] * units, [m] * units, Hq, 1, 64, page=64, seed=Hq + m)
    else:
        step = Step([300] * (units // m), [m] * (units // m), Hq, 1, 64, page=64, seed=Hq + m, k=k)
        quiet, loud = [p for p in range(256) if p % 2 == 0], [p for p in range(256) if p % 2]
        step.idx.copy_(i32(quiet + loud)[None].expand_as(step.idx))
    loud_tokens(step, (lambda p: p >= 128) if k is None else (lambda p: p % 2 == 1), [20.0, 24.0, 17.0])
    check(step, *run(step))


@pytest.mark.parametrize("k", [None, 900])
@pytest.mark.parametrize("kv,Hq,Hkv,m,d", [("bf16", 64, 1, 1, 128), ("bf16", 40, 1, 1, 64), ("bf16", 33, 1, 1, 128),
                                           ("bf16", 6, 1, 8, 64), ("bf16", 8, 1, 1, 128), ("bf16", 32, 1, 1, 64),
                                           ("e4m3", 64, 1, 1, 128), ("e4m3", 128, 1, 1, 128), ("e4m3", 8, 1, 1, 64),
                                           ("fp32", 8, 2, 2, 64), ("bf16", 8, 2, 2, 256)])
def test_values_all_alike_come_out_as_they_are(kv, Hq, Hkv, m, d, k):
    """The weights of a row sum to one in the numbers that the products saw, however its references moved: where every
    value is v0 (exact in bf16) the output is v0.  Sums of n <= 1000 terms are off by n 2^-23 < 2^-13 relative, two-part
    weights by 2^-16, both far below half a bf16 step (2^-9 at the least), so the rounding gives v0 itself; fp32 outputs
    are within 2^-13."""
    step = Step([700, 1000, 140], [m] * 3, Hq, Hkv, d, kv, page=16, seed=d + Hq, k=k)
    v0 = (1.0 + torch.arange(d, device=DEV) / 8).to(torch.bfloat16) if kv != "e4m3" else torch.ones(d, device=DEV)
    if kv == "e4m3":
        step.V.copy_(torch.where(step.V.float().isnan(), step.V.float(), v0).to(step.V.dtype))
        step.scales[1].copy_(torch.where(step.scales[1].isnan(), step.scales[1], 1.5))
        v0 = v0 * 1.5
    else:
        step.V.copy_(torch.where(step.V.float().isnan(), step.V.float(), v0.float()).to(step.V.dtype))
        # jumps below and above the slack of a reference, others beyond what old weights survive
        loud_tokens(step, lambda p: p % 131 == 130 or p >= 650, [9.3, 14.7, 23.1, 3.9, 47.3, 90.1])
    out, _ = run(step)
    if kv == "fp32":
        assert float((out / v0.float() - 1).abs().max()) <= 2.0 ** -13
    else:
        assert torch.equal(out.float(), v0.float().expand_as(out))


# ---------------------------------------------------------------------------
# weights in two parts
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("k", [None, 150])
@pytest.mark.parametrize("kv,Hq,Hkv,d", TWO_PARTS)
def test_weights_of_more_than_bf16(kv, Hq, Hkv, d, k):
    # up to 32 rows, and from e4m3, a weight goes in as two bf16 parts; on the CUDA cores it is fp32
    step = cancelling(kv, Hq, Hkv, d, k)
    bad = two_parts_exceeded(step, f64(run(step)[0]))
    assert not bad.any(), np.argwhere(bad)[:4].tolist()


# ---------------------------------------------------------------------------
# empty steps
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_no_requests_into_prepared_outputs(in_place):
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    used = i32([3])
    out = (i32([9]), torch.full((5,), 11, dtype=torch.int64, device=DEV), i32([4] * 5), none.clone(),
           used if in_place else i32([8]))
    for kw in ({}, {"workspace": torch.zeros(4096, dtype=torch.uint8, device=DEV)}, {"stream": torch.cuda.Stream()}):
        for t in out[:3]:
            t.fill_(9)
        torch.cuda.synchronize()
        got = dsa.dsa_page_plan(none, none, torch.empty((0, 4), dtype=torch.int32, device=DEV), i32([1, 2, 3, 4]), used, 16, 4, 5,
                                out=out, **kw)
        torch.cuda.synchronize()
        assert got is out
        assert out[0].tolist() == [0] and out[1].tolist() == [-1] * 5 and out[2].tolist() == [-1] * 5 and out[4].tolist() == [3]


# ---------------------------------------------------------------------------
# rows of no request
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("k", [None, 70])
@pytest.mark.parametrize("kv,d", [("bf16", 128), ("e4m3", 64), ("fp32", 64), ("bf16", 136)])
def test_rows_in_front_of_the_first_request(kv, d, k):
    # some requests of a larger batch: their offsets start behind 0, and rows of the others stay as they were
    step = Step([50, 300, 129, 7], [2, 1, 3, 1], 8, 2, d, kv, k=k, pad=2, seed=4)
    want, wl = run(step)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    out, lse = torch.full_like(step.Q, 7.0), torch.full(step.Q.shape[:2], 7.0, device=DEV)
    step.table, step.lens_t, step.q_off = step.table[1:3].contiguous(), step.lens_t[1:3].contiguous(), step.q_off[1:4].contiguous()
    run(step, out, lse, workspace=ws)
    # within the rounding of sums cut at other places: both are within check's bound, and equal where nothing is cut
    assert torch.allclose(out[2:6].float(), want[2:6].float(), atol=0.02, rtol=0.02)
    assert torch.allclose(lse[2:6], wl[2:6], atol=1e-4, rtol=0)
    for x in (out, lse):
        assert torch.all(x[:2] == 7) and torch.all(x[6:] == 7)
    dsa.dsa_check_status(ws)


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def test_calls_refuse_tensors_that_want_a_gradient():
    step = Step([40, 9], [1, 2], 4, 2, 64, "bf16", k=8)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    rows, slots = torch.randn((2, 2, 64), device=DEV).bfloat16(), torch.tensor([1, 2], device=DEV)
    for kw in ({}, {"workspace": ws}):
        for i in range(3):
            a = list(step.args())
            a[i] = a[i].detach().clone().requires_grad_()
            for call in (lambda: dsa.dsa_attend_paged(*a, step.max_q, **kw), lambda: dsa.dsa_attend_selected(*a, step.idx, **kw)):
                with pytest.raises(RuntimeError, match="gradient"):
                    call()
                with torch.no_grad():
                    call()
        with pytest.raises(RuntimeError, match="gradient"):
            dsa.dsa_page_append(rows.clone().requires_grad_(), step.K, slots, v=rows, V_pages=step.V, **kw)
        with pytest.raises(RuntimeError, match="gradient"):
            dsa.dsa_page_append(rows, step.K, slots, v=rows.clone().requires_grad_(), V_pages=step.V, **kw)
        with torch.no_grad():
            dsa.dsa_page_append(rows.clone().requires_grad_(), step.K, slots, v=rows, V_pages=step.V, **kw)


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("src", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [128, 24, 7])  # 16, 8 and one element a lane
def test_append_e4m3_shows_what_is_not_finite(src, d):
    """A row that holds an infinity or a NaN reads back as NaN, all of it, whatever the alignment; rows beside it are as
    without it."""
    gen = torch.Generator().manual_seed(d)
    x = torch.randn((9, 2, d), generator=gen)
    x[1, 0, d // 2] = float("inf")
    x[3, 1, 0] = float("-inf")
    x[4, 0, d - 1] = float("nan")
    x[6, 1, 1], x[6, 1, 2] = float("nan"), float("inf")
    x = x.to(TYPES[src]).to(DEV)
    K = torch.zeros((9, 1, 2, d), dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.zeros((9, 1, 2), device=DEV)
    dsa.dsa_page_append(x, K, torch.arange(9, device=DEV), K_scale=sc, check=True)
    got = K.float()[:, 0] * sc[:, 0, :, None]
    bad = ~torch.isfinite(x.float()).all(-1)
    assert int(bad.sum()) == 4 and torch.all(got[bad].isnan()) and torch.all(sc[:, 0][bad].isnan())
    good = x.float()[~bad]
    want = (good.cpu().abs().amax(-1) / np.float32(448)).clamp(min=2.0 ** -126)
    assert torch.equal(sc[:, 0][~bad].cpu(), want)
    assert torch.equal(K[:, 0][~bad].view(torch.uint8).cpu(), (good.cpu() / want[:, None]).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("k", [None, 150])
@pytest.mark.parametrize("kv,d,Hq", [("bf16", 128, 8), ("bf16", 64, 64), ("bf16", 128, 100), ("e4m3", 128, 8), ("e4m3", 64, 64),
                                     ("e4m3", 128, 128), ("fp32", 64, 8), ("bf16", 136, 8)])
def test_attention_shows_what_is_not_finite(kv, d, Hq, k):
    """A NaN in one query row, or in a key that a request's rows read, comes out as NaN in outputs and log-sum-exp; other
    requests stay as they are."""
    lens, news = [300, 140, 520], [1, 1, 1]
    step = Step(lens, news, Hq, 1, d, kv, page=16, k=k, seed=5)
    want, wl = run(step)
    step.Q[1] = float("nan")
    out, lse = run(step)
    assert torch.all(out[1].isnan()) and torch.all(lse[1].isnan())
    for r in (0, 2):
        assert torch.equal(out[r], want[r]) and torch.equal(lse[r], wl[r])
    step = Step(lens, news, Hq, 1, d, kv, page=16, k=k, seed=5)
    pos = 130 if k is None else int(step.idx[2][step.idx[2] >= 0][77])
    at = (int(step.table[2, pos // 16]), pos % 16)
    if kv == "e4m3":
        step.scales[0][at] = float("nan")
    else:
        step.K[at] = float("nan")
    out, lse = run(step)
    assert torch.all(out[2].isnan()) and torch.all(lse[2].isnan())
    for r in (0, 1):
        assert torch.equal(out[r], want[r]) and torch.equal(lse[r], wl[r])


# ---------------------------------------------------------------------------
# pages outside the pool
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kv,d,Hq", [("bf16", 128, 8), ("bf16", 64, 64), ("bf16", 128, 100), ("e4m3", 128, 8), ("fp32", 64, 8),
                                     ("bf16", 136, 8)])
def test_list_entries_in_pages_outside_the_pool_are_skipped(kv, d, Hq):
    step = Step([300, 129], [2, 1], Hq, Hq // 8 if Hq == 8 else 1, d, kv, page=16, k=100, seed=3)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    table = step.table
    step.table = table.clone()
    step.table[0, 2:5] = i32([-1, 1 << 29, step.K.shape[0]])
    out, lse = run(step, workspace=ws, check=False)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_status(ws)
    assert e.value.status == -1
    idx = step.idx.clone()
    idx[:2] = torch.where((idx[:2] >= 32) & (idx[:2] < 80), -1, idx[:2])
    step.table, step.idx = table, idx
    check(step, out, lse)


# ---------------------------------------------------------------------------
# the bounded waits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("k", [None, 300])
@pytest.mark.parametrize("kv,Hq", [("bf16", 8), ("bf16", 64), ("bf16", 128), ("e4m3", 8), ("e4m3", 64), ("e4m3", 128)])
def test_a_wait_that_runs_out_is_reported(kv, Hq, k):
    """The first CTA never posts its first tile (dsa_debug_set_wait): the wait for it runs out, all roles leave, and the
    launch says so; the same workspace then serves a call whose results match the oracle."""
    step = Step([3000, 700], [1, 1], Hq, 1, 128, kv, page=32, k=k, seed=2)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    dsa.dsa_debug_set_wait(2000, hold_first_tile=True)
    try:
        run(step, workspace=ws, check=False)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_check_status(ws)
        assert e.value.status == -5
    finally:
        dsa.dsa_debug_set_wait(0, hold_first_tile=False)
    torch.cuda.synchronize()
    check(step, *run(step, workspace=ws))
    # a budget far above any wait of a working launch changes nothing
    dsa.dsa_debug_set_wait(20000)
    try:
        check(step, *run(step, workspace=ws))
    finally:
        dsa.dsa_debug_set_wait(0)
