"""Float64 oracle of the paged cache: page plan, cache write, attention.

Plain numpy, written from the definitions; shares no code with the GPU path.
Bad input is the caller's to test: the oracle takes valid steps only, except
where a failing plan is itself the answer.
"""
import numpy as np

E4M3_MAX = 448.0


def page_plan(lens, new_lens, table, free_pages, used, page, max_tokens):
    """One step's plan.  Returns a dict of the outputs (``table`` a new array)
    and ``status``: 0, -1 (invalid lengths) or -8 (too few free pages)."""
    lens, new = [int(x) for x in lens], [int(x) for x in new_lens]
    table = np.array(table, dtype=np.int32, copy=True)
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int32)
    failed = {"table": table, "q_offsets": np.zeros(len(lens) + 1, np.int32), "slots": slots, "positions": positions,
              "lens": np.array(lens, np.int32), "used": used}
    if any(a < 0 or b < 0 or a + b > table.shape[1] * page for a, b in zip(lens, new)) or sum(new) > max_tokens or \
            not 0 <= used <= len(free_pages):
        return {**failed, "status": -1}
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, new))
    if used + need > len(free_pages):
        return {**failed, "status": -8}
    q_off, t = [0], 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for pos in range(n, n + m):
            if pos % page == 0:
                table[b, pos // page] = free_pages[used]
                used += 1
            slots[t] = int(table[b, pos // page]) * page + pos % page
            positions[t] = pos
            t += 1
        q_off.append(t)
    return {"table": table, "q_offsets": np.array(q_off, np.int32), "slots": slots, "positions": positions,
            "lens": np.array([a + b for a, b in zip(lens, new)], np.int32), "used": used, "status": 0}


def e4m3_scale(x):
    """Scale of one stored row [..., d]: max(amax / 448, 2^-126)."""
    return np.maximum(np.abs(np.asarray(x, np.float64)).max(-1) / E4M3_MAX, 2.0 ** -126)


def gather(pages, table_row, positions, scale=None):
    """Cache rows [n, Hkv, d] of one request at ``positions``; pages
    [n_pages, page, Hkv, d], scale [n_pages, page, Hkv] or None."""
    page = pages.shape[1]
    pos = np.asarray(positions, np.int64)
    ids, off = np.asarray(table_row, np.int64)[pos // page], pos % page
    x = pages[ids, off].astype(np.float64)
    return x if scale is None else x * scale[ids, off].astype(np.float64)[..., None]


def attend_row(q, k, v, scale):
    """One query row: q [Hq, d], k / v [n, Hkv, d] -> (out [Hq, d], lse [Hq],
    sum p |v| [Hq, d], max |scale q| . |k| [Hq])."""
    Hq, d = q.shape
    n, Hkv = k.shape[:2]
    if n == 0:
        z = np.zeros((Hq, d))
        return z, np.full(Hq, -np.inf), z, np.zeros(Hq)
    g = Hq // Hkv
    kk, vv = np.repeat(k, g, axis=1), np.repeat(v, g, axis=1)
    s = np.einsum("hd,nhd->hn", q, kk) * scale
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    mag = np.einsum("hd,nhd->hn", np.abs(q), np.abs(kk)).max(1) * abs(scale)
    return (np.einsum("hn,nhd->hd", p, vv), (np.log(total) + top)[:, 0], np.einsum("hn,nhd->hd", p, np.abs(vv)), mag)


def attend(q, k_pages, v_pages, table, lens, q_offsets, scale=None, k_scale=None, v_scale=None, idx=None):
    """All rows of a step.  Returns out [rows, Hq, d], lse [rows, Hq], the
    magnitudes of attend_row and the number of tokens each row reads; rows
    behind q_offsets[-1] hold NaN (they are padding)."""
    rows, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, mags = np.full((rows, Hq, d), np.nan), np.full((rows, Hq, d), np.nan)
    lse, tops = np.full((rows, Hq), np.nan), np.full((rows, Hq), np.nan)
    count = np.zeros(rows, np.int64)
    for b in range(len(lens)):
        q0, q1, n = int(q_offsets[b]), int(q_offsets[b + 1]), int(lens[b])
        for r in range(q0, q1):
            pos = n - (q1 - q0) + (r - q0)
            if idx is None:
                at = np.arange(max(0, pos + 1))
            else:
                at = idx[r][(idx[r] >= 0) & (idx[r] <= pos)]
            count[r] = len(at)
            out[r], lse[r], mags[r], tops[r] = attend_row(q[r].astype(np.float64), gather(k_pages, table[b], at, k_scale),
                                                          gather(v_pages, table[b], at, v_scale), scale)
    return out, lse, mags, tops, count
