"""The paged-cache operators as they are measured: cases, inputs, plain forms and work.

Four operators of the serving path that follows the indexer:
  plan      block tables and slot maps from request lengths   (dsa_page_plan)
  append    new keys and values into their cache slots        (dsa_page_append)
  attend    new queries over all cached tokens                (dsa_attend_paged)
  selected  queries over the positions the indexer chose      (dsa_attend_selected)
"""
import random

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest normal float32: the floor of a scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _plan(name, requests, longest, new, page, spare=7):
    return {"name": name, "op": "plan", "requests": requests, "longest": longest, "new": new, "page": page,
            "spare": spare}


def _append(name, tokens, kv_heads, d, src, cache, page, padded=0):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads, "d": d, "src": src,
            "cache": cache, "page": page, "padded": padded}


def _attend(name, requests, longest, ragged, new, heads, kv_heads, d, cache, page, joint=False):
    return {"name": name, "op": "attend", "requests": requests, "longest": longest, "ragged": ragged, "new": new,
            "heads": heads, "kv_heads": kv_heads, "d": d, "cache": cache, "page": page, "joint": joint}


def _selected(name, requests, longest, ragged, new, heads, kv_heads, d, cache, page, k, joint=False):
    return {**_attend(name, requests, longest, ragged, new, heads, kv_heads, d, cache, page, joint),
            "op": "selected", "k": k}


def listed():
    return [
        # a decode step of a small server: eight requests, a token or two each
        _plan("plan_decode_8", 8, 4096, 2, 64),
        # a step that admits prompts: a thousand requests, up to 2048 new tokens each, about a million slots
        _plan("plan_prompts_1024", 1024, 8192, 2048, 16),
        # one decode step's rows (32 requests, two tokens each) with a padded tail, into a bf16 cache
        _append("append_decode_bf16", 64, 8, 128, "bfloat16", "bfloat16", 64, padded=16),
        # a 32K-token prompt into an 8-bit cache with a scale for each token and head
        _append("append_prompt_e4m3", 32768, 8, 128, "bfloat16", "e4m3", 64),
        # the smallest call: one request, one token, a short cache (latency)
        _attend("attend_one_257", 1, 257, False, 1, 32, 8, 128, "bfloat16", 16),
        # an ordinary mixed batch: 64 requests of 0 to 8191 tokens, K and V of a page side by side, d = 64
        _attend("attend_ragged_64x8k", 64, 8191, True, 1, 32, 8, 64, "bfloat16", 32, joint=True),
        # the decode indexer's own shape: 32 caches of 131072 tokens, two queries each, 64 heads over one key
        _attend("attend_32x128k", 32, 131072, False, 2, 64, 1, 128, "bfloat16", 128),
        # 8-bit cache with scales, grouped heads, ragged
        _attend("attend_e4m3_16x32k", 16, 32768, True, 1, 64, 8, 128, "e4m3", 64),
        # the step that follows the decode indexer: its 2048 positions for each of 64 query rows
        _selected("selected_decode_32x128k", 32, 131072, False, 2, 64, 1, 128, "bfloat16", 64, 2048),
        # the step that follows the dense indexer: rows of one 32K prompt, 2048 positions each
        _selected("selected_prompt_4k", 1, 32768, False, 4096, 64, 1, 128, "bfloat16", 64, 2048),
        # a small batch with an 8-bit cache
        _selected("selected_e4m3_4x8k", 4, 8192, True, 1, 64, 8, 128, "e4m3", 32, 2048),
        # the exact fp32 path at the fp32 indexer's shape: 2048 rows, 4 heads of 64, 64 positions each
        _selected("selected_fp32_2k", 1, 2048, False, 2048, 4, 4, 64, "float32", 64, 64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "selected", "selected"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    if op == "plan":
        new = rng.choice([1, 4, _log(rng, 1, 2048)])
        return {**_plan("", _log(rng, 1, 1024), _log(rng, 16, 16384), new, max(8, page), rng.randint(0, 9))}
    if op == "append":
        src, cache = rng.choice([("bfloat16", "bfloat16"), ("bfloat16", "e4m3"), ("float32", "float32"),
                                 ("float32", "e4m3")])
        tokens = _log(rng, 1, 16384)
        return _append("", tokens, rng.choice([1, 2, 4, 8]), rng.choice([32, 64, 80, 128]), src, cache, page,
                       rng.randint(0, tokens // 4))
    heads, kv_heads = rng.choice([(8, 8), (32, 8), (40, 8), (64, 8), (28, 4), (16, 2), (64, 1), (16, 1), (6, 2)])
    d = rng.choice([64, 128])
    cache = rng.choice(["bfloat16", "bfloat16", "bfloat16", "e4m3"])
    ragged, joint = rng.random() < 0.7, rng.random() < 0.3 and cache != "e4m3"
    if op == "attend":
        requests, new = _log(rng, 1, 128), rng.randint(1, 4)
        # no more cached elements than 1/4 of the largest listed case's
        most = max(1, 32 * 131072 // (4 * requests * kv_heads))
        return _attend("", requests, _log(rng, 1, min(131072, most)), ragged, new, heads, kv_heads, d, cache, page,
                       joint)
    k = rng.choice([1, 63, 64, 500, 1024, 2047, 2048])
    requests, new = rng.choice([(_log(rng, 1, 64), rng.randint(1, 4)), (1, _log(rng, 16, 512))])
    most = max(new, 32 * 131072 // (4 * requests * kv_heads))
    longest = max(new, _log(rng, 16, min(65536, most)))
    return _selected("", requests, longest, ragged and requests > 1, new, heads, kv_heads, d, cache, page, k, joint)


def _rng(case):
    return random.Random(":".join(f"{k}={case[k]}" for k in sorted(case) if k != "name"))


def _lens(case):
    """Cached tokens of each request, its new ones included (plan: before them); a ragged batch holds the longest, an
    empty one and all between."""
    r, n, top = _rng(case), case["requests"], case["longest"]
    if case["op"] != "plan" and not case["ragged"]:
        return [top] * n
    lens = [r.randint(0, top) for _ in range(n)]
    lens[r.randrange(n)] = top
    if n > 2 and case["op"] != "selected":
        lens[r.randrange(n)] = 0
    if case["op"] == "selected":
        lens = [max(case["new"], v) for v in lens]
    return lens


def _news(case):
    """New tokens of each request: `new`, but for a plan up to `new` and at times none."""
    if case["op"] != "plan":
        return [case["new"]] * case["requests"]
    r = random.Random(case["new"] * 7919 + case["requests"])
    return [case["new"] if r.random() < 0.5 else r.randint(0, case["new"]) for _ in range(case["requests"])]


def _pages(tokens, page):
    return -(-tokens // page)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_TYPES = {"bfloat16": torch.bfloat16, "float32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _pool(gen, case, n_pages):
    """K and V pages [n_pages, page, kv_heads, d] and, for e4m3, scales [n_pages, page, kv_heads]."""
    page, hk, d = case["page"], case["kv_heads"], case["d"]
    dtype = _TYPES[case["cache"]]
    if case["cache"] == "e4m3":
        k = _normal(gen, (n_pages, page, hk, d), torch.float32, 150.0).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)
        v = _normal(gen, (n_pages, page, hk, d), torch.float32, 150.0).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)
        scales = [(torch.rand((n_pages, page, hk), generator=gen, device="cuda") + 0.5) / 150.0 for _ in range(2)]
        return k, v, scales[0], scales[1]
    if case.get("joint"):
        both = _normal(gen, (n_pages, 2, page, hk, d), dtype)
        return both[:, 0], both[:, 1], None, None
    return _normal(gen, (n_pages, page, hk, d), dtype), _normal(gen, (n_pages, page, hk, d), dtype), None, None


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    page = case["page"]
    # a serving program keeps one zeroed workspace for all its calls
    s = {"case": case, "workspace": torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")}
    if case["op"] == "plan":
        lens, news = _lens(case), _news(case)
        held = [_pages(n, page) for n in lens]
        width = max(_pages(a + b, page) for a, b in zip(lens, news)) + 3
        need = sum(_pages(a + b, page) - c for a, b, c in zip(lens, news, held))
        n_pages = sum(held) + need + 2 * case["spare"]
        ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), _int(held, torch.int64))
        first = torch.cumsum(_int(held, torch.int64), 0) - _int(held, torch.int64)
        table[row, torch.arange(sum(held), device="cuda") - first[row]] = ids[:sum(held)]
        s.update(lens=_int(lens), news=_int(news), table=table, free=ids[sum(held):].contiguous(),
                 used=_int([case["spare"]]), n_pages=n_pages, max_tokens=sum(news) + 5 * case["spare"])
        return s
    if case["op"] == "append":
        t, hk, d = case["tokens"], case["kv_heads"], case["d"]
        n_pages = _pages(t, page) + 3
        src = _TYPES[case["src"]]
        s["k"], s["v"] = _normal(gen, (t, hk, d), src), _normal(gen, (t, hk, d), src)
        s["kp"], s["vp"], s["ks"], s["vs"] = _pool(gen, case, n_pages)
        slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:t].contiguous()
        if case["padded"]:
            slots[t - case["padded"]:] = -1
        s["slots"] = slots
        return s
    lens, news = _lens(case), _news(case)
    held = [max(1, _pages(n, page)) for n in lens]
    n_pages, width, total = sum(held) + 2, max(held), sum(news)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), _int(held, torch.int64))
    first = torch.cumsum(_int(held, torch.int64), 0) - _int(held, torch.int64)
    table[row, torch.arange(sum(held), device="cuda") - first[row]] = ids[:sum(held)]
    q_type = torch.float32 if case["cache"] == "float32" else torch.bfloat16
    s["q"] = _normal(gen, (total, case["heads"], case["d"]), q_type, 1.5)
    s["kp"], s["vp"], s["ks"], s["vs"] = _pool(gen, case, n_pages)
    s.update(table=table, lens=_int(lens), max_len=max(lens), max_q=max(news),
             q_offsets=torch.cumsum(_int([0] + news), 0).to(torch.int32))
    if case["op"] == "selected":
        k = case["k"]
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, news)]).to("cuda")
        idx = torch.full((total, k), -1, dtype=torch.int32, device="cuda")
        for r0 in range(0, total, 512):  # k distinct positions of each row's prefix, -1 where it is shorter
            p = pos[r0:r0 + 512, None]
            noise = torch.rand((p.shape[0], max(lens)), generator=gen, device="cuda")
            noise[torch.arange(max(lens), device="cuda")[None] > p] = -1.0
            got = noise.topk(min(k, max(lens)), dim=1)
            idx[r0:r0 + 512, :got.indices.shape[1]] = torch.where(got.values >= 0, got.indices, -1).to(torch.int32)
        s["idx"] = idx
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plan_plain(s):
    c, table = s["case"], s["table"]
    page, n, m = c["page"], s["lens"].shape[0], s["max_tokens"]
    lens, news = s["lens"].long(), s["news"].long()
    after = lens + news
    held, want = (lens + page - 1) // page, (after + page - 1) // page
    q_off = torch.cat([torch.zeros(1, dtype=torch.int64, device=lens.device), torch.cumsum(news, 0)])
    first = s["used"].long() + torch.cumsum(want - held, 0) - (want - held)
    col = torch.arange(table.shape[1], device=lens.device)[None]
    fresh = (col >= held[:, None]) & (col < want[:, None])
    at = (first[:, None] + col - held[:, None]).clamp(0, s["free"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    t = torch.arange(m, device=lens.device)
    b = torch.searchsorted(q_off[1:], t, right=True).clamp(max=n - 1)
    pos = lens[b] + t - q_off[b]
    slot = table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    live = t < q_off[-1]
    return (table, q_off.to(torch.int32), torch.where(live, slot, -1), torch.where(live, pos, -1).to(torch.int32),
            after.to(torch.int32), (s["used"] + (want - held).sum()).to(torch.int32))


def _quantise(x):
    x = x.float()
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _append_plain(s):
    live = s["slots"] >= 0
    at = s["slots"][live]
    page = s["case"]["page"]
    rows, offs = at // page, at % page
    if s["ks"] is None:
        s["kp"][rows, offs] = s["k"][live]
        s["vp"][rows, offs] = s["v"][live]
        return s["kp"], s["vp"]
    (k, ks), (v, vs) = _quantise(s["k"][live]), _quantise(s["v"][live])
    s["kp"].view(torch.uint8)[rows, offs] = k.view(torch.uint8)
    s["vp"].view(torch.uint8)[rows, offs] = v.view(torch.uint8)
    s["ks"][rows, offs] = ks
    s["vs"][rows, offs] = vs
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _index(pages, ids, offs):
    """pages[ids, offs], 8-bit values by their bytes."""
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[ids, offs].view(pages.dtype)
    return pages[ids, offs]


def _rows(pages, scale, ids, offs, seen):
    """Cache rows at (page, offset) in 32 bits, zero where not `seen`."""
    x = _index(pages, ids, offs).float()
    if scale is not None:
        x = x * scale[ids, offs][..., None]
    return torch.where(seen[..., None, None], x, 0.0)


def _softmax_values(scores, seen):
    """(weights, log-sum-exp) over the last axis; a row that sees nothing has weights 0 and -inf."""
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), (torch.log(total) + top)[..., 0]


def _attend_plain(s):
    c, q, q_off = s["case"], s["q"], s["q_offsets"].long()
    page, hk, d = c["page"], c["kv_heads"], c["d"]
    b, g, n, m = len(q_off) - 1, c["heads"] // hk, s["max_len"], s["max_q"]
    lens, news = s["lens"].long(), q_off[1:] - q_off[:-1]
    pos = torch.arange(max(n, 1), device=q.device)
    held = pos[None] < lens[:, None]
    ids = torch.where(held, s["table"][:, (pos // page).clamp(max=s["table"].shape[1] - 1)], 0).long()
    offs = (pos % page).expand_as(ids)
    k, v = _rows(s["kp"], s["ks"], ids, offs, held), _rows(s["vp"], s["vs"], ids, offs, held)
    j = torch.arange(m, device=q.device)
    row = (q_off[:-1, None] + j).clamp(max=q.shape[0] - 1)
    x = q[row].float().view(b, m, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, m * g, d)
    sc = (x @ k.permute(0, 2, 3, 1)) * d ** -0.5  # [b, hk, m g, n]
    last = lens[:, None] - news[:, None] + j
    seen = (pos[None, None] <= last[:, :, None]) & held[:, None]
    seen = seen[:, None, :, None].expand(b, 1, m, g, len(pos)).reshape(b, 1, m * g, len(pos))
    p, lse = _softmax_values(sc, seen)
    o = p @ v.permute(0, 2, 1, 3)
    o = o.view(b, hk, m, g, d).permute(0, 2, 1, 3, 4).reshape(b * m, hk * g, d)
    lse = lse.view(b, hk, m, g).permute(0, 2, 1, 3).reshape(b * m, hk * g)
    live = (j[None] < news[:, None]).reshape(-1)
    return o[live].to(q.dtype), lse[live]


def _selected_plain(s):
    c, q, q_off = s["case"], s["q"], s["q_offsets"].long()
    page, hk, d = c["page"], c["kv_heads"], c["d"]
    r, g = q.shape[0], c["heads"] // hk
    t = torch.arange(r, device=q.device)
    b = torch.searchsorted(q_off[1:], t, right=True)
    pos = s["lens"].long()[b] - q_off[b + 1] + t
    idx = s["idx"].long()
    seen = (idx >= 0) & (idx <= pos[:, None])
    at = torch.where(seen, idx, 0)
    ids, offs = s["table"][b[:, None], at // page].long(), at % page
    k, v = _rows(s["kp"], s["ks"], ids, offs, seen), _rows(s["vp"], s["vs"], ids, offs, seen)
    x = q.float().view(r, hk, g, d)
    p, lse = _softmax_values((x @ k.permute(0, 2, 3, 1)) * d ** -0.5, seen[:, None, None])
    o = p @ v.permute(0, 2, 1, 3)
    return o.reshape(r, hk * g, d).to(q.dtype), lse.reshape(r, hk * g)


def _run_own(s):
    import sparse_attention_token_index_b200 as dsa
    op, ws = s["case"]["op"], s["workspace"]
    if op == "plan":
        return (s["table"],) + tuple(dsa.dsa_page_plan(s["lens"], s["news"], s["table"], s["free"], s["used"],
                                                       page=s["case"]["page"], n_pages=s["n_pages"],
                                                       max_tokens=s["max_tokens"], workspace=ws))
    if op == "append":
        dsa.dsa_page_append(s["k"], s["kp"], s["slots"], v=s["v"], V_pages=s["vp"], K_scale=s["ks"], V_scale=s["vs"],
                            workspace=ws)
        return (s["kp"], s["vp"]) if s["ks"] is None else (s["kp"], s["vp"], s["ks"], s["vs"])
    if op == "attend":
        return dsa.dsa_attend_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["q_offsets"],
                                    max_q=s["max_q"], K_scale=s["ks"], V_scale=s["vs"], return_lse=True, workspace=ws)
    return dsa.dsa_attend_selected(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["q_offsets"], s["idx"],
                                   K_scale=s["ks"], V_scale=s["vs"], return_lse=True, workspace=ws)


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain,
            "selected": _selected_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work and the 64-bit answers
# ---------------------------------------------------------------------------
def _size(name):
    return {"bfloat16": 2, "float32": 4, "e4m3": 1}[name]


def work(case):
    op = case["op"]
    if op == "plan":
        lens, news, page = _lens(case), _news(case), case["page"]
        fresh = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(lens, news))
        n = len(lens)
        # lengths in, offsets and lengths out; each new page read and entered; a slot and a position a token
        return {"bytes": 8 * n + 8 * n + 8 * fresh + 12 * sum(news), "flops": 0}
    d, hk = case["d"], case["kv_heads"]
    if op == "append":
        live = case["tokens"] - case["padded"]
        row = 2 * hk * (d * (_size(case["src"]) + _size(case["cache"])) + (4 if case["cache"] == "e4m3" else 0))
        return {"bytes": live * row + 8 * case["tokens"], "flops": 0}
    lens, m, h = _lens(case), case["new"], case["heads"]
    q = 4 if case["cache"] == "float32" else 2
    token = 2 * hk * (d * _size(case["cache"]) + (4 if case["cache"] == "e4m3" else 0))
    io = len(lens) * m * h * (2 * d * q + 4)
    if op == "attend":
        pairs = sum(max(0, n - m + j + 1) for n in lens for j in range(m))
        return {"bytes": sum(lens) * token + io, "flops": 4 * pairs * h * d}
    pairs = sum(min(case["k"], n - m + j + 1) for n in lens for j in range(m))
    # rows of one request share cached tokens: no more is read than its cache holds
    read = sum(min(n, sum(min(case["k"], n - m + j + 1) for j in range(m))) for n in lens)
    return {"bytes": read * token + io + len(lens) * m * case["k"] * 4, "flops": 4 * pairs * h * d}


def _exact_row(q, k, v, scale):
    """q [h, g, d], k / v [n, h, d] in 64 bits -> (out [h, g, d], lse [h, g])."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), dtype=q.dtype, device=q.device)
    sc = torch.einsum("hgd,nhd->hgn", q, k) * scale
    lse = torch.logsumexp(sc, -1)
    return torch.einsum("hgn,nhd->hgd", torch.exp(sc - lse[..., None]), v), lse


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    page, d, hk = case["page"], case["d"], case["kv_heads"]
    if case["op"] == "append":
        keep = s["slots"] >= 0
        to = (s["slots"][keep] // page, s["slots"][keep] % page)
        pages, scales = [], []
        for x, p, sc in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
            x, p = x[keep].double(), p.float().double()
            if sc is not None:
                top = x.abs().max(-1).values / E4M3_MAX
                sc = sc.double()
                sc[to] = top
                scales.append(sc)
                x = x / top[..., None]
            p[to] = x
            pages.append(p)
        return tuple(pages + scales)

    def wide(pages, sc, i, o):
        x = _index(pages, i, o).double()
        return x if sc is None else x * sc[i, o].double()[..., None]

    q = s["q"].double().view(s["q"].shape[0], hk, case["heads"] // hk, d)
    lens, news, outs, lses = _lens(case), _news(case), [], []
    row = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        every = torch.arange(n, device="cuda")
        if case["op"] == "attend":
            at = s["table"][b].long()[every // page], every % page
            k, v = wide(s["kp"], s["ks"], *at), wide(s["vp"], s["vs"], *at)
        for j in range(m):
            if case["op"] == "selected":
                i = s["idx"][row].long()
                i = i[i >= 0]
                at = s["table"][b].long()[i // page], i % page
                o, e = _exact_row(q[row], wide(s["kp"], s["ks"], *at), wide(s["vp"], s["vs"], *at), d ** -0.5)
            else:
                seen = max(0, n - m + j + 1)
                o, e = _exact_row(q[row], k[:seen], v[:seen], d ** -0.5)
            outs.append(o.reshape(-1, d))
            lses.append(e.reshape(-1))
            row += 1
    return torch.stack(outs), torch.stack(lses)
