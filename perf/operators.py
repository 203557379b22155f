"""The paged cache of committed context, operator by operator: what is timed and checked.

Three operators work on a pool of pages [n_pages, page, kv heads, head dim] of keys and one of values, with an
int32 page table [sequences, pages of a sequence]:

  append  per-head RMS norm of queries and keys (optional), rotation by position, keys and values into their pages
  attend  attention of one new token of each sequence over its cached positions; optionally adds the weight every
          position got, summed over the query heads that share its KV head, to an fp32 accumulator
  evict   keeps `budget` positions per sequence and KV head (the first, the most recent, and the heaviest of the
          rest) and moves them, in order, to the front of another set of pages

`run` has two forms of each: elementary torch operations (`own` false), and the package's calls (`own` true).
Head counts are those of the package's own workloads (4/2 x 64, and 12/2, 28/4, 32/8, 40/8 x 128) and a few
generic ones in `draw`.
"""
import math
import random

import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6


def _case(name, op, heads, dtype, page, n_seqs, length, **kw):
    """lengths: every sequence `length` long, or with ragged=True spread over 0..length (the first one exactly
    `length`, the second empty, the third a single position)."""
    return dict(name=name, op=op, nq=heads[0], nkv=heads[1], hd=heads[2], dtype=dtype, page=page, n_seqs=n_seqs,
                length=length, ragged=False, **kw)


def listed():
    return [
        # one sequence decodes its next token: latency
        _case("append_one", "append", (12, 2, 128), "bf16", 32, 1, 512, rows=1, norm=True),
        # a ragged batch of sequences, one new token each
        dict(_case("append_batch", "append", (40, 8, 128), "bf16", 32, 67, 1000, rows=1, norm=True), ragged=True),
        # the prompts of four requests enter the cache at once (8,188 rows)
        _case("append_prompt", "append", (40, 8, 128), "bf16", 32, 4, 2047, rows=2047, norm=True),
        # fp32 model without head norms, a page size that is no power of two
        _case("append_f32", "append", (4, 2, 64), "f32", 24, 3, 111, rows=111, norm=False),
        # one sequence, a short context: latency
        _case("attend_one", "attend", (12, 2, 128), "bf16", 32, 1, 512, weights=False),
        # four requests with the context length of the largest workload
        _case("attend_four", "attend", (40, 8, 128), "bf16", 32, 4, 4096, weights=False),
        # one sequence with a very long context: the split over its length
        _case("attend_long", "attend", (28, 4, 128), "bf16", 64, 1, 131071, weights=False),
        # a serving batch of very different lengths that also tracks what each position is worth
        dict(_case("attend_ragged", "attend", (32, 8, 128), "bf16", 16, 64, 16384, weights=True), ragged=True),
        # fp32, odd pages, an empty sequence and one of a single position
        dict(_case("attend_f32", "attend", (4, 2, 64), "f32", 24, 5, 1999, weights=True), ragged=True),
        # one sequence halves its context: latency
        _case("evict_one", "evict", (12, 2, 128), "bf16", 32, 1, 2048, budget=1024, n_first=4, n_recent=256),
        # four requests come back to the prefix capacity of the largest workload
        _case("evict_four", "evict", (40, 8, 128), "bf16", 32, 4, 16384, budget=4096, n_first=4, n_recent=512),
        # fp32, ragged: some sequences are shorter than the budget and move whole
        dict(_case("evict_f32", "evict", (4, 2, 64), "f32", 24, 33, 5001, budget=701, n_first=0, n_recent=33),
             ragged=True),
    ]


HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (10, 5, 128)]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "evict"])
    heads = rng.choice(HEADS)
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    page = rng.choice([8, 16, 24, 32, 64, 100])
    row = 2 * heads[1] * heads[2] * (4 if dtype == "f32" else 2)   # bytes of one cached position
    cap = 1.6e9 / row                                              # positions that cost what the largest listed case does
    n_seqs = _log_uniform(rng, 1, 64)
    c = dict(op=op, nq=heads[0], nkv=heads[1], hd=heads[2], dtype=dtype, page=page, n_seqs=n_seqs,
             ragged=rng.random() < 0.5)
    if op == "append":
        rows = 1 if rng.random() < 0.4 else _log_uniform(rng, 1, max(1, min(8192, 16384 // n_seqs)))
        c.update(length=rows + _log_uniform(rng, 1, 1000), rows=rows, norm=rng.random() < 0.6)
        c["ragged"] = c["ragged"] and rows == 1
    elif op == "attend":
        c.update(length=_log_uniform(rng, 1, int(min(131072, cap / n_seqs))), weights=rng.random() < 0.5)
    else:
        length = _log_uniform(rng, 2, int(min(65536, cap / 2 / n_seqs)))
        budget = rng.randint(1, length)
        first = rng.choice([0, min(4, budget)])
        c.update(length=length, budget=budget, n_first=first, n_recent=rng.randint(0, budget - first))
    return c


# ---------------------------------------------------------------- inputs

def _lens(case):
    """Cached positions of every sequence (for append: with the new rows), from the case alone."""
    n, top = case["n_seqs"], case["length"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random("%d %d" % (n, top))
    lens = [top, 0, 1] + [r.randint(0, top) for _ in range(n)]
    lens = lens[:n]
    return [max(1, x) for x in lens] if case["op"] == "append" else lens


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _table(lens, page, width, gen_np, n_pages):
    """Pages of every sequence, in an order that pages come to have after some time of use."""
    need = [-(-x // page) for x in lens]
    ids = gen_np.permutation(n_pages).astype(np.int32)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    return table


def _pages(lens, page):
    return max(1, sum(-(-x // page) for x in lens))


def _inputs(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    rs = np.random.default_rng([seed, 17])
    lens, page, dt = _lens(case), case["page"], _dtype(case)
    nq, nkv, hd, n = case["nq"], case["nkv"], case["hd"], case["n_seqs"]
    width = max(1, -(-case["length"] // page))
    n_pages = _pages(lens, page)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    s = dict(case=case, lens=ints(lens), table=ints(_table(lens, page, width, rs, n_pages)),
             max_len=case["length"], k=normal(n_pages, page, nkv, hd), v=normal(n_pages, page, nkv, hd))
    if case["op"] == "append":
        # the last `rows` positions of each sequence are new; some sequences have lost earlier positions, so that
        # a token's position is further on than its place in the cache
        rows = case["rows"]
        index = np.concatenate([np.arange(x - rows, x) for x in lens])
        seq = np.repeat(np.arange(n), rows)
        shift = rs.integers(0, 30000, n) * (rs.random(n) < 0.5)
        s.update(qkv=normal(n * rows, nq + 2 * nkv, hd), index=ints(index), seq=ints(seq),
                 pos=ints(index + shift[seq]), max_pos=case["length"] + 30000)
        if case["norm"]:
            s.update(q_gain=1.0 + 0.2 * normal(hd, dtype=torch.float32),
                     k_gain=1.0 + 0.2 * normal(hd, dtype=torch.float32))
    elif case["op"] == "attend":
        s["q"] = normal(n, nq, hd) * 2
        if case["weights"]:
            # what the attention of some 50 earlier tokens left: positive, of a wide spread
            s["w"] = (torch.exp(2 * normal(n, nkv, case["length"], dtype=torch.float32) - 2)
                      * (50 * (nq // nkv) / case["length"]))
    else:
        w = torch.exp(2 * normal(n, nkv, case["length"], dtype=torch.float32) - 3)
        w = torch.where(normal(n, nkv, case["length"], dtype=torch.float32) > 1.6, torch.zeros_like(w), w)
        s["w"] = w.to(torch.bfloat16).float() if seed % 2 else w   # coarse values: many ties
        kept = [max(1, min(x, case["budget"])) for x in lens]   # an empty sequence has a page too
        n_out = _pages(kept, page)
        s["table_out"] = ints(_table(kept, page, max(1, -(-case["budget"] // page)), rs, n_out))
        s["k_out"] = torch.zeros((n_out, page, nkv, hd), device="cuda", dtype=dt)
        s["v_out"] = torch.zeros((n_out, page, nkv, hd), device="cuda", dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import sparse_reuse_gb300 as sf
        s["cache"] = sf.PagedCache(n_q_heads=case["nq"], n_kv_heads=case["nkv"], head_dim=case["hd"],
                                   dtype=case["dtype"], page_size=case["page"], max_seqs=case["n_seqs"],
                                   max_len=case["length"], max_pos=s.get("max_pos", case["length"]), rms_eps=EPS,
                                   rope_theta=THETA, track_weights=bool(case.get("weights")))
        # outputs that a serving loop keeps
        if case["op"] == "append":
            s["q_out"] = torch.empty((s["qkv"].shape[0], case["nq"], case["hd"]), device="cuda", dtype=_dtype(case))
        elif case["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            if case["weights"]:
                s["w_out"] = torch.zeros_like(s["w"])
        else:
            s["w_out"] = torch.zeros_like(s["w"])
            s["lens_out"] = torch.empty_like(s["lens"])
            s["kept"] = torch.empty((case["n_seqs"], case["nkv"], case["budget"]), device="cuda", dtype=torch.int32)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        c = s["cache"]
        if op == "append":
            q = c.append(s["qkv"], s["index"], s["table"], s["k"], s["v"], pos=s["pos"], seq=s["seq"],
                         q_gain=s.get("q_gain"), k_gain=s.get("k_gain"), q=s["q_out"])
            return {"q": q, "k": s["k"], "v": s["v"]}
        if op == "attend":
            if s["case"]["weights"]:
                out = c.attend(s["q"], s["k"], s["v"], s["table"], s["lens"], out=s["out"], weights=s["w"],
                               weights_out=s["w_out"])
                return {"out": out, "w": s["w_out"]}
            return {"out": c.attend(s["q"], s["k"], s["v"], s["table"], s["lens"], out=s["out"])}
        case = s["case"]
        lens, kept = c.evict(s["k"], s["v"], s["table"], s["lens"], s["w"], case["budget"], n_first=case["n_first"],
                             n_recent=case["n_recent"], k_out=s["k_out"], v_out=s["v_out"],
                             table_out=s["table_out"], weights_out=s["w_out"], lens_out=s["lens_out"],
                             kept=s["kept"])
        return {"lens": lens, "kept": kept, "w": s["w_out"], "k": s["k_out"], "v": s["v_out"]}
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _plain_attend(s)
    return _plain_evict(s)


def _slots(table, seq, index, page):
    return table[seq, index // page].long() * page + index % page


def _plain_append(s):
    case = s["case"]
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    x = s["qkv"].float()
    qk = x[:, :nq + nkv]
    if "q_gain" in s:
        qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS)
        qk = torch.cat([qk[:, :nq] * s["q_gain"], qk[:, nq:] * s["k_gain"]], 1)
    j = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = s["pos"].double()[:, None] * (THETA ** (-2.0 * j / hd))
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = qk[..., :hd // 2], qk[..., hd // 2:]
    qk = torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(s["qkv"].dtype)
    slot = _slots(s["table"], s["seq"].long(), s["index"].long(), page)
    s["k"].view(-1, nkv, hd)[slot] = qk[:, nq:]
    s["v"].view(-1, nkv, hd)[slot] = s["qkv"][:, nq + nkv:]
    return {"q": qk[:, :nq].contiguous(), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    case = s["case"]
    nq, nkv, hd, page, n, m = case["nq"], case["nkv"], case["hd"], case["page"], case["n_seqs"], s["max_len"]
    j = torch.arange(m, device="cuda")
    live = j[None] < s["lens"][:, None]                                        # [n, m]
    slot = _slots(s["table"], torch.arange(n, device="cuda")[:, None], j[None], page)
    k = torch.where(live[..., None, None], s["k"].view(-1, nkv, hd)[slot], 0).float().permute(0, 2, 3, 1)
    v = torch.where(live[..., None, None], s["v"].view(-1, nkv, hd)[slot], 0).float().permute(0, 2, 1, 3)
    q = s["q"].float().view(n, nkv, nq // nkv, hd)
    score = torch.matmul(q, k) * (1.0 / math.sqrt(hd))                         # [n, nkv, group, m]
    score = torch.where(live[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1)
    out = {"out": torch.matmul(p, v).to(s["q"].dtype).view(n, nq, hd)}
    if case["weights"]:
        out["w"] = torch.where(live[:, None], s["w"] + p.sum(2), 0)
    return out


def _plain_evict(s):
    case = s["case"]
    nkv, hd, page, n, m = case["nkv"], case["hd"], case["page"], case["n_seqs"], s["max_len"]
    budget, first, recent = case["budget"], case["n_first"], case["n_recent"]
    lens = s["lens"].long()[:, None, None]                                     # [n, 1, 1]
    j = torch.arange(m, device="cuda")[None, None]
    key = torch.where((j < first) | (j >= lens - recent), math.inf, s["w"])
    key = torch.where(j < lens, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]  # heaviest first, then lowest index
    keep = torch.clamp(lens, max=budget)                                       # [n, 1, 1]
    b = torch.arange(min(budget, m), device="cuda")[None, None]
    order = torch.sort(torch.where(b < keep, order, m), dim=-1)[0]
    kept = torch.where(b < keep, order, -1)                                    # [n, nkv, budget]
    # rows behind a sequence's last kept one are written again with that one's value; an empty sequence's first
    # row with what it has
    src = torch.gather(kept, 2, torch.minimum(b, (keep - 1).clamp(min=0)).expand_as(kept)).clamp(min=0)
    dst = torch.minimum(b, (keep - 1).clamp(min=0))[:, 0]                      # [n, budget]
    row = torch.arange(n, device="cuda")
    at = _slots(s["table"], row[:, None, None], src, page)                     # [n, nkv, budget]
    to = _slots(s["table_out"], row[:, None], dst, page)                       # [n, budget]
    head = torch.arange(nkv, device="cuda")[None, :, None]
    to, some = to[:, None].expand_as(at), (keep > 0)[..., None]
    for_k, for_v = s["k_out"].view(-1, nkv, hd), s["v_out"].view(-1, nkv, hd)
    for_k[to, head] = torch.where(some, s["k"].view(-1, nkv, hd)[at, head], for_k[to, head])
    for_v[to, head] = torch.where(some, s["v"].view(-1, nkv, hd)[at, head], for_v[to, head])
    w = torch.zeros_like(s["w"])
    w[..., :b.shape[-1]] = torch.where(b < keep, torch.gather(s["w"], 2, src), 0)
    return {"lens": keep[:, 0, 0].int(), "kept": kept.int(), "w": w, "k": s["k_out"], "v": s["v_out"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    lens = _lens(case)
    row = nkv * hd * es
    if case["op"] == "append":
        t = case["n_seqs"] * case["rows"]
        # each row in and out once, its three numbers and its page's entry
        return {"bytes": t * (2 * (nq * hd * es + 2 * row) + 16), "flops": t * (nq + nkv) * hd * 10}
    total = sum(lens)
    entries = 4 * sum(-(-x // page) for x in lens)
    if case["op"] == "attend":
        return {"bytes": 2 * total * row + 2 * case["n_seqs"] * nq * hd * es + entries
                + (8 * total * nkv if case["weights"] else 0),
                "flops": 4 * total * nq * hd}
    kept = sum(min(x, case["budget"]) for x in lens)
    # accumulated weights in and out, the kept rows in and out, the list of kept positions
    return {"bytes": 8 * total * nkv + 4 * kept * row + 4 * case["n_seqs"] * nkv * case["budget"] + 2 * entries,
            "flops": total * nkv}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    nq, nkv, hd, page, n = case["nq"], case["nkv"], case["hd"], case["page"], case["n_seqs"]
    lens, group = _lens(case), nq // nkv
    table = s["table"].cpu().numpy()

    def places(tab, i, idx):
        idx = np.asarray(idx)
        return torch.from_numpy(tab[i, idx // page].astype(np.int64) * page + idx % page).cuda()

    if case["op"] == "append":
        q_out = torch.empty((s["qkv"].shape[0], nq, hd), dtype=torch.float64, device="cuda")
        k, v = s["k"].double().view(-1, nkv, hd), s["v"].double().view(-1, nkv, hd)
        freq = torch.tensor([THETA ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
        for i in range(n):
            at = slice(i * case["rows"], (i + 1) * case["rows"])
            x = s["qkv"][at].double()
            parts = []
            for y, gain in ((x[:, :nq], s.get("q_gain")), (x[:, nq:nq + nkv], s.get("k_gain"))):
                if gain is not None:
                    y = y * gain.double() * torch.rsqrt((y * y).sum(-1, keepdim=True) / hd + EPS)
                z = torch.complex(y[..., :hd // 2], y[..., hd // 2:])
                turn = torch.polar(torch.ones_like(freq), torch.zeros_like(freq))[None] * torch.exp(
                    1j * s["pos"][at].double()[:, None] * freq)
                z = z * turn[:, None]
                parts.append(torch.cat([z.real, z.imag], -1))
            to = places(table, i, s["index"][at].cpu().numpy())
            q_out[at] = parts[0]
            k[to], v[to] = parts[1], x[:, nq + nkv:]
        return {"q": q_out, "k": k.view_as(s["k"]), "v": v.view_as(s["v"])}
    if case["op"] == "attend":
        out = torch.zeros((n, nq, hd), dtype=torch.float64, device="cuda")
        w = torch.zeros((n, nkv, case["length"]), dtype=torch.float64, device="cuda") if case["weights"] else None
        for i in range(n):
            if not lens[i]:
                continue
            at = places(table, i, np.arange(lens[i]))
            k, v = s["k"].view(-1, nkv, hd)[at], s["v"].view(-1, nkv, hd)[at]
            for h in range(nkv):
                heads = slice(h * group, (h + 1) * group)
                p = torch.softmax(k[:, h].double() @ s["q"][i, heads].double().t() / math.sqrt(hd), 0)
                out[i, heads] = p.t() @ v[:, h].double()
                if w is not None:
                    w[i, h, :lens[i]] = s["w"][i, h, :lens[i]].double() + p.sum(1)
        return {"out": out, "w": w} if w is not None else {"out": out}
    budget = case["budget"]
    w_in = s["w"].cpu().numpy()
    table_out = s["table_out"].cpu().numpy()
    kept = np.full((n, nkv, budget), -1, np.int32)
    w = np.zeros(w_in.shape, np.float64)
    k, v = s["k_out"].double().view(-1, nkv, hd), s["v_out"].double().view(-1, nkv, hd)
    for i in range(n):
        m = min(lens[i], budget)
        if not m:
            continue
        to = places(table_out, i, np.arange(m))
        rest = np.arange(case["n_first"], max(case["n_first"], lens[i] - case["n_recent"]))
        for h in range(nkv):
            if lens[i] > budget:
                best = rest[np.lexsort((rest, -w_in[i, h, rest].astype(np.float64)))]
                best = best[:m - case["n_first"] - case["n_recent"]]
                ids = np.sort(np.concatenate([best, np.setdiff1d(np.arange(lens[i]), rest)]))
            else:
                ids = np.arange(m)
            kept[i, h, :m] = ids
            w[i, h, :m] = w_in[i, h, ids]
            at = places(table, i, ids)
            k[to, h], v[to, h] = s["k"].view(-1, nkv, hd)[at, h].double(), s["v"].view(-1, nkv, hd)[at, h].double()
    return {"lens": np.array([min(x, budget) for x in lens], np.int32), "kept": kept, "w": w,
            "k": k.view_as(s["k_out"]), "v": v.view_as(s["v_out"])}
