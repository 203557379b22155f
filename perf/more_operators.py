"""More operators on the paged cache of committed context: what is timed and checked.

Keys and values live in pools of pages [n_pages, page, kv heads, head dim] with an int32 page table [sequences, pages of
a sequence].  Four operators:

  append      per-head RMS norm of queries and keys (optional), rotation by position in one of its forms (halves or
              neighbours paired, part of the head, frequencies scaled for long contexts), keys and values into their pages
  reposition  keys that are in the cache already, turned from the positions they were stored for to new ones
  rows        attention of a block of rows of every sequence over all of its cached positions (no mask among the
              rows: a denoising block over its prefix, or a decoder's rows over an encoder's states)
  shared      attention of one new token per sequence, where groups of sequences share a prefix (the branches of a
              request) and each has some positions of its own behind it

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
ORIGINAL = 4096   # positions that scaled frequencies were made for


def _case(name, op, heads, dtype, page, **kw):
    return dict(name=name, op=op, nq=heads[0], nkv=heads[1], hd=heads[2], dtype=dtype, page=page, **kw)


def listed():
    return [
        # one sequence decodes its next token, neighbours paired, frequencies of a context stretched by 8: latency
        _case("append_one", "append", (12, 2, 128), "bf16", 32, n_seqs=1, length=512, rows=1, norm=True,
              layout="interleaved", rdim=128, scaling="yarn", factor=8.0),
        # the prompts of four requests enter the cache at once (8,188 rows), half of each head rotated
        _case("append_prompt", "append", (40, 8, 128), "bf16", 32, n_seqs=4, length=2047, rows=2047, norm=True,
              layout="half", rdim=64, scaling="linear", factor=4.0),
        # fp32 model without head norms, part of the head in neighbouring pairs, a page size that is no power of two
        _case("append_f32", "append", (4, 2, 64), "f32", 24, n_seqs=3, length=111, rows=111, norm=False,
              layout="interleaved", rdim=32, scaling="bands", factor=8.0),
        # one sequence after it has halved its context: latency
        _case("reposition_one", "reposition", (12, 2, 128), "bf16", 32, n_seqs=1, length=1024, before=2048,
              ragged=False, layout="half", rdim=128, scaling="none", factor=1.0),
        # four requests that came back to the prefix capacity of the largest workload: their keys become a prefix
        # at positions 0..4095 again
        _case("reposition_four", "reposition", (40, 8, 128), "bf16", 32, n_seqs=4, length=4096, before=16384,
              ragged=False, layout="half", rdim=128, scaling="none", factor=1.0),
        # one sequence's denoising block over a short prefix: latency
        _case("rows_one", "rows", (12, 2, 128), "bf16", 32, n_seqs=1, rows=32, length=512, ragged=False),
        # the blocks of all branches (9 x 32 rows) of four requests over the largest workload's prefixes
        _case("rows_four", "rows", (40, 8, 128), "bf16", 32, n_seqs=4, rows=288, length=4096, ragged=False),
        # a ragged batch of decoder rows over encoder states of other lengths
        _case("rows_ragged", "rows", (32, 8, 128), "bf16", 16, n_seqs=16, rows=1021, length=8191, ragged=True),
        # fp32, odd pages, a sequence without rows or states and one of a single row
        _case("rows_f32", "rows", (4, 2, 64), "f32", 24, n_seqs=5, rows=33, length=1999, ragged=True),
        # nine branches of one request, each some tokens past the shared context: latency
        _case("shared_one", "shared", (12, 2, 128), "bf16", 32, n_groups=1, members=9, prefix=512, tail=32,
              ragged=False),
        # the branches of four requests over the largest workload's prefixes
        _case("shared_four", "shared", (40, 8, 128), "bf16", 32, n_groups=4, members=9, prefix=4096, tail=32,
              ragged=False),
        # a serving batch: system prompts of very different lengths and use, tails likewise, some sequences without one
        _case("shared_ragged", "shared", (32, 8, 128), "bf16", 16, n_groups=5, members=61, prefix=32767, tail=701,
              ragged=True),
    ]


HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (10, 5, 128)]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "reposition", "rows", "rows", "shared", "shared"])
    heads = rng.choice(HEADS)
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    nq, nkv, hd = heads
    c = _case("", op, heads, dtype, rng.choice([8, 16, 24, 32, 64, 100]))
    del c["name"]
    row = 2 * nkv * hd * (4 if dtype == "f32" else 2)   # bytes of one cached position
    if op in ("append", "reposition"):
        c.update(layout=rng.choice(["half", "interleaved"]), rdim=rng.choice([x for x in (16, 32, 48, 64, 96, 128) if x <= hd]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), factor=rng.choice([2.0, 4.0, 8.0, 3.5]))
        c["factor"] = 1.0 if c["scaling"] == "none" else c["factor"]
    if op == "append":
        n = _log_uniform(rng, 1, 64)
        rows = 1 if rng.random() < 0.4 else _log_uniform(rng, 1, max(1, min(4096, 8000 // n)))
        c.update(n_seqs=n, rows=rows, length=rows + _log_uniform(rng, 1, 1000), norm=rng.random() < 0.6)
    elif op == "reposition":
        n = _log_uniform(rng, 1, 64)
        length = _log_uniform(rng, 1, int(min(32768, 130e6 / row / n)))
        c.update(n_seqs=n, length=length, before=length + _log_uniform(rng, 1, 20000), ragged=rng.random() < 0.5)
    elif op == "rows":
        # at most what the largest listed case computes (fp32, on slower units, a fraction of it)
        top = 3.6e7 if dtype == "bf16" else 1e6
        n = _log_uniform(rng, 1, 32)
        rows = _log_uniform(rng, 1, 1024)
        length = _log_uniform(rng, 1, int(max(1, min(65536, top * 32 / nq / n / rows, 3.9e8 / row / n))))
        c.update(n_seqs=n, rows=rows, length=length, ragged=rng.random() < 0.5)
    else:
        g, m = _log_uniform(rng, 1, 8), _log_uniform(rng, 1, 64)
        c.update(n_groups=g, members=m, prefix=_log_uniform(rng, 1, int(min(65536, 3e8 / row / g, 1e8 / nq / g / m))),
                 tail=_log_uniform(rng, 1, int(max(1, min(2048, 9e7 / row / g / m)))), ragged=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- inputs

def _spread(top, n, ragged, least=0):
    """n lengths: every one `top`, or spread over 0..top (the first exactly `top`, the second 0, the third 1)."""
    if not ragged:
        return [top] * n
    r = random.Random("%d %d" % (n, top))
    return [max(least, x) for x in ([top, 0, 1] + [r.randint(0, top) for _ in range(n)])[:n]]


def _lens(case):
    """Cached positions of every sequence (for append: with the new rows), from the case alone."""
    if case["op"] == "shared":
        return _spread(case["tail"], sum(_members(case)), case["ragged"])
    return _spread(case["length"], case["n_seqs"], case.get("ragged", False))


def _rows(case):
    """Rows of every sequence ("rows"): a sequence without states has rows, one of a single state has none."""
    n = _spread(case["rows"], case["n_seqs"], case["ragged"])
    return n if not case["ragged"] else n[:1] + n[1:][::-1]


def _members(case):
    """Sequences of every group ("shared"), then those of no group."""
    return _spread(case["members"], case["n_groups"], case["ragged"]) + [3 if case["ragged"] else 0]


def _prefixes(case):
    n = _spread(case["prefix"], case["n_groups"], case["ragged"])
    return n if not case["ragged"] else n[:1] + n[1:][::-1]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _table(lens, page, width, gen_np, n_pages, first=0):
    """Pages of every sequence, in an order that pages come to have after some time of use."""
    need = [-(-x // page) for x in lens]
    ids = gen_np.permutation(n_pages).astype(np.int32) + first
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    return table


def _pages(lens, page):
    return max(1, sum(-(-x // page) for x in lens))


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)])


def _inputs(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    rs = np.random.default_rng([seed, 23])
    lens, page, dt = _lens(case), case["page"], _dtype(case)
    nq, nkv, hd, n = case["nq"], case["nkv"], case["hd"], len(lens)

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    top = max(1, max(lens))
    n_pages = _pages(lens, page)
    s = dict(case=case, lens=ints(lens), table=ints(_table(lens, page, -(-top // page), rs, n_pages)), max_len=top,
             n_seqs=n, max_pos=top)
    if case["op"] == "shared":
        prefixes, members = _prefixes(case), _members(case)
        width, more = -(-max(1, max(prefixes)) // page), _pages(prefixes, page)
        s.update(prefix_lens=ints(prefixes), starts=ints(_offsets(members[:-1])), max_len=max(top, max(prefixes)),
                 prefix_table=ints(_table(prefixes, page, width, rs, more, n_pages)), q=normal(n, nq, hd) * 2,
                 prefix_top=max(1, max(prefixes)), tail_top=top)
        n_pages += more
    s["k"], s["v"] = normal(n_pages, page, nkv, hd), normal(n_pages, page, nkv, hd)
    if case["op"] == "append":
        # the last `rows` positions of each sequence are new; some sequences have lost earlier positions, so that
        # a token's position is further on than its place in the cache
        rows = case["rows"]
        index = np.concatenate([np.arange(x - rows, x) for x in lens])
        seq = np.repeat(np.arange(n), rows)
        shift = rs.integers(0, 100000, n) * (rs.random(n) < 0.5)
        s.update(qkv=normal(n * rows, nq + 2 * nkv, hd), index=ints(index), seq=ints(seq),
                 pos=ints(index + shift[seq]), max_pos=case["length"] + 100000)
        if case["norm"]:
            s.update(q_gain=1.0 + 0.2 * normal(hd, dtype=torch.float32),
                     k_gain=1.0 + 0.2 * normal(hd, dtype=torch.float32))
    elif case["op"] == "reposition":
        # what an eviction kept: some of `before` positions in ascending order, others for every head; the new ones
        # are the places
        at = np.sort(rs.random((n, nkv, case["length"])), -1) * (case["before"] - case["length"] + 1)
        s.update(pos_from=ints(at.astype(np.int64) + np.arange(case["length"])), max_pos=case["before"])
    elif case["op"] == "rows":
        # some rows of padding behind the last sequence's
        rows = _rows(case)
        s.update(starts=ints(_offsets(rows)), rows_top=max(1, max(rows)), total=sum(rows),
                 q=normal(sum(rows) + 3, nq, hd) * 2)
    if case["op"] in ("rows", "shared"):
        s["out"] = torch.zeros_like(s["q"])   # an output that a serving loop keeps
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import sparse_reuse_gb300 as sf
        more = {}
        if "layout" in case:
            freq, magnitude = sf.rotary_frequencies(case["rdim"], THETA, scaling=case["scaling"], factor=case["factor"],
                                                    original_len=ORIGINAL)
            more = dict(rotary_dim=case["rdim"], rotary_layout=case["layout"], inv_freq=freq, rotary_magnitude=magnitude)
        if "q" in s:
            more = dict(max_rows=s["q"].shape[0])
        s["cache"] = sf.PagedCache(n_q_heads=case["nq"], n_kv_heads=case["nkv"], head_dim=case["hd"],
                                   dtype=case["dtype"], page_size=case["page"], max_seqs=s["n_seqs"],
                                   max_len=s["max_len"], max_pos=s["max_pos"], rms_eps=EPS, rope_theta=THETA, **more)
        if case["op"] == "append":
            s["q_out"] = torch.empty((s["qkv"].shape[0], case["nq"], case["hd"]), device="cuda", dtype=_dtype(case))
        elif case["op"] == "rows":
            s["lse"] = torch.zeros((s["q"].shape[0], case["nq"]), device="cuda", dtype=torch.float32)
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
        if op == "reposition":
            c.reposition(s["k"], s["table"], s["lens"], s["pos_from"])
            return {"k": s["k"]}
        if op == "rows":
            out = c.attend_rows(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], out=s["out"], lse=s["lse"])
            return {"out": out, "lse": s["lse"]}
        return {"out": c.attend_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix_table"],
                                       s["prefix_lens"], s["starts"], out=s["out"])}
    if op == "append":
        return _plain_append(s)
    if op == "reposition":
        return _plain_reposition(s)
    if op == "rows":
        return _plain_rows(s)
    return _plain_shared(s)


def _slots(table, seq, index, page):
    return table[seq, index // page].long() * page + index % page


def _frequencies(case):
    """Angle of a step of one position for every rotated pair, and the factor on sine and cosine."""
    d, factor = case["rdim"], case["factor"]
    j = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    f = THETA ** (-2.0 * j / d)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "ntk":
        return (THETA * factor ** (d / (d - 2.0))) ** (-2.0 * j / d), 1.0
    if case["scaling"] == "yarn":
        # pairs that turn more than 32 times within the original context keep their frequency, those that turn less
        # than once are stretched, those between are blended by their index
        low = max(0.0, float(math.floor(d * math.log(ORIGINAL / (32.0 * 2 * math.pi)) / (2 * math.log(THETA)))))
        high = min(d - 1.0, float(math.ceil(d * math.log(ORIGINAL / (1.0 * 2 * math.pi)) / (2 * math.log(THETA)))))
        ramp = torch.clamp((j - low) / max(high - low, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if case["scaling"] == "bands":
        # the same by the number of turns: four or more stay, one or fewer are stretched
        ramp = torch.clamp((ORIGINAL * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0, 1)
        return f * ramp + f / factor * (1 - ramp), 1.0
    return f, 1.0


def _turn(x, angle, case, magnitude):
    """[..., heads, hd] turned by angles [..., 1 or heads, rdim / 2] (in 64 bits)."""
    cos, sin = (torch.cos(angle) * magnitude).float(), (torch.sin(angle) * magnitude).float()
    d = case["rdim"]
    if case["layout"] == "half":
        a, b = x[..., :d // 2], x[..., d // 2:d]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., :d:2], x[..., 1:d:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., d:]], -1)


def _plain_append(s):
    case = s["case"]
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    qk = s["qkv"][:, :nq + nkv].float()
    if "q_gain" in s:
        qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS)
        qk = torch.cat([qk[:, :nq] * s["q_gain"], qk[:, nq:] * s["k_gain"]], 1)
    freq, magnitude = _frequencies(case)
    qk = _turn(qk, (s["pos"].double()[:, None] * freq)[:, None], case, magnitude).to(s["qkv"].dtype)
    slot = _slots(s["table"], s["seq"].long(), s["index"].long(), page)
    s["k"].view(-1, nkv, hd)[slot] = qk[:, nq:]
    s["v"].view(-1, nkv, hd)[slot] = s["qkv"][:, nq + nkv:]
    return {"q": qk[:, :nq].contiguous(), "k": s["k"], "v": s["v"]}


def _plain_reposition(s):
    case = s["case"]
    nkv, hd = case["nkv"], case["hd"]
    n, top = s["n_seqs"], s["max_len"]
    live = torch.arange(top, device="cuda")[None] < s["lens"][:, None]
    seq, j = torch.nonzero(live, as_tuple=True)
    slot = _slots(s["table"], seq, j, case["page"])
    back = (j[:, None] - s["pos_from"][seq, :, j].long()).double()              # [live positions, nkv]
    k = s["k"].view(-1, nkv, hd)
    freq, _ = _frequencies(case)
    k[slot] = _turn(k[slot].float(), back[..., None] * freq, case, 1.0).to(k.dtype)
    return {"k": s["k"]}


def _gather(s, table, lens, top, page, nkv, hd):
    """Keys [n, nkv, hd, top] and values [n, nkv, top, hd] in fp32, zeros behind a length, and which are live."""
    n = table.shape[0]
    j = torch.arange(top, device="cuda")
    live = j[None] < lens[:, None]
    slot = _slots(table, torch.arange(n, device="cuda")[:, None], j[None], page)
    k = torch.where(live[..., None, None], s["k"].view(-1, nkv, hd)[slot], 0).float().permute(0, 2, 3, 1)
    v = torch.where(live[..., None, None], s["v"].view(-1, nkv, hd)[slot], 0).float().permute(0, 2, 1, 3)
    return k, v, live


def _plain_rows(s):
    case = s["case"]
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    n, r, grp = s["n_seqs"], s["rows_top"], nq // nkv
    k, v, live = _gather(s, s["table"], s["lens"], s["max_len"], page, nkv, hd)
    at = s["starts"][:-1, None].long() + torch.arange(r, device="cuda")[None]   # [n, r]
    mine = at < s["starts"][1:, None]
    q = s["q"][torch.where(mine, at, 0)].float().view(n, r, nkv, grp, hd).permute(0, 2, 1, 3, 4).reshape(n, nkv, r * grp, hd)
    score = torch.matmul(q, k) * (1.0 / math.sqrt(hd))                          # [n, nkv, r * grp, top]
    score.masked_fill_(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1)
    lse = (top + torch.log(total))[..., 0]                                      # -inf where nothing is live
    back = lambda x, *shape: x.reshape(n, nkv, r, grp, *shape).transpose(1, 2).reshape(n, r, nq, *shape)  # noqa: E731
    s["out"][at[mine]] = back(o, hd)[mine].to(s["out"].dtype)
    kept = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float32)
    kept[at[mine]] = back(lse)[mine]
    return {"out": s["out"], "lse": kept}


def _plain_shared(s):
    case = s["case"]
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    n, groups, grp = s["n_seqs"], case["n_groups"], nq // nkv
    m = max(1, case["members"])
    scale = 1.0 / math.sqrt(hd)
    q = s["q"].float().view(n, nkv, grp, hd)
    k, v, live = _gather(s, s["table"], s["lens"], s["tail_top"], page, nkv, hd)
    tail = torch.matmul(q, k) * scale                                           # [n, nkv, grp, tail]
    tail = torch.where(live[:, None, None], tail, -math.inf)
    pk, pv, plive = _gather(s, s["prefix_table"], s["prefix_lens"], s["prefix_top"], page, nkv, hd)
    at = s["starts"][:-1, None].long() + torch.arange(m, device="cuda")[None]   # [groups, m]
    mine = at < s["starts"][1:, None]
    qg = q[torch.where(mine, at, 0)].transpose(1, 2).reshape(groups, nkv, m * grp, hd)
    pre = torch.matmul(qg, pk) * scale                                          # [groups, nkv, m * grp, prefix]
    pre = torch.where(plive[:, None, None], pre, -math.inf)
    # every sequence's row in its group's product: an empty group of none
    where = torch.zeros(n, device="cuda", dtype=torch.long)
    where[at[mine]] = torch.arange(groups * m, device="cuda").view(groups, m)[mine]
    some = torch.zeros(n, device="cuda", dtype=torch.bool)
    some[at[mine]] = True

    def rows(x):   # [groups, nkv, m * grp, d] -> [n, nkv, grp, d]
        return x.view(groups, nkv, m, grp, -1).transpose(1, 2).reshape(groups * m, nkv, grp, -1)[where]

    pre_top = torch.where(some[:, None, None, None], rows(pre.amax(-1, keepdim=True)), -math.inf)
    top = torch.maximum(tail.amax(-1, keepdim=True), pre_top)
    top = torch.where(torch.isfinite(top), top, 0)
    own_top = pre.amax(-1, keepdim=True)
    own_top = torch.where(torch.isfinite(own_top), own_top, 0)
    p = torch.exp(pre - own_top)
    weigh = torch.where(some[:, None, None, None], torch.exp(rows(own_top) - top), 0)   # 1 where the prefix leads
    weigh = torch.where(torch.isfinite(pre_top), weigh, 0)
    t = torch.exp(tail - top)
    total = t.sum(-1, keepdim=True) + weigh * rows(p.sum(-1, keepdim=True))
    o = (torch.matmul(t, v) + weigh * rows(torch.matmul(p, pv))) / torch.where(total > 0, total, 1)
    s["out"].copy_(o.view(n, nq, hd))
    return {"out": s["out"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    lens = _lens(case)
    row = nkv * hd * es
    entries = 4 * sum(-(-x // page) for x in lens)
    if case["op"] == "append":
        t = case["n_seqs"] * case["rows"]
        # each row in and out once, its three numbers and its page's entry
        return {"bytes": t * (2 * (nq * hd * es + 2 * row) + 16), "flops": t * (nq + nkv) * hd * 10}
    if case["op"] == "reposition":
        # the rotated part of every key in and out, its old position
        total = sum(lens) * nkv
        return {"bytes": total * (2 * case["rdim"] * es + 4) + entries, "flops": total * case["rdim"] * 3}
    if case["op"] == "rows":
        rows = _rows(case)
        # keys and values of the sequences that have rows, queries in and outputs and log-sums out
        read = sum(x for x, r in zip(lens, rows) if r)
        return {"bytes": 2 * read * row + sum(rows) * nq * (2 * hd * es + 4) + entries,
                "flops": 4 * sum(x * r for x, r in zip(lens, rows)) * nq * hd}
    members, prefixes = _members(case), _prefixes(case)
    read = sum(lens) + sum(x for x, m in zip(prefixes, members) if m)
    pairs = sum(lens) + sum(x * m for x, m in zip(prefixes, members))
    return {"bytes": 2 * read * row + 2 * len(lens) * nq * hd * es + entries + 4 * sum(-(-x // page) for x in prefixes),
            "flops": 4 * pairs * nq * hd}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_turns(case, steps):
    """e^(i angle) for an array of whole numbers of positions, and the factor on them."""
    d, factor, turns = case["rdim"], case["factor"], []
    for i in range(d // 2):
        base = THETA
        if case["scaling"] == "ntk":
            base = THETA * math.pow(factor, d / (d - 2))
        w = math.exp(-2 * i / d * math.log(base))
        if case["scaling"] == "linear":
            w = w / factor
        elif case["scaling"] == "bands":
            rounds = ORIGINAL * w / math.tau
            if rounds <= 1:
                w = w / factor
            elif rounds < 4:
                w = w / factor + (w - w / factor) * (rounds - 1) / 3
        elif case["scaling"] == "yarn":
            edge = [math.log(ORIGINAL / (r * math.tau)) / math.log(THETA) * d / 2 for r in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
            keep = 1 if i <= lo else 0 if i >= hi else 1 - (i - lo) / (hi - lo)
            w = w * keep + w / factor * (1 - keep)
        turns.append(w)
    m = 1 + 0.1 * math.log(factor) if case["scaling"] == "yarn" else 1.0
    phase = steps.double()[..., None] * torch.tensor(turns, dtype=torch.float64, device="cuda")
    return torch.exp(1j * phase), m


def _exact_turn(x, turns, case):
    d = case["rdim"]
    pairs = x[..., :d].unflatten(-1, (2, d // 2)).transpose(-1, -2) if case["layout"] == "half" else x[..., :d].unflatten(-1, (d // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turns)
    z = z.transpose(-1, -2) if case["layout"] == "half" else z
    return torch.cat([z.flatten(-2), x[..., d:]], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    nq, nkv, hd, page = case["nq"], case["nkv"], case["hd"], case["page"]
    lens, group = _lens(case), nq // nkv
    tables = {t: s[t].cpu().numpy() for t in ("table", "prefix_table") if t in s}

    def places(t, i, idx):
        idx = np.asarray(idx, np.int64)
        return torch.from_numpy(tables[t][i, idx // page].astype(np.int64) * page + idx % page).cuda()

    k, v = s["k"].view(-1, nkv, hd), s["v"].view(-1, nkv, hd)
    if case["op"] == "append":
        q_out = torch.empty((s["qkv"].shape[0], nq, hd), dtype=torch.float64, device="cuda")
        k, v = k.double(), v.double()
        for i in range(case["n_seqs"]):
            at = slice(i * case["rows"], (i + 1) * case["rows"])
            x = s["qkv"][at].double()
            turns, m = _exact_turns(case, s["pos"][at])
            parts = []
            for y, gain in ((x[:, :nq], s.get("q_gain")), (x[:, nq:nq + nkv], s.get("k_gain"))):
                if gain is not None:
                    y = y * gain.double() * torch.rsqrt((y * y).sum(-1, keepdim=True) / hd + EPS)
                parts.append(_exact_turn(y, m * turns[:, None], case))
            to = places("table", i, s["index"][at].cpu().numpy())
            q_out[at] = parts[0]
            k[to], v[to] = parts[1], x[:, nq + nkv:]
        return {"q": q_out, "k": k.view_as(s["k"]), "v": v.view_as(s["v"])}
    if case["op"] == "reposition":
        k = k.double()
        for i, x in enumerate(lens):
            if x:
                at = places("table", i, np.arange(x))
                for h in range(nkv):
                    steps = torch.arange(x, device="cuda") - s["pos_from"][i, h, :x]
                    k[at, h] = _exact_turn(k[at, h], _exact_turns(case, steps)[0], case)
        return {"k": k.view_as(s["k"])}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")

    def attend(q, at):   # [rows, nq, hd] over the positions `at` of the pools -> output, log-sums
        o, sums = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for h in range(nkv if len(at) else 0):
            heads = slice(h * group, (h + 1) * group)
            x = torch.einsum("rgd,jd->rgj", q[:, heads], k[at, h].double()) / math.sqrt(hd)
            sums[:, heads] = torch.logsumexp(x, -1)
            o[:, heads] = torch.softmax(x, -1) @ v[at, h].double()
        return o, sums

    if case["op"] == "rows":
        if work(case)["flops"] > 2e12:
            return None
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        starts = _offsets(_rows(case))
        for i, x in enumerate(lens):
            for a in range(starts[i], starts[i + 1], 128):   # so many rows at a time
                at = slice(a, min(a + 128, starts[i + 1]))
                out[at], lse[at] = attend(s["q"][at].double(), places("table", i, np.arange(x)))
        return {"out": out, "lse": lse}
    members, prefixes, i = _members(case), _prefixes(case), 0
    for g, m in enumerate(members):
        shared = places("prefix_table", g, np.arange(prefixes[g])) if g < len(prefixes) else places("table", 0, [])
        for _ in range(m):
            out[i] = attend(s["q"][i:i + 1].double(), torch.cat([shared, places("table", i, np.arange(lens[i]))]))[0][0]
            i += 1
    return {"out": out}
