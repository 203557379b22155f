"""Attention of blocks of rows and of batches that share prefixes, over the
paged cache, against float64 (needs a GB300).

Tolerances as for the attention of one token (u = 2^-24, e the half step of the
output type): a score is off by d = (HD + 4) 2u sum_d |q_d k_d| |scale|, the sums
over len keys by 2 (len + 64) 2u, the exponential by 8u, and softmax weights
enter a bf16 product rounded to bf16 (2^-8, half a step) or as the sum of two
bf16 numbers (2^-16):
    r = 2 d + 2 (len + 64) 2u + 8u + (2^-8 in bf16, 0 in fp32)
    out:  r sum_j p_j |v_j| (1 + e) + e |ref|
    lse:  d + 2 (len + 64) 2u + 8u, and 4u of the largest score and of itself in
          log2 units (with 27 added and taken off again): 8u (|top| + |lse| + 30).
A prefix and a tail joined add a few products each: the 64 covers them."""
import numpy as np
import pytest
import torch

from test_gpu_cache import DT, E, U, blank_behind, i32, make_pages, pool, sf  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (10, 5, 128)]


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def check(a, what, q, out, lse, slots, scale, dtype):
    """One set of rows q [R, nq, hd] over the positions in `slots` of the pools."""
    R, nq, hd = q.shape
    nkv = a["k"].shape[2]
    G, e, n = nq // nkv, E[dtype], len(slots)
    if n == 0:
        assert not out.any() and (lse is None or torch.all(lse == -torch.inf)), what
        return
    slots = torch.as_tensor(slots, device="cuda")
    for c in range(nkv):
        h = slice(c * G, (c + 1) * G)
        k, v = (a[x].view(-1, nkv, hd)[slots, c].double() for x in ("k", "v"))
        x = q[:, h].double().reshape(R * G, hd)
        s = x @ k.T * scale
        d = (hd + 4) * 2 * U * abs(scale) * (x.abs() @ k.abs().T).amax(1)
        p = torch.softmax(s, 1)
        ref, mag = p @ v, p @ v.abs()
        r = 2 * d + 4 * (n + 64) * U + 8 * U + (2.0 ** -8 if dtype == "bf16" else 0.0)
        tol = r[:, None] * mag * (1 + e) + e * ref.abs()
        off = (out[:, h].double().reshape(R * G, hd) - ref).abs()
        assert torch.all(off <= tol), (what, c, float((off / tol).max()), int((off > tol).sum()))
        if lse is not None:
            want = torch.logsumexp(s, 1)
            top = s.abs().amax(1)
            tol = d + 4 * (n + 64) * U + 8 * U + 8 * U * (top + want.abs() + 30)
            off = (lse[:, h].double().reshape(R * G) - want).abs()
            assert torch.all(off <= tol), (what, c, float((off / tol).max()))


def places(table, s, n, page):
    j = np.arange(n)
    return table[s, j // page].astype(np.int64) * page + j % page


def rows_inputs(sf, heads, dtype, page, rows, lens, seed=0, front=0, behind=3, cols=None, q_std=2.0, max_len=None):
    nq, nkv, hd = heads
    rng = np.random.default_rng([seed, page, sum(lens), sum(rows)])
    table, total = make_pages(rng, lens, page, cols=cols)
    k, v = (pool(rng, total, page, nkv, hd, dtype) for _ in range(2))
    blank_behind(k, table, lens, page, float("nan"))
    blank_behind(v, table, lens, page, float("inf"))
    T = front + sum(rows) + behind
    q = (torch.from_numpy(rng.standard_normal((T, nq, hd)).astype(np.float32)) * q_std).cuda().to(DT[dtype])
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(lens),
                      max_len=max_len or max(1, max(lens)), max_rows=max(T, 1))
    return dict(c=c, rng=rng, table=table, k=k, v=v, q=q, starts=offsets(rows) + front, lens=lens, rows=rows, page=page)


def run_rows(a, **kw):
    out, lse = torch.full_like(a["q"], 7.0), torch.full(a["q"].shape[:2], 7.0, device="cuda")
    a["c"].attend_rows(a["q"], a["k"], a["v"], i32(a["table"]), i32(a["lens"]), i32(a["starts"]), out=out, lse=lse, **kw)
    return out, lse


def check_rows(a, out, lse, dtype, scale=None, seqs=None):
    scale = a["q"].shape[2] ** -0.5 if scale is None else scale
    st = a["starts"]
    for s, n in enumerate(a["lens"]):
        if seqs is None or s in seqs:
            at = slice(int(st[s]), int(st[s + 1]))
            if at.stop > at.start:
                check(a, s, a["q"][at], out[at], None if lse is None else lse[at], places(a["table"], s, n, a["page"]),
                      scale, dtype)
    for at in (slice(0, int(st[0])), slice(int(st[-1]), None)):      # rows of no sequence: as they were
        assert torch.all(out[at] == 7.0) and (lse is None or torch.all(lse[at] == 7.0))


ROWS = [
    # heads, dtype, page, rows, lens
    ((4, 2, 64), "f32", 16, [1], [1]),
    ((4, 2, 64), "f32", 24, [5, 0, 1, 33, 64], [0, 7, 1, 130, 333]),
    ((12, 2, 128), "f32", 7, [3, 20], [129, 64]),
    ((10, 5, 128), "f32", 1, [31, 5], [31, 5]),
    ((3, 1, 64), "f32", 32, [100], [1000]),
    ((16, 1, 128), "f32", 64, [9, 1, 70], [100, 260, 63]),
    ((8, 8, 64), "f32", 100, [65, 1], [20, 4000]),
    ((12, 2, 128), "bf16", 32, [1], [1]),
    ((12, 2, 128), "bf16", 32, [32], [512]),
    ((4, 2, 64), "bf16", 5, [1, 64, 0, 65, 2, 128, 129], [127, 128, 129, 0, 1, 255, 700]),
    ((28, 4, 128), "bf16", 16, [18, 19, 37, 1], [2047, 1, 64, 0]),
    ((40, 8, 128), "bf16", 100, [25, 26, 51, 52, 103], [255, 256, 257, 1, 384]),
    ((8, 8, 64), "bf16", 1, [127, 257, 3], [63, 200, 3]),
    ((6, 6, 128), "bf16", 24, [513], [77]),
    ((16, 1, 128), "bf16", 48, [8, 9, 33], [1500, 9, 129]),
    ((21, 1, 64), "bf16", 16, [90, 6], [90, 513]),
    ((80, 2, 128), "bf16", 16, [7, 3], [70, 1]),
    ((7, 7, 128), "bf16", 65536, [200], [300]),
    ((32, 8, 128), "bf16", 64, [3, 300], [20000, 130]),
    ((14, 2, 64), "bf16", 16, [4], [40000]),
    ((1, 1, 128), "bf16", 8, [129, 128, 127], [129, 128, 127]),
    ((1024, 1, 64), "bf16", 16, [1, 2], [40, 100]),
]


@pytest.mark.parametrize("heads,dtype,page,rows,lens", ROWS)
def test_rows(sf, heads, dtype, page, rows, lens):
    a = rows_inputs(sf, heads, dtype, page, rows, lens, front=2)
    out, lse = run_rows(a)
    a["c"].sync()
    check_rows(a, out, lse, dtype)
    for _ in range(3):                                               # the same bits again
        o2, l2 = run_rows(a)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    o2 = torch.full_like(out, 7.0)                                   # without log-sums too
    a["c"].attend_rows(a["q"], a["k"], a["v"], i32(a["table"]), i32(a["lens"]), i32(a["starts"]), out=o2)
    assert torch.equal(o2, out)
    a["c"].close()


@pytest.mark.parametrize("seed", range(24))
def test_rows_random_batches(sf, seed):
    rng = np.random.default_rng(1000 + seed)
    heads, dtype = HEADS[rng.integers(len(HEADS))], "f32" if seed % 4 == 3 else "bf16"
    S = int(rng.choice([1, 2, 3, 7, 40, 400]))
    top_r, top_l = int(rng.choice([1, 5, 60, 400])), int(rng.choice([1, 30, 300, 3000]))
    if S == 400:
        top_r, top_l = min(top_r, 5), min(top_l, 300)
    if dtype == "f32":
        top_r = min(top_r, 60)
    rows = (rng.integers(0, top_r + 1, S) * (rng.random(S) < 0.8)).tolist()
    lens = (rng.integers(0, top_l + 1, S) * (rng.random(S) < 0.8)).tolist()
    a = rows_inputs(sf, heads, dtype, int(rng.choice([1, 8, 16, 24, 100])), rows, lens, seed=seed, front=seed % 3)
    out, lse = run_rows(a)
    a["c"].sync()
    check_rows(a, out, lse, dtype)
    a["c"].close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0, 1e-30])
def test_rows_strided_and_scaled(sf, dtype, scale):
    """Rows of a wider projection, an output of other strides, a table with columns to spare, any scale."""
    a = rows_inputs(sf, (12, 2, 128), dtype, 16, [40, 3], [200, 300], cols=33)
    T = a["q"].shape[0]
    wide = torch.randn((T, 12 * 128 + 256), device="cuda").to(DT[dtype])
    a["q"] = wide[:, 128:128 + 12 * 128].view(T, 12, 128)
    out = torch.full((T, 13, 128), 7.0, device="cuda", dtype=DT[dtype])
    lse = torch.full((T, 12), 7.0, device="cuda")
    got = a["c"].attend_rows(wide[:, 128:128 + 12 * 128], a["k"], a["v"], i32(a["table"]), i32(a["lens"]),
                             i32(a["starts"]), scale=scale, out=out[:, :12], lse=lse)
    a["c"].sync()
    check_rows(a, got, lse, dtype, scale=scale)
    assert torch.all(out[:, 12] == 7.0)
    a["c"].close()


def values_of(a, s, rows):
    """Write rows {position: (k or None, v or None)} into sequence s of the pools, all KV heads."""
    for j, (k, v) in rows.items():
        page, at = int(a["table"][s, j // a["page"]]), j % a["page"]
        if k is not None:
            a["k"][page, at] = k
        if v is not None:
            a["v"][page, at] = v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 90])
def test_rows_extreme_values(sf, dtype, rows):
    """Large scores stay finite; scores of -infinity weigh nothing, rows without any other get zeros; NaN and infinite
    values reach exactly the rows that see them; largest values do not overflow in unnormalised sums."""
    heads = (4, 2, 64)
    a = rows_inputs(sf, heads, dtype, 16, [rows, rows, rows, rows], [300, 300, 300, 200], q_std=60.0)
    a["q"].clamp_(min=0.5)                                           # all positive: -inf keys give -inf scores
    # 0: large scores of both signs; 1: some keys at -infinity; 2: all of them; 3: a NaN value of head 1
    values_of(a, 0, {5: (40.0, None), 299: (-40.0, None)})
    values_of(a, 1, {j: (-torch.inf, None) for j in range(0, 300, 3)})
    values_of(a, 2, {j: (-torch.inf, None) for j in range(300)})
    page = int(a["table"][3, 0])
    a["v"][page, 3, 1, 7] = torch.nan
    out, lse = run_rows(a)
    a["c"].sync()
    check_rows(a, out, lse, dtype, seqs=[0])
    st = a["starts"]
    one = slice(int(st[1]), int(st[2]))
    keep = np.array([j for j in range(300) if j % 3])
    check(a, 1, a["q"][one], out[one], lse[one], places(a["table"], 1, 300, 16)[keep], 64 ** -0.5, dtype)
    two = slice(int(st[2]), int(st[3]))
    assert not out[two].any() and torch.all(lse[two] == -torch.inf)
    three = slice(int(st[3]), int(st[4]))
    bad = torch.isnan(out[three])
    want = torch.zeros_like(bad)
    want[:, 2:, 7] = True                                            # query heads of KV head 1
    assert torch.equal(bad, want)
    # a NaN key and one that scores +infinity: the heads that see them are not finite
    a["v"][page, 3, 1, 7] = 0.0
    a["k"][page, 3, 1, 0] = torch.nan
    a["k"][int(a["table"][0, 1]), 2, 0] = torch.inf
    out, lse = run_rows(a)
    a["c"].sync()
    assert not torch.isfinite(out[three][:, 2:]).any() and torch.isfinite(out[three][:, :2]).all()
    zero = slice(int(st[0]), int(st[1]))
    assert not torch.isfinite(out[zero][:, :2]).any() and torch.isfinite(out[zero][:, 2:]).all()
    # equal scores and the type's largest values: their mean
    big = torch.finfo(DT[dtype]).max
    a["q"].zero_()
    values_of(a, 0, {j: (1.0, big) for j in range(300)})
    out, lse = run_rows(a)
    assert torch.isfinite(out[zero]).all() and torch.all(out[zero].double() >= big * (1 - 2 * E[dtype]))
    a["c"].close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_growing_scores(sf, dtype):
    """The running maximum grows with every key, and falls."""
    for sign in (1, -1):
        a = rows_inputs(sf, (2, 1, 128), dtype, 16, [200, 5], [900, 1300], q_std=0.0)
        a["q"].fill_(1.0)
        for s in range(2):
            n = a["lens"][s]
            ramp = sign * torch.linspace(-6, 6, n, device="cuda")
            at = torch.as_tensor(places(a["table"], s, n, 16), device="cuda")
            a["k"].view(-1, 128)[at] = ramp[:, None].expand(n, 128).to(DT[dtype])
        out, lse = run_rows(a)
        a["c"].sync()
        check_rows(a, out, lse, dtype)
        a["c"].close()


def test_rows_share_pages_and_long_pools(sf):
    """The same pages in several sequences, one of them several times in a row; slots past 2^31 elements."""
    heads, page = (8, 8, 64), 64
    rng = np.random.default_rng(5)
    n_pages = 2 ** 31 // (page * 512) + 40
    k, v = (torch.zeros((n_pages, page, 8, 64), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    used = [0, n_pages - 1, n_pages - 2, 17]
    for p in used:
        for t in (k, v):
            t[p] = torch.from_numpy(rng.standard_normal((page, 8, 64))).cuda().to(torch.bfloat16)
    table = np.array([[used[0], used[1], used[1]], [used[1], used[2], used[3]], [used[3], used[3], used[0]]], np.int32)
    a = rows_inputs(sf, heads, "bf16", page, [20, 150, 1], [190, 192, 65])
    a.update(k=k, v=v, table=table)
    out, lse = run_rows(a)
    a["c"].sync()
    check_rows(a, out, lse, "bf16")
    a["c"].close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 4, 7, 8, 16, 17])
def test_rows_smallest_pools(sf, dtype, page):
    """A pool of one page: fewer positions than a load takes together."""
    for n in {1, page}:
        a = rows_inputs(sf, (4, 2, 64), dtype, page, [1, 70], [n, 0])
        a["k"], a["v"] = (a[x][int(a["table"][0, 0])][None].contiguous() for x in ("k", "v"))
        a["table"] = np.zeros_like(a["table"])
        a["lens"] = [n, n]
        out, lse = run_rows(a)
        a["c"].sync()
        check_rows(a, out, lse, dtype)
        a["c"].close()


def test_rows_largest_call(sf):
    """1,048,576 rows: queries and outputs past 2^31 elements."""
    rows = [5, 2 ** 20 - 105, 100]
    a = rows_inputs(sf, (33, 3, 64), "bf16", 16, [1, 1, 1], [70, 33, 200], behind=0)
    a["c"].close()
    T = sum(rows)
    a["q"] = torch.randn((T, 33, 64), device="cuda", dtype=torch.bfloat16)
    a["starts"] = offsets(rows)
    a["c"] = sf.PagedCache(n_q_heads=33, n_kv_heads=3, head_dim=64, dtype="bf16", page_size=16, max_seqs=3, max_len=200,
                           max_rows=T)
    out, lse = run_rows(a)
    a["c"].sync()
    for s, at in ((0, 0), (1, 5), (1, 500000), (1, T - 100 - 64), (2, T - 100), (2, T - 36)):
        at = slice(at, at + (5 if s == 0 else 36))
        check(a, (s, at), a["q"][at], out[at], lse[at], places(a["table"], s, a["lens"][s], 16), 64 ** -0.5, "bf16")
    a["c"].close()
    with pytest.raises(sf.SpecFoldError) as e:
        sf.PagedCache(n_q_heads=33, n_kv_heads=3, head_dim=64, dtype="bf16", page_size=16, max_seqs=3, max_len=200,
                      max_rows=T + 1)
    assert e.value.status == sf.SF_ERR_UNSUPPORTED


def test_rows_report_bad_lengths_pages_and_starts(sf):
    heads, page = (12, 2, 128), 16
    a = rows_inputs(sf, heads, "bf16", page, [30, 40, 5], [100, 50, 70])
    good, glse = run_rows(a)
    a["c"].sync()

    def reported(text):
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and text in str(e.value)
        a["c"].sync()

    one = slice(30, 70)
    for bad in (-1, 101, 2 ** 31 - 1, -2 ** 31):
        lens = list(a["lens"])
        lens[1] = bad
        out, lse = run_rows(dict(a, lens=lens))
        reported("length")
        assert not out[one].any() and torch.all(lse[one] == -torch.inf)
        check_rows(a, out, lse, "bf16", seqs=[0, 2])
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        table = a["table"].copy()
        table[1, 1] = bad
        out, lse = run_rows(dict(a, table=table))
        reported("page")
        check_rows(a, out, lse, "bf16", seqs=[0, 2])
        keep = np.r_[0:16, 32:50]
        check(a, "kept", a["q"][one], out[one], lse[one], places(a["table"], 1, 50, page)[keep], 128 ** -0.5, "bf16")
    out, lse = run_rows(dict(a, table=np.full_like(a["table"], -7)))
    reported("page")
    assert not out[:75].any() and torch.all(lse[:75] == -torch.inf)
    for bad in ([-1, 30, 70, 75], [0, 30, 29, 75], [0, 30, 70, 79], [0, 2 ** 31 - 1, 70, 75], [5, 4, 70, 75]):
        out, lse = run_rows(dict(a, starts=np.array(bad, np.int32)))
        reported("row")
        assert torch.all(out == 7.0) and torch.all(lse == 7.0)
    out, lse = run_rows(a)
    a["c"].sync()
    assert torch.equal(out, good) and torch.equal(lse, glse)
    a["c"].close()


def test_rows_in_graphs_and_on_streams(sf):
    """Captured, replayed with other lengths, offsets and pages; on a side stream; two objects at once."""
    heads, page = (12, 2, 128), 16
    a = rows_inputs(sf, heads, "bf16", page, [30, 200, 5], [400, 700, 90])
    b = rows_inputs(sf, heads, "bf16", page, [200, 30, 5], [90, 400, 700])
    lens, starts, table = i32(a["lens"]), i32(a["starts"]), i32(np.pad(a["table"], ((0, 0), (0, 8))))
    out, lse = torch.zeros_like(a["q"]), torch.zeros(a["q"].shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a["c"].attend_rows(a["q"], a["k"], a["v"], table, lens, starts, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    want, wlse = run_rows(a)
    assert torch.equal(out[:235], want[:235]) and torch.equal(lse[:235], wlse[:235])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a["c"].attend_rows(a["q"], a["k"], a["v"], table, lens, starts, out=out, lse=lse)
    for rows, n in (([30, 200, 5], [400, 700, 90]), ([0, 235, 0], [0, 700, 1]), ([100, 100, 35], [0, 5, 90])):
        starts.copy_(i32(offsets(rows)))
        lens.copy_(i32(n))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        check_rows(dict(a, lens=n, starts=offsets(rows)), out, lse, "bf16")
    a["c"].sync()
    # two objects, two streams, many calls
    other = torch.cuda.Stream()
    ref_b, _ = run_rows(b)
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        with torch.cuda.stream(side):
            x = run_rows(a)[0]
        with torch.cuda.stream(other):
            y = run_rows(b)[0]
        outs.append((x, y))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, want) and torch.equal(y, ref_b)
    a["c"].close()
    b["c"].close()


# ---------------------------------------------------------------- shared prefixes

SHARED = [
    # heads, dtype, page, members, prefixes, sequences in front and behind, tails
    ((4, 2, 64), "f32", 16, [1], [1], 0, 0, [0]),
    ((4, 2, 64), "f32", 24, [3, 0, 2], [100, 50, 0], 1, 2, [0, 1, 2, 33, 0, 7, 0, 64]),
    ((12, 2, 128), "f32", 7, [9], [200], 0, 0, [1, 2, 3, 4, 5, 6, 7, 0, 30]),
    ((12, 2, 128), "bf16", 32, [9], [512], 0, 0, [32] * 9),
    ((40, 8, 128), "bf16", 16, [9, 1, 30], [1000, 77, 300], 0, 0, list(range(40))),
    ((32, 8, 128), "bf16", 100, [70], [4000], 2, 3, [17] * 75),
    ((4, 2, 64), "bf16", 5, [65, 64, 0, 1], [129, 128, 5, 0], 1, 1, [3] * 132),
    ((8, 8, 64), "bf16", 1, [130, 5], [300, 1], 0, 0, [0, 1] * 67 + [90]),
    ((16, 1, 128), "bf16", 48, [17, 16], [1500, 20000], 0, 1, [50] * 33 + [0]),
    ((28, 4, 128), "bf16", 16, [2, 2], [0, 0], 0, 0, [0, 9, 300, 0]),
    ((7, 7, 128), "bf16", 24, [300], [40], 0, 0, [1] * 300),
    ((12, 2, 128), "bf16", 16, [0, 1, 0, 0, 1, 0, 0], [9, 300, 0, 4, 129, 1, 2], 0, 0, [3, 0]),
    ((4, 2, 64), "f32", 16, [1] + [0] * 400, [70] * 401, 0, 0, [3]),
    ((32, 8, 128), "bf16", 16, [40], [100], 0, 0, list(range(0, 1600, 40))),
    ((4, 2, 64), "bf16", 16, [3], [50], 0, 0, [5000, 1, 300]),
]


def shared_inputs(sf, heads, dtype, page, members, prefixes, front, behind, tails, seed=0):
    nq, nkv, hd = heads
    S = front + sum(members) + behind
    assert S == len(tails)
    rng = np.random.default_rng([seed, page, S])
    both, total = make_pages(rng, list(tails) + list(prefixes), page)
    k, v = (pool(rng, total, page, nkv, hd, dtype) for _ in range(2))
    blank_behind(k, both, list(tails) + list(prefixes), page, float("nan"))
    blank_behind(v, both, list(tails) + list(prefixes), page, float("inf"))
    q = (torch.from_numpy(rng.standard_normal((S, nq, hd)).astype(np.float32)) * 2).cuda().to(DT[dtype])
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=S,
                      max_len=max(1, max(tails), max(prefixes)), max_rows=S)
    return dict(c=c, k=k, v=v, q=q, table=both[:S], ptable=both[S:], starts=offsets(members) + front, lens=list(tails),
                plens=list(prefixes), page=page, members=members)


def run_shared(a, **kw):
    out, lse = torch.full_like(a["q"], 7.0), torch.full(a["q"].shape[:2], 7.0, device="cuda")
    a["c"].attend_shared(a["q"], a["k"], a["v"], i32(a["table"]), i32(a["lens"]), i32(a["ptable"]), i32(a["plens"]),
                         i32(a["starts"]), out=out, lse=lse, **kw)
    return out, lse


def check_shared(a, out, lse, dtype, scale=None):
    scale = a["q"].shape[2] ** -0.5 if scale is None else scale
    st = a["starts"]
    for s, n in enumerate(a["lens"]):
        g = int(np.searchsorted(st, s, side="right")) - 1
        pre = places(a["ptable"], g, a["plens"][g], a["page"]) if 0 <= g < len(a["plens"]) else np.zeros(0, np.int64)
        check(a, s, a["q"][s:s + 1], out[s:s + 1], lse[s:s + 1], np.r_[pre, places(a["table"], s, n, a["page"])], scale,
              dtype)


@pytest.mark.parametrize("heads,dtype,page,members,prefixes,front,behind,tails", SHARED)
def test_shared(sf, heads, dtype, page, members, prefixes, front, behind, tails):
    a = shared_inputs(sf, heads, dtype, page, members, prefixes, front, behind, tails)
    out, lse = run_shared(a)
    a["c"].sync()
    check_shared(a, out, lse, dtype)
    o2, l2 = run_shared(a)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    out, lse = run_shared(a, scale=-0.2)
    check_shared(a, out, lse, dtype, scale=-0.2)
    a["c"].close()


@pytest.mark.parametrize("seed", range(12))
def test_shared_random_batches(sf, seed):
    rng = np.random.default_rng(2000 + seed)
    heads, dtype = HEADS[rng.integers(len(HEADS))], "f32" if seed % 4 == 3 else "bf16"
    G = int(rng.choice([1, 2, 5, 40]))
    members = rng.integers(0, int(rng.choice([2, 12, 90])) // (1 + G // 10) + 1, G).tolist()
    prefixes = (rng.integers(0, int(rng.choice([10, 300, 5000])) + 1, G) * (rng.random(G) < 0.8)).tolist()
    front, behind = int(rng.integers(0, 3)), int(rng.integers(1, 3))
    S = front + sum(members) + behind
    tails = (rng.integers(0, int(rng.choice([2, 50, 700])) + 1, S) * (rng.random(S) < 0.8)).tolist()
    a = shared_inputs(sf, heads, dtype, int(rng.choice([1, 8, 16, 100])), members, prefixes, front, behind, tails, seed)
    out, lse = run_shared(a)
    a["c"].sync()
    check_shared(a, out, lse, dtype)
    a["c"].close()


def test_shared_equals_one_table(sf):
    """A prefix in the group's table, or the same pages in every sequence's own: the same attention."""
    heads, page = (12, 2, 128), 16
    a = shared_inputs(sf, heads, "bf16", page, [6, 4], [160, 320], 0, 0, [5, 16, 17, 40, 1, 0, 3, 33, 64, 9])
    out, lse = run_shared(a)
    cols = [10] * 6 + [20] * 4
    table = np.full((10, 24), -1, np.int32)
    for s in range(10):
        row = np.r_[a["ptable"][0 if s < 6 else 1, :cols[s]], a["table"][s, :-(-a["lens"][s] // page)]]
        table[s, :len(row)] = row
    lens = [n + page * c for n, c in zip(a["lens"], cols)]
    c = sf.PagedCache(n_q_heads=12, n_kv_heads=2, head_dim=128, dtype="bf16", page_size=page, max_seqs=10, max_len=400)
    one = c.attend(a["q"], a["k"], a["v"], i32(table), i32(lens))
    c.sync()
    a["c"].sync()
    check_shared(a, out, lse, "bf16")
    check_shared(a, one, lse, "bf16")                    # both within the bound of the same exact value
    a["c"].close()
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_extreme_values(sf, dtype):
    """Prefix or tail at -infinity, or far below the other; NaN stays with the sequences that see it."""
    a = shared_inputs(sf, (4, 2, 64), dtype, 16, [3, 3, 3], [40, 40, 40], 0, 0, [20] * 9)
    a["q"].abs_().clamp_(min=0.5)
    minus = -torch.inf

    def fill(table, s, n, value, pool="k"):
        for j in range(n):
            a[pool][int(table[s, j // 16]), j % 16] = value

    fill(a["ptable"], 0, 40, minus)                     # group 0: nothing from the prefix
    for s in (3, 4, 5):
        fill(a["table"], s, 20, minus)                  # group 1: nothing from the tails
    fill(a["ptable"], 2, 40, 30.0)                      # group 2: the prefix far above the tails
    out, lse = run_shared(a)
    a["c"].sync()
    sc = 64 ** -0.5
    for s in range(9):
        pre = [] if s < 3 else places(a["ptable"], s // 3, 40, 16)
        tail = [] if 3 <= s < 6 else places(a["table"], s, 20, 16)
        check(a, s, a["q"][s:s + 1], out[s:s + 1], lse[s:s + 1], np.r_[pre, tail].astype(np.int64), sc, dtype)
    for s in (0, 1, 2):
        fill(a["table"], s, 20, minus)                  # neither
    a["k"][int(a["ptable"][1, 0]), 3] = torch.nan       # a prefix key: its whole group
    a["k"][int(a["table"][7, 0]), 0] = torch.nan        # a tail's: one sequence
    out, lse = run_shared(a)
    a["c"].sync()
    assert not out[:3].any() and torch.all(lse[:3] == minus)
    assert not torch.isfinite(out[3:6]).any() and not torch.isfinite(out[7]).any()
    assert torch.isfinite(out[6]).all() and torch.isfinite(out[8]).all()
    a["c"].close()


def test_shared_reports(sf):
    heads, page = (12, 2, 128), 16
    a = shared_inputs(sf, heads, "bf16", page, [4, 3], [100, 60], 0, 1, [9] * 8)
    good, glse = run_shared(a)
    a["c"].sync()

    def reported(text):
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and text in str(e.value)

    out, lse = run_shared(dict(a, plens=[-1, 60]))
    reported("length")                                  # counts as an empty prefix
    check_shared(dict(a, plens=[0, 60]), out, lse, "bf16")
    out, lse = run_shared(dict(a, lens=[9, 101] + [9] * 6))
    reported("length")
    check_shared(dict(a, lens=[9, 0] + [9] * 6), out, lse, "bf16")
    table = a["ptable"].copy()
    table[1, 3] = 2 ** 30
    out, lse = run_shared(dict(a, ptable=table))
    reported("page")
    check_shared(dict(a, plens=[100, 48]), out, lse, "bf16")
    for bad in ([0, 5, 4], [-1, 4, 7], [0, 4, 9]):
        out, lse = run_shared(dict(a, starts=np.array(bad, np.int32)))
        reported("row")
        assert torch.all(out == 7.0) and torch.all(lse == 7.0)
    out, lse = run_shared(a)
    a["c"].sync()
    assert torch.equal(out, good) and torch.equal(lse, glse)
    a["c"].close()


def test_shared_in_graphs(sf):
    """A decode step of appended tokens and shared prefixes, captured and replayed."""
    heads, page = (12, 2, 128), 16
    a = shared_inputs(sf, heads, "bf16", page, [5, 4], [300, 200], 0, 0, [30] * 9)
    table, ptable, starts = i32(a["table"]), i32(a["ptable"]), i32(a["starts"])
    lens, plens = i32([1] * 9), i32(a["plens"])
    index = torch.zeros(9, dtype=torch.int32, device="cuda")
    qkv = torch.empty((9, 16, 128), dtype=torch.bfloat16, device="cuda")
    q, out = torch.empty_like(a["q"]), torch.empty_like(a["q"])
    lse = torch.empty(a["q"].shape[:2], device="cuda")
    gen = torch.Generator("cuda")
    gen.manual_seed(3)
    g = torch.cuda.CUDAGraph()

    def step():
        a["c"].append(qkv, index, table, a["k"], a["v"], q=q)
        torch.add(index, 1, out=lens)
        a["c"].attend_shared(q, a["k"], a["v"], table, lens, ptable, plens, starts, out=out, lse=lse)

    qkv.normal_(generator=gen)
    step()
    with torch.cuda.graph(g):
        step()
    for i in range(30):
        qkv.normal_(generator=gen)
        index.fill_(i)
        g.replay()
        if i % 7 == 0:
            check_shared(dict(a, q=q, lens=[i + 1] * 9), out, lse, "bf16")
    a["c"].sync()
    a["c"].close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_largest_batches(sf, dtype):
    """As many sequences and groups as an object takes: most groups empty, most prefixes unused."""
    S, G = 4096, 65536
    rng = np.random.default_rng(11)
    members = np.zeros(G, np.int64)
    members[np.sort(rng.choice(G, 300, replace=False))] = 13
    members[-1] = S - 3 - members[:-1].sum()
    used = np.flatnonzero(members)
    prefixes = rng.integers(0, 60, G)
    tails = rng.integers(0, 20, S)
    a = shared_inputs(sf, (4, 2, 64), dtype, 16, members[used].tolist(), prefixes[used].tolist(), 1, 2, tails.tolist())
    wide = np.full((G, a["ptable"].shape[1]), -1, np.int32)              # groups of none: pages never looked at
    wide[used] = a["ptable"]
    prefixes[members == 0] = np.minimum(prefixes[members == 0], a["c"].shapes.max_len)
    a.update(ptable=wide, plens=prefixes.tolist(), starts=offsets(members) + 1)
    out, lse = run_shared(a)
    a["c"].sync()
    some = np.r_[0, 1, 2, np.arange(13, 4096, 97), 4093, 4094, 4095]
    group = np.searchsorted(a["starts"], np.arange(S), side="right") - 1
    for s in some:
        g = group[s]
        pre = places(wide, g, int(prefixes[g]), 16) if 0 <= g < G else np.zeros(0, np.int64)
        check(a, s, a["q"][s:s + 1], out[s:s + 1], lse[s:s + 1], np.r_[pre, places(a["table"], s, int(tails[s]), 16)],
              64 ** -0.5, dtype)
    assert torch.isfinite(out).all()
    a["c"].close()


def test_shared_beside_other_calls(sf):
    """Two objects on two streams at once, and calls of one object that share its workspace one after another."""
    a = shared_inputs(sf, (12, 2, 128), "bf16", 16, [5, 4], [900, 200], 1, 0, [30] * 9 + [2000])
    b = shared_inputs(sf, (8, 8, 64), "bf16", 16, [70], [300], 0, 0, [9] * 70)
    want = [run_shared(x) for x in (a, b)]
    one = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(a["lens"]))
    rows = a["c"].attend_rows(a["q"], a["k"], a["v"], i32(a["ptable"]), i32(a["plens"]), i32(a["starts"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            x = run_shared(a)
            y = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(a["lens"]))
            z = a["c"].attend_rows(a["q"], a["k"], a["v"], i32(a["ptable"]), i32(a["plens"]), i32(a["starts"]))
            w = run_shared(a)
        with torch.cuda.stream(streams[1]):
            got.append((x, y, z, w, run_shared(b), run_shared(b)))
    torch.cuda.synchronize()
    members = slice(int(a["starts"][0]), int(a["starts"][-1]))
    for x, y, z, w, u, v in got:
        for p, q in ((x, want[0]), (w, want[0]), (u, want[1]), (v, want[1])):
            assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
        assert torch.equal(y, one) and torch.equal(z[members], rows[members])
    for x in (a, b):
        x["c"].sync()
        x["c"].close()


def test_many_calls_in_a_row(sf):
    """Calls that follow one another without a wait, on inputs in turn: the same bits every time, no wait that runs
    out (tiles of one half with odd and even numbers of blocks, cut and whole)."""
    heads, page = (40, 8, 128), 32
    cases = [shared_inputs(sf, heads, "bf16", page, [9] * 4, [4096, 640, 129, 1000], 0, 0, [32] * 36, seed=s) for s in range(3)]
    more = [rows_inputs(sf, (12, 2, 128), "bf16", page, [3, 30, 1, 9], [700, 129, 3000, 257], seed=s) for s in range(3)]
    want = [run_shared(a)[0] for a in cases] + [run_rows(a)[0] for a in more]
    for a in cases + more:
        a["c"].sync()
    args = [[i32(a[x]) for x in ("table", "lens", "ptable", "plens", "starts")] for a in cases]
    rargs = [[i32(a[x]) for x in ("table", "lens", "starts")] for a in more]
    outs = [torch.empty_like(a["q"]) for a in cases] + [torch.full_like(a["q"], 7.0) for a in more]
    for i in range(300):
        j = i % 3
        a, (t, n, pt, pn, st) = cases[j], args[j]
        a["c"].attend_shared(a["q"], a["k"], a["v"], t, n, pt, pn, st, out=outs[j])
        a, (t, n, st) = more[j], rargs[j]
        a["c"].attend_rows(a["q"], a["k"], a["v"], t, n, st, out=outs[3 + j])
        if i % 25 < 3:
            torch.cuda.synchronize()
            assert torch.equal(outs[j], want[j]) and torch.equal(outs[3 + j], want[3 + j])
            outs[j].zero_()
            outs[3 + j].fill_(7.0)
    for a in cases + more:
        a["c"].sync()
        a["c"].close()
