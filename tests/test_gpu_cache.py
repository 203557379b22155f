"""The paged-cache operators against float64 (needs a GB300).

Tolerances, with u = 2^-24 (half a step of fp32) and e the half step of the
output type (bf16 2^-8, fp32 2^-24):

append  A normalised element costs at most 16 + 3 additions for its mean square
        (halved by the root), a root, a quotient and three products: under
        20 u.  The rotated value x cos - y sin adds two products, a sum and the
        table's own rounding: 4 u of |x| + |y|.  Then one rounding:
            24 u (|x| + |y|) (1 + e) + e |ref|.
attend  Products of bf16 values are exact in fp32, those of fp32 values round;
        a score is HD products summed: at most (HD + 4) 2u sum_d |q_d k_d| scale
        =: d off (2u: the tensor core's sums may truncate), so its exponential
        (1 + 2d).  The weighted sum and the denominator add up len terms, in at
        worst len additions (2u each) and a few rescalings: (len + 64) 2u each.
        The exponential itself is good to 4 u, and 2^-16 covers weights that
        enter the product as a sum of two bf16 numbers:
            r = 2 d + 2 (len + 64) 2u + 8u + 2^-16
            out:      r sum_j p_j |v_j| (1 + e) + e |ref|
            weights:  r sum_g p_g + (G + 1) u |ref|.
evict   copies and choices: exact."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import cache as oc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


def make_pages(rng, lens, page, extra=3, cols=None):
    """A page table whose pages lie in random order, unused entries far out of
    range (they must never be read), and the number of pages of the pool."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra
    ids = rng.permutation(total)
    cols = cols or max(1, max(need))
    table = np.full((len(lens), cols), 2 ** 30, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    return table, total


def pool(rng, total, page, nkv, hd, dtype, fill=None):
    t = torch.from_numpy(rng.standard_normal((total, page, nkv, hd)).astype(np.float32)).cuda().to(DT[dtype])
    if fill is not None:
        t.fill_(fill)
    return t


def blank_behind(pages, table, lens, page, value):
    """Every slot that holds no live position gets `value`."""
    live = torch.zeros(pages.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens):
        for c in range(-(-n // page)):
            live[table[s, c], :min(page, n - c * page)] = True
    pages[~live.cuda()] = value


# ---------------------------------------------------------------- append

APPEND = [
    # heads, dtype, page, lens before, new rows of each, norm, what
    ((4, 2, 64), "f32", 16, [0], [1], False),
    ((4, 2, 64), "f32", 24, [5, 0, 100], [1, 1, 1], True),
    ((12, 2, 128), "bf16", 32, [511], [1], True),
    ((28, 4, 128), "bf16", 7, [3, 60], [40, 1], True),
    ((40, 8, 128), "bf16", 32, [31, 0, 64], [33, 130, 1], False),
    ((10, 5, 128), "f32", 1, [2, 2], [5, 3], True),
    ((16, 1, 128), "bf16", 100, [99], [257], True),
    ((8, 8, 64), "bf16", 64, [0], [777], True),
    ((3, 1, 64), "f32", 5, [1], [11], False),
]


def append_case(sf, heads, dtype, page, before, new, norm, seed=0, far=0):
    rng = np.random.default_rng([seed, page, sum(new)])
    nq, nkv, hd = heads
    lens = [a + b for a, b in zip(before, new)]
    table, total = make_pages(rng, lens, page)
    seq = np.repeat(np.arange(len(new)), new)
    index = np.concatenate([np.arange(a, a + b) for a, b in zip(before, new)])
    order = rng.permutation(len(seq))               # rows of sequences mixed up
    seq, index = seq[order], index[order]
    pos = index + far
    T = len(seq)
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(new),
                      max_len=max(lens), max_pos=max(lens) + far)
    wide = torch.from_numpy(rng.standard_normal((T, (nq + 2 * nkv) * hd + 64)).astype(np.float32)).cuda().to(DT[dtype])
    gq, gk = ((torch.from_numpy(1 + 0.3 * rng.standard_normal(hd)).float().cuda() for _ in range(2)) if norm
              else (None, None))
    return dict(c=c, rng=rng, table=table, total=total, seq=seq, index=index, pos=pos, T=T, gq=gq, gk=gk,
                qkv=wide[:, 16:16 + (nq + 2 * nkv) * hd], lens=lens)


def check_append(heads, dtype, page, a, q, k, v, k0, v0, rows=None):
    nq, nkv, hd = heads
    x = f64(a["qkv"]).reshape(a["T"], nq + 2 * nkv, hd)
    rows = range(a["T"]) if rows is None else rows
    e = E[dtype]
    wk, wv = f64(k0).reshape(-1, nkv, hd), f64(v0).reshape(-1, nkv, hd)
    tk = np.zeros_like(wk)
    for t in rows:
        for part, gain, sl in ((0, a["gq"], slice(0, nq)), (1, a["gk"], slice(nq, nq + nkv))):
            n = oc.head_norm(x[t, sl], None if gain is None else f64(gain), 1e-6)
            ref = oc.rotate(n, np.array(a["pos"][t]), 10000.0)
            mag = np.abs(n)
            mag = np.concatenate([mag[:, :hd // 2] + mag[:, hd // 2:]] * 2, -1)
            tol = 24 * U * mag * (1 + e) + e * np.abs(ref)
            if part == 0:
                assert np.all(np.abs(f64(q[t]) - ref) <= tol), (t, np.abs(f64(q[t]) - ref).max())
            elif a["index"][t] >= 0:
                slot = a["table"][a["seq"][t], a["index"][t] // page] * page + a["index"][t] % page
                wk[slot], tk[slot] = ref, tol
                wv[slot] = x[t, nq + nkv:]
    assert np.all(np.abs(f64(k).reshape(wk.shape) - wk) <= tk)     # untouched slots: bit for bit
    assert np.array_equal(f64(v).reshape(wv.shape), wv)


@pytest.mark.parametrize("heads,dtype,page,before,new,norm", APPEND)
def test_append(sf, heads, dtype, page, before, new, norm):
    a = append_case(sf, heads, dtype, page, before, new, norm, far=1000)
    k, v = (pool(a["rng"], a["total"], page, heads[1], heads[2], dtype) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    q = a["c"].append(a["qkv"], i32(a["index"]), i32(a["table"]), k, v, pos=i32(a["pos"]), seq=i32(a["seq"]),
                      q_gain=a["gq"], k_gain=a["gk"])
    a["c"].sync()
    check_append(heads, dtype, page, a, q, k, v, k0, v0)
    # in place of the query part of the rows, the same bits
    k2, v2 = k0.clone(), v0.clone()
    packed = a["qkv"].clone()
    nq, hd = heads[0], heads[2]
    q2 = a["c"].append(packed, i32(a["index"]), i32(a["table"]), k2, v2, pos=i32(a["pos"]), seq=i32(a["seq"]),
                       q_gain=a["gq"], k_gain=a["gk"], q=packed[:, :nq * hd])
    assert torch.equal(q2.reshape(q.shape), q) and torch.equal(k2, k) and torch.equal(v2, v)
    assert torch.equal(packed[:, nq * hd:], a["qkv"][:, nq * hd:])
    a["c"].close()


def test_append_far_positions(sf):
    """Angles of about 10^6 radians: fp32 angles would be off by 0.03."""
    heads, page = (4, 2, 64), 16
    a = append_case(sf, heads, "f32", page, [0], [9], False, far=1000003)
    k, v = (pool(a["rng"], a["total"], page, 2, 64, "f32") for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    q = a["c"].append(a["qkv"], i32(a["index"]), i32(a["table"]), k, v, pos=i32(a["pos"]), seq=i32(a["seq"]))
    a["c"].sync()
    check_append(heads, "f32", page, a, q, k, v, k0, v0)
    a["c"].close()


def test_append_defaults_padding_and_only_one_gain(sf):
    """seq NULL: row t of sequence t; pos NULL: the place; padding rows and rows
    without a place leave everything of theirs as it was."""
    heads, page = (4, 2, 64), 16
    a = append_case(sf, heads, "bf16", page, [3, 9, 16, 20], [1, 1, 1, 1], True, seed=3)
    a["gq"] = None
    a["seq"], a["index"] = np.arange(4), np.array([3, 9, 16, 20])
    a["pos"] = a["index"].copy()
    k, v = (pool(a["rng"], a["total"], page, 2, 64, "bf16") for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    q = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    index = a["index"].copy()
    index[2] = -1                                   # no position either: padding
    a["c"].append(a["qkv"], i32(index), i32(a["table"]), k, v, k_gain=a["gk"], q=q)
    a["c"].sync()
    check_append(heads, "bf16", page, a, q, k, v, k0, v0, rows=[0, 1, 3])
    assert torch.all(q[2] == 7.0)
    # a position without a place: the query only
    k, v = k0.clone(), v0.clone()
    a["index"] = index
    a["c"].append(a["qkv"], i32(index), i32(a["table"]), k, v, pos=i32(a["pos"]), k_gain=a["gk"], q=q)
    a["c"].sync()
    check_append(heads, "bf16", page, a, q, k, v, k0, v0)
    # nothing to do
    none = torch.zeros((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    assert a["c"].append(none, i32([]), i32(a["table"]), k, v, seq=i32([])).shape == (0, 4, 64)
    a["c"].sync()
    a["c"].close()


def test_append_reports_bad_rows_and_pages(sf):
    """Out-of-range sequences, places, positions and pages are skipped and
    reported; the other rows are written; the report is read once."""
    heads, page = (4, 2, 64), 16
    a = append_case(sf, heads, "f32", page, [0, 0], [20, 20], False, seed=5)
    order = np.lexsort((a["index"], a["seq"]))
    a["seq"], a["index"], a["pos"] = a["seq"][order], a["index"][order], a["pos"][order]
    good = dict(seq=a["seq"].copy(), index=a["index"].copy(), pos=a["pos"].copy(), table=a["table"].copy())

    def run(**kw):
        b = dict(good, **kw)
        k, v = (torch.zeros((a["total"], page, 2, 64), device="cuda") for _ in range(2))
        q = torch.zeros((a["T"], 4, 64), device="cuda")
        a["c"].append(a["qkv"], i32(b["index"]), i32(b["table"]), k, v, pos=i32(b["pos"]), seq=i32(b["seq"]), q=q)
        return k, v, q

    def changed(key, row, value):
        x = good[key].copy()
        x[row] = value
        return {key: x}

    k0, v0, q0 = run()
    a["c"].sync()
    for kw, q_kept in ((changed("seq", 4, 2), True), (changed("seq", 4, -1), True), (changed("index", 4, 20), True),
                       (changed("index", 4, 2 ** 31 - 1), True), (changed("pos", 4, 20), False),
                       (changed("pos", 4, 2 ** 31 - 1), False)):
        k, v, q = run(**kw)
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "row" in str(e.value)
        slot = int(a["table"][0, 0]) * page + 4
        keep = torch.ones(a["total"] * page, dtype=torch.bool, device="cuda")
        keep[slot] = False
        assert torch.equal(k.view(-1, 128)[keep], k0.view(-1, 128)[keep]) and not k.view(-1, 128)[slot].any()
        assert torch.equal(v.view(-1, 128)[keep], v0.view(-1, 128)[keep]) and not v.view(-1, 128)[slot].any()
        assert torch.equal(q[torch.arange(a["T"]) != 4], q0[torch.arange(a["T"]) != 4])
        assert torch.equal(q[4], q0[4]) if q_kept else not q[4].any()
        a["c"].sync()                               # read once
    for bad in (-1, a["total"], 2 ** 31 - 1, -2 ** 31):
        t = good["table"].copy()
        t[1, 1] = bad
        k, v, q = run(table=t)
        with pytest.raises(sf.SpecFoldError) as e:
            run()                                   # a later call reports it too (once it has been met)
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT
        torch.cuda.synchronize()
        try:
            a["c"].sync()
        except sf.SpecFoldError:
            pass
        assert torch.equal(q, q0)
        page1 = int(a["table"][1, 1])
        rest = torch.arange(a["total"], device="cuda") != page1
        assert torch.equal(k[rest], k0[rest]) and not k[page1].any()
    a["c"].close()


# ---------------------------------------------------------------- attend

ATTEND = [
    # heads, dtype, page, lens
    ((4, 2, 64), "f32", 16, [1]),
    ((4, 2, 64), "f32", 24, [0, 1, 2, 17, 333]),
    ((12, 2, 128), "f32", 7, [129, 0, 64]),
    ((10, 5, 128), "f32", 1, [31, 5]),
    ((3, 1, 64), "f32", 32, [1000]),
    ((16, 1, 128), "f32", 64, [100, 260]),
    ((12, 2, 128), "bf16", 32, [1]),
    ((12, 2, 128), "bf16", 32, [512]),
    ((4, 2, 64), "bf16", 5, [0, 1, 15, 16, 17, 31, 32, 33, 127, 129, 700]),
    ((28, 4, 128), "bf16", 16, [1, 2047, 0, 64]),
    ((40, 8, 128), "bf16", 100, [255, 256, 257]),
    ((8, 8, 64), "bf16", 1, [63, 3]),
    ((6, 6, 128), "bf16", 24, [77]),
    ((16, 1, 128), "bf16", 48, [1500, 9]),
    ((21, 1, 64), "bf16", 16, [90, 513]),
    ((80, 2, 128), "bf16", 16, [70, 1]),
    ((7, 7, 128), "bf16", 65536, [300]),
    ((32, 8, 128), "bf16", 64, [20000, 3]),
    ((14, 2, 64), "bf16", 16, [40000]),
]


def attend_inputs(sf, heads, dtype, page, lens, seed=0, track=True, q_std=2.0, cols=None):
    nq, nkv, hd = heads
    rng = np.random.default_rng([seed, page, sum(lens)])
    table, total = make_pages(rng, lens, page, cols=cols)
    k, v = (pool(rng, total, page, nkv, hd, dtype) for _ in range(2))
    blank_behind(k, table, lens, page, float("nan"))
    blank_behind(v, table, lens, page, float("inf"))
    q = (torch.from_numpy(rng.standard_normal((len(lens), nq, hd)).astype(np.float32)) * q_std).cuda().to(DT[dtype])
    w = torch.from_numpy(rng.random((len(lens), nkv, max(1, max(lens)) + 5)).astype(np.float32)).cuda()
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(lens),
                      max_len=max(1, max(lens)), track_weights=track)
    return dict(c=c, rng=rng, table=table, k=k, v=v, q=q, w=w, lens=lens)


def check_attend(heads, dtype, page, a, out, w_out, scale=None, w_in=None, seqs=None):
    nq, nkv, hd = heads
    G, e = nq // nkv, E[dtype]
    scale = hd ** -0.5 if scale is None else scale
    for s, n in enumerate(a["lens"]):
        if seqs is not None and s not in seqs:
            continue
        idx = np.arange(n)
        slot = torch.from_numpy(a["table"][s, idx // page].astype(np.int64) * page + idx % page).cuda()
        k, v = (f64(a[x].view(-1, nkv, hd)[slot]) for x in ("k", "v"))
        q = f64(a["q"][s])
        ref, p = oc.attend_one(q, k, v, scale)
        wref = np.zeros((nkv, n))
        wtol = np.zeros((nkv, n))
        for h in range(nq):
            c = h // G
            d = ((hd + 4) * 2 * U * abs(scale) * (np.abs(k[:, c]) @ np.abs(q[h]))).max() if n else 0.0
            r = 2 * d + 4 * (n + 64) * U + 8 * U + 2.0 ** -16
            tol = r * (p[h] @ np.abs(v[:, c])) * (1 + e) + e * np.abs(ref[h])
            got = f64(out[s, h])
            assert np.all(np.abs(got - ref[h]) <= tol), (s, h, np.abs(got - ref[h]).max(), tol.min())
            wref[c] += p[h]
            wtol[c] += r * p[h]
        if w_out is not None:
            base = 0.0 if w_in is None else f64(w_in[s, :, :n])
            full = base + wref
            assert np.all(np.abs(f64(w_out[s, :, :n]) - full) <= wtol + (G + 1) * U * np.abs(full)), s


@pytest.mark.parametrize("heads,dtype,page,lens", ATTEND)
def test_attend(sf, heads, dtype, page, lens):
    """Output and weights; NaN keys and infinite values behind every length;
    table entries behind it far out of range."""
    a = attend_inputs(sf, heads, dtype, page, lens)
    table, ln = i32(a["table"]), i32(lens)
    w_out = torch.full_like(a["w"], -3.0)
    out = a["c"].attend(a["q"], a["k"], a["v"], table, ln, weights=a["w"], weights_out=w_out)
    a["c"].sync()
    check_attend(heads, dtype, page, a, out, w_out, w_in=a["w"])
    for s, n in enumerate(lens):
        assert torch.all(w_out[s, :, n:] == -3.0)                      # behind the sequence: as it was
        if n == 0:
            assert not out[s].any()
    # without weights the same bits, call after call; in place; this call's weights alone
    assert torch.equal(a["c"].attend(a["q"], a["k"], a["v"], table, ln), out)
    assert torch.equal(a["c"].attend(a["q"], a["k"], a["v"], table, ln), out)
    w2 = a["w"].clone()
    a["c"].attend(a["q"], a["k"], a["v"], table, ln, weights=w2)
    only = torch.zeros_like(a["w"])
    a["c"].attend(a["q"], a["k"], a["v"], table, ln, weights_out=only)
    a["c"].sync()
    for s, n in enumerate(lens):
        assert torch.equal(w2[s, :, :n], w_out[s, :, :n]) and torch.equal(w2[s, :, n:], a["w"][s, :, n:])
        if n:
            total = f64(only[s, :, :n]).sum(1)
            np.testing.assert_allclose(total, heads[0] // heads[1], rtol=1e-4)
    a["c"].close()


def test_attend_strided_rows_scale_and_wide_table(sf):
    heads, page, lens = (12, 2, 128), 16, [100, 40, 7]
    a = attend_inputs(sf, heads, "bf16", page, lens, seed=9, cols=40)
    wide = torch.zeros((3, 2048 + 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 64:64 + 1536] = a["q"].view(3, -1)
    tab = torch.full((3, 64), -5, dtype=torch.int32, device="cuda")
    tab[:, 10:50] = i32(a["table"])
    dst = torch.full((3, 4000), 9.0, dtype=torch.bfloat16, device="cuda")
    for scale in (0.01, 1.5, -0.3, 0.0):
        out = a["c"].attend(wide[:, 64:64 + 1536], a["k"], a["v"], tab[:, 10:50], i32(lens), scale=scale,
                            out=dst[:, 8:8 + 1536])
        a["c"].sync()
        check_attend(heads, "bf16", page, a, out.view(3, 12, 128) if out.is_contiguous() else out.reshape(3, 12, 128),
                     None, scale=scale)
        assert torch.all(dst[:, :8] == 9.0) and torch.all(dst[:, 8 + 1536:] == 9.0)
    a["c"].close()


def test_attend_shared_pages(sf):
    """A prefix that several sequences share, and the same page twice in one."""
    heads, page = (28, 4, 128), 32
    lens = [200, 200, 64]
    a = attend_inputs(sf, heads, "bf16", page, lens, seed=4)
    a["table"][1, :4] = a["table"][0, :4]
    a["table"][2, :2] = a["table"][0, 1]
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens))
    a["c"].sync()
    check_attend(heads, "bf16", page, a, out, None)
    a["c"].close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (12, 2, 128)])
def test_attend_extreme_scores(sf, heads, dtype):
    """Scores of +-10^4 (one key takes all), equal scores, values of the type's
    largest size, and a key of minus infinity score."""
    page, lens = 16, [50, 50, 50, 50]
    a = attend_inputs(sf, heads, dtype, page, lens, seed=6)
    nkv, hd = heads[1:]

    def row(s, j):
        return a["table"][s, j // page], j % page

    a["q"][0] *= 2000                                   # one key far above all others
    a["q"][1] = 0                                       # all scores equal
    for j in range(50):
        a["v"][row(2, j)] = 1e38 if j % 2 else -1e38    # large values
    a["k"][row(3, 7)] = -float("inf")                   # with q > 0: weight exactly 0
    a["q"][3] = a["q"][3].abs() + 0.1
    w = torch.zeros_like(a["w"])
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights_out=w)
    a["c"].sync()
    assert torch.isfinite(out).all() and torch.isfinite(w[..., :50]).all()
    assert not w[3, :, 7].any()
    a["k"][row(3, 7)] = -1e30                           # float64 agrees: the same weights
    check_attend(heads, dtype, page, a, out, None, seqs=(1, 2))
    for s in (0, 3):
        for h in range(heads[0]):
            c = h // (heads[0] // nkv)
            idx = np.arange(50)
            slot = torch.from_numpy(a["table"][s, idx // page].astype(np.int64) * page + idx % page).cuda()
            k, v = (f64(a[x].view(-1, nkv, hd)[slot])[:, c] for x in ("k", "v"))
            sc = k @ f64(a["q"][s, h]) * hd ** -0.5
            top = np.sort(sc)
            if s == 3 or top[-1] - top[-2] > 100:       # decided: the winner's value, rounded
                e = np.exp(sc - sc.max())
                ref = (e / e.sum()) @ v
                d = ((hd + 4) * 2 * U * hd ** -0.5 * (np.abs(k[np.arange(50) != 7]) @ np.abs(f64(a["q"][s, h])))).max()
                r = (2 * d if s == 3 else 0) + 4 * 114 * U + 2.0 ** -16
                assert np.all(np.abs(f64(out[s, h]) - ref) <= r * (e / e.sum() @ np.abs(v)) + E[dtype] * np.abs(ref))
    # NaN and infinities among the live keys follow the formula
    a["k"][row(1, 3)] = float("nan")
    a["v"][row(2, 5)] = float("inf")
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens))
    a["c"].sync()
    assert torch.isnan(out[1]).all() and not torch.isfinite(out[2]).any()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[3]).all()
    a["k"][row(3, 7)] = float("inf")                    # a score of +infinity: infinity - infinity
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens))
    a["c"].sync()
    assert torch.isnan(out[3]).all()
    a["c"].close()


def test_attend_reports_bad_lengths_and_pages(sf):
    heads, page, lens = (12, 2, 128), 16, [40, 33, 20]
    a = attend_inputs(sf, heads, "bf16", page, lens, seed=8)
    w = a["w"].clone()
    ref = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens))
    a["c"].sync()
    for bad in (-1, 41, 2 ** 31 - 1, -2 ** 31):
        out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32([40, bad, 20]), weights=w)
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "length" in str(e.value)
        # without sequence 1 the batch is split elsewhere: the others to rounding
        check_attend(heads, "bf16", page, a, out, None, seqs=(0, 2))
        assert not out[1].any() and torch.equal(w[1], a["w"][1])
    for bad in (-1, a["k"].shape[0], 2 ** 31 - 1):
        t = a["table"].copy()
        t[1, 1] = bad                                   # positions 16..31 of sequence 1
        w = a["w"].clone()
        out = a["c"].attend(a["q"], a["k"], a["v"], i32(t), i32(lens), weights=w)
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "page" in str(e.value)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
        assert torch.equal(w[1, :, 16:32], a["w"][1, :, 16:32])       # absent: no weight
        # what is left of sequence 1 is attended
        b = dict(a, lens=[17])
        b["table"] = np.stack([np.concatenate([t[1, :1], t[1, 2:3]])])
        b["q"] = a["q"][1:2]
        check_attend(heads, "bf16", page, b, out[1:2], None)
    a["c"].close()


def test_attend_many_sequences(sf):
    """More sequences than thread blocks: mostly short, some empty, a few long."""
    heads, page = (8, 2, 64), 16
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 40, 600)]
    lens[17], lens[400], lens[599] = 3000, 1023, 1
    a = attend_inputs(sf, heads, "bf16", page, lens, seed=12)
    w = torch.zeros_like(a["w"])
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights_out=w)
    a["c"].sync()
    check_attend(heads, "bf16", page, a, out, w)
    a["c"].close()


# ---------------------------------------------------------------- evict

EVICT = [
    # heads, dtype, page, lens, budget, n_first, n_recent
    ((4, 2, 64), "f32", 16, [1], 1, 0, 0),
    ((4, 2, 64), "f32", 24, [0, 1, 2, 40, 333], 33, 2, 5),
    ((12, 2, 128), "bf16", 32, [512], 256, 4, 64),
    ((12, 2, 128), "bf16", 7, [50, 20, 0], 20, 0, 20),
    ((40, 8, 128), "bf16", 16, [700, 65], 64, 0, 0),
    ((8, 8, 64), "bf16", 1, [1025, 1024, 1023], 1024, 1, 1),
    ((6, 6, 128), "f32", 100, [1999], 1, 0, 0),
    ((3, 1, 64), "f32", 5, [4097], 4096, 100, 3000),
    ((16, 1, 128), "bf16", 64, [9000, 100], 5000, 4, 0),
    ((10, 5, 128), "bf16", 48, [40000], 777, 4, 128),
]


def weights_like(rng, shape, kind):
    if kind == "spread":
        w = np.exp(3 * rng.standard_normal(shape))
    elif kind == "ties":
        w = rng.integers(0, 4, shape) / 2.0
    elif kind == "equal":
        w = np.full(shape, 0.25)
    else:                                                # anything that floats can be
        w = rng.standard_normal(shape)
        for x in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, 3e38):
            w[rng.random(shape) < 0.06] = x
    return w.astype(np.float32)


def evict_ref(a, heads, page, budget, n_first, n_recent):
    nkv = heads[1]
    k, v, w = (a[x].cpu() for x in ("k", "v", "w"))
    kept, rows = [], []
    for s, n in enumerate(a["lens"]):
        ks, vs = (oc.sequence(x.float().numpy(), a["table"][s], n, page) for x in (k, v))
        for c in range(nkv):
            ids = oc.choose(w[s, c].numpy(), n, budget, n_first, n_recent)
            kept.append(ids)
            rows.append((ks[ids, c], vs[ids, c], w[s, c].numpy()[ids]))
    return kept, rows


def check_evict(a, heads, page, budget, kept, rows, got_kept, lens_out, w0, w_out, k0, k_out, v_out, table_out):
    nkv = heads[1]
    for s, n in enumerate(a["lens"]):
        m = min(n, budget)
        assert int(lens_out[s]) == m
        for c in range(nkv):
            ids, (ks, vs, ws) = kept[s * nkv + c], rows[s * nkv + c]
            g = got_kept[s, c].cpu().numpy()
            assert g[:m].tolist() == ids and np.all(g[m:] == -1), (s, c)
            w = w_out[s, c].cpu().numpy()
            assert np.array_equal(w[:m], ws, equal_nan=True) and not w[m:n].any()
            assert np.array_equal(w[n:], w0[s, c, n:].cpu().numpy(), equal_nan=True)
        for x, i in ((k_out, 0), (v_out, 1)):
            got = oc.sequence(x.float().cpu().numpy(), table_out[s], m, page)
            for c in range(nkv):
                assert np.array_equal(got[:, c], rows[s * nkv + c][i]), (s, c, i)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "any"])
@pytest.mark.parametrize("heads,dtype,page,lens,budget,n_first,n_recent", EVICT)
def test_evict(sf, heads, dtype, page, lens, budget, n_first, n_recent, kind):
    nq, nkv, hd = heads
    a = attend_inputs(sf, heads, dtype, page, lens, seed=2, track=False)
    blank_behind(a["k"], a["table"], lens, page, 1.0)
    blank_behind(a["v"], a["table"], lens, page, 1.0)
    a["w"] = torch.from_numpy(weights_like(a["rng"], tuple(a["w"].shape), kind)).cuda()
    kept, rows = evict_ref(a, heads, page, budget, n_first, n_recent)
    # to other pages
    out_lens = [min(n, budget) for n in lens]
    table_out, total_out = make_pages(a["rng"], out_lens, page, cols=-(-budget // page) + 2)
    k_out, v_out = (torch.full((total_out, page, nkv, hd), 5.0, device="cuda", dtype=DT[dtype]) for _ in range(2))
    k0, v0, w0 = a["k"].clone(), a["v"].clone(), a["w"].clone()
    w_out = torch.full_like(a["w"], 4.0)
    lens_out, got = a["c"].evict(a["k"], a["v"], i32(a["table"]), i32(lens), a["w"], budget, n_first=n_first,
                                 n_recent=n_recent, k_out=k_out, v_out=v_out, table_out=i32(table_out),
                                 weights_out=w_out)
    a["c"].sync()
    check_evict(a, heads, page, budget, kept, rows, got, lens_out, torch.full_like(w0, 4.0), w_out, k0, k_out, v_out,
                table_out)
    assert torch.equal(a["k"], k0) and torch.equal(a["v"], v0)          # the input is only read
    blank = k_out.clone()
    blank_behind(blank, table_out, out_lens, page, 5.0)
    assert torch.equal(blank, k_out)                                    # slots behind the kept rows: as they were
    # in place, lens and weights too
    ln = i32(lens)
    lens_out, got2 = a["c"].evict(a["k"], a["v"], i32(a["table"]), ln, a["w"], budget, n_first=n_first,
                                  n_recent=n_recent, lens_out=ln)
    a["c"].sync()
    assert torch.equal(got2, got)
    check_evict(a, heads, page, budget, kept, rows, got2, ln, w0, a["w"], k0, a["k"], a["v"], a["table"])
    moved = torch.zeros_like(k0)
    blank_behind(moved, a["table"], out_lens, page, 1.0)
    assert torch.equal(a["k"][moved.bool()], k0[moved.bool()])          # slots behind the kept rows: as they were
    a["c"].close()


def test_evict_reports_bad_lengths_and_pages(sf):
    heads, page, lens = (4, 2, 64), 16, [60, 60, 60]
    a = attend_inputs(sf, heads, "f32", page, lens, seed=3, track=False)
    k0, v0, w0 = a["k"].clone(), a["v"].clone(), a["w"].clone()
    for bad in (-1, 61, 2 ** 31 - 1):
        lens_out, kept = a["c"].evict(a["k"], a["v"], i32(a["table"]), i32([60, bad, 60]), a["w"], 60)
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "length" in str(e.value)
        assert lens_out.tolist() == [60, 0, 60] and torch.all(kept[1] == -1)
        assert torch.equal(a["w"], w0)
        assert torch.equal(a["k"].nan_to_num(9.0), k0.nan_to_num(9.0))
    table_out, total = make_pages(a["rng"], [20] * 3, page)
    for bad in (-1, total, 2 ** 31 - 1):
        for which in ("in", "out"):
            t, to = a["table"].copy(), table_out.copy()
            (t if which == "in" else to)[1, 1] = bad
            k_out, v_out = (torch.zeros((total, page, 2, 64), device="cuda") for _ in range(2))
            w_out = torch.zeros_like(w0)
            _, kept = a["c"].evict(a["k"], a["v"], i32(t), i32(lens), w0, 20, k_out=k_out, v_out=v_out,
                                   table_out=i32(to), weights_out=w_out)
            if bad == total and which == "in":          # a page of the larger input pool: fine
                a["c"].sync()
                continue
            with pytest.raises(sf.SpecFoldError) as e:
                a["c"].sync()
            assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "page" in str(e.value)
            for s in range(3):
                for c in range(2):
                    for i in range(20):
                        j = int(kept[s, c, i])
                        if s == 1 and (i if which == "out" else j) // page == 1:
                            if which == "in":
                                assert not k_out[to[s, i // page], i % page, c].any()
                            continue
                        assert torch.equal(k_out[to[s, i // page], i % page, c], k0[a["table"][s, j // page],
                                                                                    j % page, c])
    a["c"].close()


# ---------------------------------------------------------------- together

def _decode(sf, c, steps, tensors, budget, stream=None):
    """Rows of `steps` tokens through append, attend and evict, as a decode loop runs them."""
    outs = []
    for qkv, index, pos in steps:
        q = c.append(qkv, index, tensors["table"], tensors["k"], tensors["v"], pos=pos, q_gain=tensors["g"],
                     k_gain=tensors["g"], stream=stream)
        outs.append(c.attend(q, tensors["k"], tensors["v"], tensors["table"], index + 1, weights=tensors["w"],
                             stream=stream))
    lens, kept = c.evict(tensors["k"], tensors["v"], tensors["table"], steps[-1][1] + 1, tensors["w"], budget,
                         n_first=1, n_recent=4, stream=stream)
    return outs, lens, kept


def _decode_inputs(sf, dtype, seed, n=3, steps=20):
    heads, page = (12, 2, 128), 16
    rng = np.random.default_rng([seed, 77])
    table, total = make_pages(rng, [64] * n, page)
    c = sf.PagedCache(n_q_heads=12, n_kv_heads=2, head_dim=128, dtype=dtype, page_size=page, max_seqs=n, max_len=64,
                      max_pos=5000, track_weights=True)
    t = dict(table=i32(table), k=torch.zeros((total, page, 2, 128), dtype=DT[dtype], device="cuda"),
             w=torch.zeros((n, 2, 64), device="cuda"),
             g=torch.from_numpy(1 + 0.2 * rng.standard_normal(128)).float().cuda())
    t["v"] = t["k"].clone()
    rows = torch.from_numpy(rng.standard_normal((40, n, 16, 128)).astype(np.float32)).cuda().to(DT[dtype])
    return heads, page, table, c, t, rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_loop_with_eviction(sf, dtype):
    """40 tokens of three sequences with an eviction to 16 positions half way;
    every step against float64 on the keys and values as stored."""
    heads, page, table, c, t, rows = _decode_inputs(sf, dtype, 1)
    ref_w = np.zeros((3, 2, 64))
    tol_w = 0.0
    n = 0
    for i in range(40):
        index = i32([n] * 3)
        q = c.append(rows[i], index, t["table"], t["k"], t["v"], pos=i32([i + 7] * 3), q_gain=t["g"], k_gain=t["g"])
        out = c.attend(q, t["k"], t["v"], t["table"], index + 1, weights=t["w"])
        n += 1
        a = dict(table=table, k=t["k"], v=t["v"], q=q, lens=[n] * 3)
        check_attend(heads, dtype, page, a, out, None)
        x = f64(rows[i])
        for s in range(3):
            slot = table[s, (n - 1) // page] * page + (n - 1) % page
            want = oc.rotate(oc.head_norm(x[s, 12:14], f64(t["g"]), 1e-6), np.array(i + 7), 10000.0)
            got = f64(t["k"].view(-1, 2, 128)[slot])
            np.testing.assert_allclose(got, want, rtol=1.01 * E[dtype], atol=24 * U * 2 * np.abs(x).max())
            idx = np.arange(n)
            slots = torch.from_numpy(table[s, idx // page].astype(np.int64) * page + idx % page).cuda()
            k, v = (f64(t[y].view(-1, 2, 128)[slots]) for y in ("k", "v"))
            _, p = oc.attend_one(f64(q[s]), k, v, 128 ** -0.5)
            ref_w[s, 0, :n] += p[:6].sum(0)
            ref_w[s, 1, :n] += p[6:].sum(0)
        np.testing.assert_allclose(f64(t["w"]), ref_w, rtol=1e-3, atol=1e-4)
        if n == 36:
            a = dict(table=table, k=t["k"].clone(), v=t["v"].clone(), w=t["w"].clone(), lens=[36] * 3)
            kept, want = evict_ref(a, heads, page, 16, 1, 4)
            lens, got = c.evict(t["k"], t["v"], t["table"], index + 1, t["w"], 16, n_first=1, n_recent=4)
            check_evict(a, heads, page, 16, kept, want, got, lens, a["w"], t["w"], a["k"], t["k"], t["v"], table)
            ref_w = f64(t["w"]).copy()
            n = 16
    c.sync()
    c.close()


def test_graph_capture_and_side_stream(sf):
    """The loop captured into a graph on one object and replayed gives the bits
    of the eager loop on another, on a side stream; both objects' calls overlap."""
    res = []
    for mode in ("eager", "graph"):
        heads, page, table, c, t, rows = _decode_inputs(sf, "bf16", 2)
        steps = [(rows[i], i32([i] * 3), i32([i] * 3)) for i in range(30)]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        if mode == "eager":
            outs, lens, kept = _decode(sf, c, steps, t, 16, stream=st)
            c.sync(st)
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs, lens, kept = _decode(sf, c, steps, t, 16)
            for x in ("k", "v", "w"):
                t[x].zero_()
            for o in outs:
                o.fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            first = [o.clone() for o in outs]
            for x in ("k", "v", "w"):
                t[x].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, outs))
            c.sync()
        res.append((outs, lens, kept, t["k"], t["v"], t["w"], c))
    (o1, l1, k1, *p1, c1), (o2, l2, k2, *p2, c2) = res
    assert all(torch.equal(a, b) for a, b in zip(o1, o2))
    assert torch.equal(l1, l2) and torch.equal(k1, k2) and all(torch.equal(a, b) for a, b in zip(p1, p2))
    c1.close()
    c2.close()


def test_two_objects_at_once(sf):
    """Attend calls of two objects on two streams, interleaved, against each alone."""
    cases = [attend_inputs(sf, (12, 2, 128), "bf16", 16, [3000, 500], seed=20),
             attend_inputs(sf, (28, 4, 128), "bf16", 32, [1000, 5000, 7], seed=21)]
    alone = []
    for a in cases:
        a["t"], a["l"] = i32(a["table"]), i32(a["lens"])
        alone.append(a["c"].attend(a["q"], a["k"], a["v"], a["t"], a["l"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(20):
        for i, a in enumerate(cases):
            got[i].append(a["c"].attend(a["q"], a["k"], a["v"], a["t"], a["l"], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, alone[i]) for x in got[i])
        cases[i]["c"].sync()
        cases[i]["c"].close()


def test_append_writes_the_prefix_of_a_pass(sf):
    """The prefix buffer of SpecFold.verify as the pool: append fills it from
    projected rows, the fp32 pass on it meets the oracle's pass on the oracle's
    prefix; after an eviction in place the pass takes the shorter prefix."""
    cfg = synth.CONFIGS["tiny"].with_(n_layers=2, n_requests=2, prefix_len=64)
    wl = synth.make_workload(cfg, seed=31, device="cuda")
    nq, nkv, hd, P, R, page = cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, 64, 2, 16
    rng = np.random.default_rng(5)
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype="f32", page_size=page, max_seqs=R, max_len=P,
                      track_weights=True)
    pk, pv = torch.zeros_like(wl.prefix_k), torch.zeros_like(wl.prefix_v)
    table = i32(np.arange(R * P // page).reshape(R, -1))
    index, seq = i32(np.tile(np.arange(P), R)), i32(np.repeat(np.arange(R), P))
    want_k = np.zeros(pk.shape)
    for l in range(2):
        qkv = torch.from_numpy(rng.standard_normal((R * P, nq + 2 * nkv, hd)).astype(np.float32)).cuda() * 0.3
        pools = [x[l].view(R * P // page, page, nkv, hd) for x in (pk, pv)]
        c.append(qkv, index, table, *pools, seq=seq)
        x = f64(qkv).reshape(R, P, -1, hd)
        want_k[l] = np.stack([oracle.rope(x[r, :, nq:nq + nkv], np.arange(P), cfg.rope_theta) for r in range(R)])
        assert torch.equal(pv[l], qkv.view(R, P, -1, hd)[:, :, nq + nkv:])
    c.sync()
    ctx = sf.from_config(cfg, wl.weights)
    out, fold, _, _ = ctx.verify(wl.hidden, wl.parents, pk, pv, cfg.delta)
    ctx.sync()
    Ws = [oracle.layer_weights_f64(w) for w in wl.weights]
    ref = oracle.verify_pass(f64(wl.hidden), wl.parents, cfg.delta, lambda l: Ws[l], want_k, f64(pv), cfg)
    assert np.array_equal(fold.cpu().numpy().astype(bool), ref["fold"])
    got, want = f64(out).reshape(-1, cfg.d_model), ref["out"].reshape(-1, cfg.d_model)
    assert np.max(np.abs(got - want).max(1) / np.maximum(np.abs(want).max(1), 1e-6)) <= 1e-4
    ctx.close()
    # half the prefix goes: what is left lies at the front of each request's buffer
    q = torch.randn((R, nq, hd), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    pools = [x[0].view(R * P // page, page, nkv, hd) for x in (pk, pv)]
    w = torch.zeros((R, nkv, P), device="cuda")
    c.attend(q, *pools, table, i32([P] * R), weights=w)
    k0 = pk[0].clone()
    lens, kept = c.evict(*pools, table, i32([P] * R), w, 32, n_recent=8)
    c.sync()
    assert lens.tolist() == [32, 32]
    for r in range(R):
        for h in range(nkv):
            assert torch.equal(pk[0, r, :32, h], k0[r, kept[r, h].long(), h])
    c.close()
