"""The paged-cache operators at the edges of what their header allows (needs a
GB300): rows without any score, outputs made on another stream, weights of
large scores, signed zeros, short rows in large objects, sums of the longest
sequence."""
import numpy as np
import pytest
import torch

from test_gpu_cache import attend_inputs, check_attend, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


# ---------------------------------------------------------------- rows without a score above -infinity

# heads, page, lens, sequences that lose every score; the blocks and the join that the batch's plan gives them
NOTHING = [
    ((12, 2, 128), 32, [100], [0]),                                          # a block a segment, no join
    ((12, 2, 128), 16, [15, 1], [1]),                                        # one position
    ((12, 2, 128), 16, [1000, 40], [0]),                                     # 8 blocks a segment, joined by the last
    ((14, 2, 64), 16, [20000], [0]),                                         # more than 24 parts: the join kernel
    ((16, 1, 128), 64, [9000, 77], [0, 1]),                                  # wide groups
    ((4, 4, 64), 16, [1 + 7 * i % 62 for i in range(300)], [0, 5, 123, 299]),  # a warp a segment
]


@pytest.mark.parametrize("how", ["pages", "scores"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,page,lens,gone", NOTHING)
def test_attend_without_a_score_gives_zeros(sf, heads, page, lens, gone, dtype, how):
    """Every page out of range (reported), or every score -infinity: zeros, and
    weights as they were; the other sequences of the batch are not affected."""
    a = attend_inputs(sf, heads, dtype, page, lens, seed=30)
    table = a["table"].copy()
    for s in gone:
        pages = -(-lens[s] // page)
        if how == "pages":
            a["table"][s, :pages] = -1
        else:
            a["q"][s] = a["q"][s].abs() + 0.1
            for c in range(pages):
                a["k"][table[s, c], :min(page, lens[s] - c * page)] = -float("inf")
    w_out = torch.full_like(a["w"], -3.0)
    calls = [a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights=a["w"], weights_out=w_out)]
    if how == "pages":
        with pytest.raises(sf.SpecFoldError) as e:
            a["c"].sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and "page" in str(e.value)
    calls.append(a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens)))
    torch.cuda.synchronize()
    for out in calls:
        for s in gone:
            assert not out[s].any(), s
    for s in gone:
        assert torch.equal(w_out[s, :, :lens[s]], a["w"][s, :, :lens[s]])
    rest = [s for s in range(len(lens)) if s not in gone]
    check_attend(heads, dtype, page, a, calls[0], w_out, w_in=a["w"], seqs=rest)
    check_attend(heads, dtype, page, a, calls[1], None, seqs=rest)
    a["c"].close()


# ---------------------------------------------------------------- outputs made by a call on another stream

def _current_stream_is_late(numel, dtype):
    """The current stream, asleep for some 100 ms, will then copy a block that is already free again: its copy, the
    block's address and its bytes."""
    block = torch.full((numel,), 7, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    return block.clone(), block.data_ptr(), block.numel() * block.element_size()


def _apart(t, address, size):
    assert t.data_ptr() + t.numel() * t.element_size() <= address or t.data_ptr() >= address + size


def test_outputs_on_a_side_stream_wait_for_nobody_and_spoil_nothing(sf):
    """A call on a stream makes its outputs in that stream's memory: never in a
    block that the current stream has freed but has still to read."""
    heads, page, n = (40, 8, 128), 32, 400
    lens = [40 + i % 9 for i in range(n)]
    a = attend_inputs(sf, heads, "bf16", page, lens, seed=31)
    c, table, ln, last = a["c"], i32(a["table"]), i32(lens), i32([x - 1 for x in lens])
    qkv = torch.randn((n, 56, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    st = torch.cuda.Stream()

    def calls(stream):
        k, v, w = a["k"].clone(), a["v"].clone(), a["w"].clone()
        torch.cuda.synchronize()
        blocks, got = [], []
        if stream is not None:
            blocks.append(_current_stream_is_late(n * 40 * 128, torch.bfloat16))
        got.append(c.append(qkv, last, table, k, v, stream=stream))
        if stream is not None:
            blocks.append(_current_stream_is_late(n * 40 * 128, torch.bfloat16))
        got.append(c.attend(got[0], k, v, table, ln, weights=w, stream=stream))
        if stream is not None:
            blocks.append(_current_stream_is_late(n * 8 * 30, torch.int32))
        got += c.evict(k, v, table, ln, w, 30, n_recent=4, stream=stream)
        for t in got:
            for copy, address, size in blocks:
                if t.dtype == copy.dtype:
                    _apart(t, address, size)
        c.sync(stream)
        torch.cuda.synchronize()
        assert all(bool((copy == 7).all()) for copy, _, _ in blocks)
        return got + [k, v, w]

    want = calls(None)
    for stream in (st, st.cuda_stream):
        for x, y in zip(calls(stream), want):
            assert torch.equal(x.view(torch.int8), y.view(torch.int8))    # bits: there is NaN behind the lengths
    c.close()


def test_decode_on_a_side_stream_with_ordered_inputs(sf):
    """Steps on a side stream, their inputs made before it waits for the current
    stream and kept until it is done, give the bits of the same steps on the
    current stream; and so does a graph of them replayed twice."""
    from test_gpu_cache import _decode_inputs

    def loop(c, t, rows, index, lens, stream):
        outs = []
        for i in range(30):
            q = c.append(rows[i], index[i], t["table"], t["k"], t["v"], q_gain=t["g"], k_gain=t["g"], stream=stream)
            outs.append(c.attend(q, t["k"], t["v"], t["table"], lens[i], weights=t["w"], stream=stream))
        return outs, c.evict(t["k"], t["v"], t["table"], lens[29], t["w"], 16, n_first=1, n_recent=4, stream=stream)

    res = []
    for mode in ("current", "side", "graph"):
        _, _, _, c, t, rows = _decode_inputs(sf, "bf16", 2)
        index, lens = [i32([i] * 3) for i in range(30)], [i32([i + 1] * 3) for i in range(30)]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        if mode == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs, (n, kept) = loop(c, t, rows, index, lens, None)
            for _ in range(2):
                for x in ("k", "v", "w"):
                    t[x].zero_()
                g.replay()
                torch.cuda.synchronize()
                c.sync()
        else:
            outs, (n, kept) = loop(c, t, rows, index, lens, st if mode == "side" else None)
            c.sync(st if mode == "side" else None)
        res.append([x.clone() for x in (*outs, n, kept, t["k"], t["v"], t["w"])])
        torch.cuda.synchronize()
        c.close()
    for other in res[1:]:
        assert all(torch.equal(x, y) for x, y in zip(res[0], other))


# ---------------------------------------------------------------- signed zeros

@pytest.mark.parametrize("budget", [50, 49, 12])
def test_evict_turns_minus_zero_into_zero(sf, budget):
    """Weights of -0 come out as 0 whether the sequence moves whole or in part,
    in place or elsewhere; NaN stays NaN."""
    heads, page, lens = (4, 2, 64), 16, [50, 7, 0]
    a = attend_inputs(sf, heads, "f32", page, lens, seed=32, track=False)
    w = torch.zeros_like(a["w"])
    w[:, :, ::2] = -0.0
    w[:, :, 3] = float("nan")
    for place in ("elsewhere", "in place"):
        w_in = w.clone()
        w_out = torch.full_like(w, -3.0) if place == "elsewhere" else w_in
        n, kept = a["c"].evict(a["k"].clone(), a["v"].clone(), i32(a["table"]), i32(lens), w_in, budget, n_first=4,
                               weights_out=w_out)
        a["c"].sync()
        assert n.tolist() == [min(x, budget) for x in lens]
        for s in range(2):
            got = w_out[s, :, :int(n[s])]
            assert torch.isnan(got[:, 3]).all()
            got = torch.cat([got[:, :3], got[:, 4:]], 1)
            assert not got.view(torch.int32).any()          # +0, bit for bit
    a["c"].close()


# ---------------------------------------------------------------- weights of large scores

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,page,lens", [((12, 2, 128), 16, [100, 37]), ((14, 2, 64), 16, [20003]),
                                             ((4, 4, 64), 16, [3 + i % 60 for i in range(300)])])
def test_weights_of_equal_large_scores(sf, heads, page, lens, dtype):
    """All keys of a sequence the same, scores around 500 (whose fp32 step is
    6e-5 in log2): every position gets 1 / len of each head.

    Equal scores are computed alike, so that every exponential is 2^0 = 1 and
    the denominator a count: exact.  What rounds is the reciprocal (1 u), the
    product (1 u) and the sum over the group's heads (G u at most)."""
    nq, nkv, hd = heads
    a = attend_inputs(sf, heads, dtype, page, lens, seed=33)
    rng = np.random.default_rng(34)
    for s, n in enumerate(lens):
        key = torch.from_numpy(rng.standard_normal((nkv, hd)).astype(np.float32)).cuda().to(a["k"].dtype)
        for c in range(-(-n // page)):
            a["k"][a["table"][s, c], :min(page, n - c * page)] = key
        reach = torch.from_numpy(rng.uniform(400, 600, (nkv, nq // nkv, 1))).cuda() * hd ** 0.5
        unit = key.double() / (key.double() ** 2).sum(-1, keepdim=True)
        a["q"][s] = (reach * unit[:, None]).reshape(nq, hd).to(a["q"].dtype)
    w = torch.zeros_like(a["w"])
    out = a["c"].attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights_out=w)
    a["c"].sync()
    G = nq // nkv
    for s, n in enumerate(lens):
        want = G / n
        assert ((w[s, :, :n].double() - want).abs() <= (G + 2) * 2.0 ** -24 * want).all()
        assert not w[s, :, n:].any()
    assert torch.isfinite(out).all()
    a["c"].close()


# ---------------------------------------------------------------- sums of long sequences

U = 2.0 ** -24
SUMS = [
    # heads, dtype, lens: chunks and the join kernel, then a line
    ((2, 1, 64), "bf16", [262144, 5]),
    ((12, 1, 128), "bf16", [262144]),
    ((2, 1, 64), "f32", [262144, 5]),
    ((10, 2, 128), "f32", [131071, 100001]),
    ((8, 8, 64), "bf16", [30000] * 25),
]


def _bounds(q, k, v, heads, tiles_of_a_warp, parts):
    """Weights, output and their bounds in float64 for one sequence, q [nkv, G, hd], k and v [n, nkv, hd].

    A term of the output is added into a warp's sum with the others of its tiles (two products of 16 keys a tile, in
    any order inside the tensor core), which is rescaled at most once a tile; then 8 warps' sums are scaled and added;
    then the parts (at most one a block), by 8 or 16 groups, then the groups' sums, each scaled; then the quotient (3
    roundings):
        D = 33 tiles + 16 + 2 (parts / 8 + 1 + 16) + 3 roundings of 2u of sum p |v| (2u: tensor cores may truncate),
    and the same for the denominator.  A score is two chains of hd / 2 products, their sum, and the scale:
        d = (hd / 2 + 4) 2u scale sum |q k|,
    which moves the output by d of sum p |v - out| <= sum p |v| + |out|, and a weight by 2 d of itself.  The
    exponential is good to 4u, and two bf16 numbers for a weight to 2^-16."""
    hd = heads[2]
    scale = hd ** -0.5
    s = torch.einsum("cgd,ncd->cgn", q, k) * scale
    p = torch.softmax(s, -1)
    out = torch.einsum("cgn,ncd->cgd", p, v)
    mag = torch.einsum("cgn,ncd->cgd", p, v.abs())
    d = (hd / 2 + 4) * 2 * U * scale * torch.einsum("cgd,ncd->cgn", q.abs(), k.abs()).amax(-1)
    D = 33 * tiles_of_a_warp + 16 + 2 * (parts / 8 + 1 + 16) + 3
    r = 2 * D * 2 * U + 4 * U + 2.0 ** -16
    return p, out, d[..., None] * (mag + out.abs()) + r * mag, 2 * d + r


@pytest.mark.parametrize("heads,dtype,lens", SUMS)
def test_sums_of_long_sequences(sf, heads, dtype, lens):
    """Outputs and weights within a bound over the real depth of the sums, which
    does not let pass an output of zeros or one that lacks a block's keys."""
    from test_gpu_cache import DT, E, make_pages
    nq, nkv, hd = heads
    page, G = 64, nq // nkv
    table, total = make_pages(np.random.default_rng(8), lens, page)
    g = torch.Generator("cuda").manual_seed(4)
    k, v = (torch.randn((total, page, nkv, hd), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = (2 * torch.randn((len(lens), nq, hd), generator=g, device="cuda")).to(DT[dtype])
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(lens),
                      max_len=max(lens), max_pos=16, track_weights=True)
    w = torch.zeros((len(lens), nkv, max(lens)), device="cuda")
    out = c.attend(q, k, v, i32(table), i32(lens), weights=w)
    c.sync()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = sum(-(-n // 16) for n in lens) * nkv
    # a block takes at most an even share, rounded up, and 64 tiles; a warp takes every eighth tile of a segment
    share = -(-units // sms) + 64
    e = E[dtype]
    for s in sorted({0, 1, len(lens) - 1} & set(range(len(lens)))):
        n = lens[s]
        idx = np.arange(n)
        slot = torch.from_numpy(table[s, idx // page].astype(np.int64) * page + idx % page).cuda()
        ks, vs = (x.view(-1, nkv, hd)[slot].double() for x in (k, v))
        per_block = min(-(-n // 16), share)
        p, ref, tol, rel = _bounds(q[s].double().view(nkv, G, hd), ks, vs, heads, -(-per_block // 8), sms)
        tol = tol * (1 + e) + e * ref.abs()
        err = (out[s].double().view(nkv, G, hd) - ref).abs()
        assert (err <= tol).all(), (err - tol).max().item()
        want = p.sum(1)
        werr = (w[s, :, :n].double() - want).abs()
        assert (werr <= (p * rel[..., None]).sum(1) + G * U * want).all()
        assert not w[s, :, n:].any()
        if n < 1000:
            continue
        # mistakes that the bound has to see, made in the reference
        assert not (ref.abs() <= tol).all()
        for lost in (slice(0, n // 200), slice(n // 2, n // 2 + n // 200)):
            part = p.clone()
            part[..., lost] = 0
            less = torch.einsum("cgn,ncd->cgd", part / part.sum(-1, keepdim=True), vs)
            assert not ((less - ref).abs() <= tol).all()
            assert not ((part.sum(1) - want).abs() <= (p * rel[..., None]).sum(1) + G * U * want).all()
    c.close()


# ---------------------------------------------------------------- short sequences in objects for long ones

@pytest.mark.parametrize("heads,dtype,lens", [((12, 2, 128), "bf16", [512]), ((40, 8, 128), "bf16", [1000, 0, 1, 2000]),
                                              ((4, 2, 64), "f32", [700, 33]), ((8, 8, 64), "bf16", [60] * 40)])
def test_attend_in_an_object_for_long_sequences(sf, heads, dtype, lens):
    """An object and a table for 262,144 positions: the launch is planned for
    those, the sequences are far shorter."""
    page = 64
    a = attend_inputs(sf, heads, dtype, page, lens, seed=35, cols=4096)
    a["c"].close()
    nq, nkv, hd = heads
    a["c"] = c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page,
                               max_seqs=len(lens), max_len=262144, max_pos=16, track_weights=True)
    w = torch.zeros((len(lens), nkv, 262144), device="cuda")
    out = c.attend(a["q"], a["k"], a["v"], i32(a["table"]), i32(lens), weights=w)
    # a table cut to the columns that the batch needs plans the call for those, whatever the object holds
    cols = -(-max(lens) // page)
    less = c.attend(a["q"], a["k"], a["v"], i32(a["table"])[:, :cols], i32(lens))
    c.sync()
    check_attend(heads, dtype, page, a, out, w, w_in=torch.zeros_like(w))
    check_attend(heads, dtype, page, a, less, None)
    assert not out[[s for s, n in enumerate(lens) if n == 0]].any()
    c.close()


@pytest.mark.parametrize("kind", ["spread", "few values", "equal", "any"])
@pytest.mark.parametrize("heads,lens,budget", [((1, 1, 64), [9000, 8999, 300], 4000), ((1, 1, 64), [300, 40, 269], 20),
                                               ((2, 2, 64), [5, 9, 0, 33], 4), ((2, 2, 64), [2047] * 6, 1000)])
def test_evict_in_an_object_for_long_sequences(sf, monkeypatch, heads, lens, budget, kind):
    """Clusters of eight blocks with tables for 262,144 positions: few weights a
    block, or none in most of them."""
    import test_gpu_cache_batches as batches
    make = batches.make_pages
    monkeypatch.setattr(batches, "make_pages", lambda rng, lens, page, cols=None: make(rng, lens, page, cols=cols or 4096))
    batches.run_evict(sf, 7, heads, "bf16", 64, lens, budget, 1, 2, kind, max_len=262144)
