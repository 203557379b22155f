"""Rotary forms of append, and keys moved to other positions, against float64
(needs a GB300).

Tolerances, u = 2^-24 and e the half step of the type: a normalised element is
good to 20 u, the rotated value x cos - y sin to 4 u more of |x| + |y| (append's
own derivation), times the magnitude m:
    append:      24 u m (|x| + |y|) (1 + e) + e |ref|
    reposition:  cosine and sine are the table's (1 u), times 1 / m (1 u each
                 for the quotient and the product): 8 u (|x| + |y|) (1 + e) + e |ref|."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import cache as oc
from test_gpu_cache import DT, E, U, f64, i32, make_pages, pool, sf  # noqa: F401

pytestmark = pytest.mark.gpu


def pair_sums(n, dim, layout):
    """|a| + |b| of every dimension's pair, |x| of dimensions that are not turned."""
    m = np.abs(n).copy()
    h = dim // 2
    if layout == "half":
        m[..., :h], m[..., h:dim] = (np.abs(n[..., :h]) + np.abs(n[..., h:dim]),) * 2
    else:
        m[..., 0:dim:2], m[..., 1:dim:2] = (np.abs(n[..., 0:dim:2]) + np.abs(n[..., 1:dim:2]),) * 2
    return m


def within(got, want, tol):
    """Infinite where that is wanted, and as near as tol everywhere else."""
    fine = np.isfinite(want)
    return np.array_equal(got[~fine], want[~fine]) and np.all(np.abs(got[fine] - want[fine]) <= tol[fine])


FORMS = [
    # heads, dtype, page, new rows, norm, layout, dim, magnitude
    ((4, 2, 64), "f32", 16, [1], False, "half", 16, 1.0),
    ((4, 2, 64), "f32", 24, [5, 1, 100], True, "interleaved", 64, 1.0),
    ((12, 2, 128), "bf16", 32, [1], True, "interleaved", 128, 1.2),
    ((12, 2, 128), "bf16", 32, [3, 70], True, "half", 64, 1.0),
    ((28, 4, 128), "bf16", 7, [40, 1], True, "half", 96, 0.7),
    ((40, 8, 128), "bf16", 32, [33, 130, 1], False, "interleaved", 32, 1.0),
    ((10, 5, 128), "f32", 1, [5, 3], True, "half", 48, 1.3),
    ((16, 1, 128), "bf16", 100, [257], True, "interleaved", 112, 1.0),
    ((8, 8, 64), "bf16", 64, [777], True, "half", 48, 1.0),
    ((8, 8, 64), "bf16", 64, [777], False, "half", 64, 1.1),
    ((3, 1, 64), "f32", 5, [11], False, "interleaved", 16, 1.0),
    ((40, 8, 128), "bf16", 16, [2500], True, "half", 16, 1.0),
    ((40, 8, 128), "f32", 16, [1500], True, "interleaved", 80, 1.0),
]


@pytest.mark.parametrize("heads,dtype,page,new,norm,layout,dim,magnitude", FORMS)
def test_append_forms(sf, heads, dtype, page, new, norm, layout, dim, magnitude):
    nq, nkv, hd = heads
    rng = np.random.default_rng([dim, page, sum(new)])
    table, total = make_pages(rng, new, page)
    freq = oc.frequencies(dim, 10000.0, 3.7)
    far = 50000
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(new),
                      max_len=max(new), max_pos=max(new) + far, rotary_dim=dim, rotary_layout=layout, inv_freq=freq,
                      rotary_magnitude=magnitude)
    seq = np.repeat(np.arange(len(new)), new)
    index = np.concatenate([np.arange(b) for b in new])
    pos = index + far * (index % 2)
    T = len(seq)
    qkv = torch.from_numpy(rng.standard_normal((T, nq + 2 * nkv, hd)).astype(np.float32)).cuda().to(DT[dtype])
    if dim < hd and not norm:
        qkv[T // 2, :, dim] = torch.inf                              # not turned: reaches nothing else
    gq, gk = ((torch.from_numpy(1 + 0.3 * rng.standard_normal(hd)).float().cuda() for _ in range(2)) if norm
              else (None, None))
    k, v = (pool(rng, total, page, nkv, hd, dtype) for _ in range(2))
    wk, wv = f64(k).reshape(-1, nkv, hd), f64(v).reshape(-1, nkv, hd)
    q = c.append(qkv, i32(index), i32(table), k, v, pos=i32(pos), seq=i32(seq), q_gain=gq, k_gain=gk)
    c.sync()
    x, e = f64(qkv), E[dtype]
    parts = []
    for sl, gain in ((slice(0, nq), gq), (slice(nq, nq + nkv), gk)):
        n = oc.head_norm(x[:, sl], None if gain is None else f64(gain), 1e-6)
        ref = oc.turn(n, pos[:, None], freq, layout, magnitude)
        tol = 24 * U * max(magnitude, 1) * pair_sums(n, dim, layout) * (1 + e) + e * np.abs(ref)
        parts.append((ref, tol))
    assert within(f64(q), *parts[0])
    slot = table[seq, index // page] * page + index % page
    tk = np.zeros_like(wk)
    wk[slot], tk[slot] = parts[1]
    wv[slot] = x[:, nq + nkv:]
    assert within(f64(k).reshape(wk.shape), wk, tk)
    assert np.array_equal(f64(v).reshape(wv.shape), wv)
    # in place of the query part of the rows, the same bits
    packed = qkv.clone()
    q2 = c.append(packed, i32(index), i32(table), k, v, pos=i32(pos), seq=i32(seq), q_gain=gq, k_gain=gk,
                  q=packed[:, :nq])
    assert torch.equal(q2, q)
    c.close()


def test_plain_rotation_is_what_it_was(sf):
    """The default form, and the same by its options: bit for bit."""
    rng = np.random.default_rng(1)
    table, total = make_pages(rng, [300], 16)
    qkv = torch.randn((300, 16, 128), device="cuda").to(torch.bfloat16)
    got = []
    for kw in ({}, dict(rotary_dim=128, rotary_layout="half", rotary_magnitude=1.0)):
        c = sf.PagedCache(n_q_heads=12, n_kv_heads=2, head_dim=128, dtype="bf16", page_size=16, max_seqs=1, max_len=300, **kw)
        k, v = (torch.zeros((total, 16, 2, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        q = c.append(qkv, i32(np.arange(300)), i32(table), k, v, seq=i32(np.zeros(300)))
        c.sync()
        got.append((q, k, v))
        c.close()
    assert all(torch.equal(x, y) for x, y in zip(*got))


TURN = [
    # heads, dtype, page, lens, layout, dim, magnitude
    ((4, 2, 64), "f32", 16, [1], "half", 64, 1.0),
    ((4, 2, 64), "f32", 24, [0, 5, 100], "interleaved", 32, 1.3),
    ((12, 2, 128), "bf16", 32, [1024], "half", 128, 1.0),
    ((40, 8, 128), "bf16", 7, [33, 0, 500, 31, 32], "half", 96, 0.6),
    ((10, 5, 128), "bf16", 100, [257, 1], "interleaved", 128, 1.0),
    ((8, 8, 64), "bf16", 1, [65], "interleaved", 16, 1.0),
    ((16, 1, 128), "f32", 64, [2000], "half", 16, 1.0),
    ((16, 1, 128), "f32", 64, [3, 4000], "interleaved", 112, 2.0),
]


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("heads,dtype,page,lens,layout,dim,magnitude", TURN)
def test_reposition(sf, heads, dtype, page, lens, layout, dim, magnitude, given):
    nq, nkv, hd = heads
    rng = np.random.default_rng([dim, page, sum(lens)])
    table, total = make_pages(rng, lens, page)
    top, far = max(lens), 70000
    freq = oc.frequencies(dim, 500.0)
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=len(lens),
                      max_len=top, max_pos=far, rope_theta=500.0, rotary_dim=dim, rotary_layout=layout,
                      rotary_magnitude=magnitude)
    k = pool(rng, total, page, nkv, hd, dtype)
    before = f64(k).reshape(-1, nkv, hd)
    S, ld = len(lens), top + 3
    frm, to = (rng.integers(0, far, (S, nkv, ld)).astype(np.int32) for _ in range(2))
    frm[rng.random(frm.shape) < 0.1] = -1                            # left alone
    if given:
        to[rng.random(to.shape) < 0.1] = -2 ** 31
    else:
        to[:] = np.arange(ld)
    c.reposition(k, i32(table), i32(lens), i32(frm), pos_to=i32(to) if given else None)
    c.sync()
    want, tol, e = before.copy(), np.zeros_like(before), E[dtype]
    for s, n in enumerate(lens):
        for h in range(nkv):
            j = np.arange(n)
            j = j[(frm[s, h, :n] >= 0) & (to[s, h, :n] >= 0)]
            slot = table[s, j // page] * page + j % page
            x = before[slot, h]
            steps = to[s, h, j].astype(np.int64) - frm[s, h, j]
            want[slot, h] = oc.turn(x[:, None], steps[:, None], freq, layout)[:, 0]
            t = tol[slot, h]
            t[:, :dim] = (8 * U * pair_sums(x, dim, layout) * (1 + e) + e * np.abs(want[slot, h]))[:, :dim]
            tol[slot, h] = t
    assert np.all(np.abs(f64(k).reshape(want.shape) - want) <= tol)
    c.close()


def test_reposition_reports(sf):
    page = 16
    rng = np.random.default_rng(0)
    table, total = make_pages(rng, [40, 40], page)
    c = sf.PagedCache(n_q_heads=4, n_kv_heads=2, head_dim=64, dtype="f32", page_size=page, max_seqs=2, max_len=60, max_pos=100)
    k0 = pool(rng, total, page, 2, 64, "f32")
    frm = rng.integers(0, 100, (2, 2, 45)).astype(np.int32)

    def run(table=table, lens=(40, 40), frm=frm, to=None):
        k = k0.clone()
        c.reposition(k, i32(table), i32(list(lens)), i32(frm), pos_to=None if to is None else i32(to))
        return k

    good = run()
    c.sync()

    def reported(text):
        with pytest.raises(sf.SpecFoldError) as e:
            c.sync()
        assert e.value.status == sf.SF_ERR_DEVICE_ASSERT and text in str(e.value)

    pages0, pages1 = (torch.as_tensor(table[s, :3].astype(np.int64), device="cuda") for s in (0, 1))
    for n in (-1, 46, 2 ** 31 - 1):                                  # beyond the positions that are given
        k = run(lens=(40, n))
        reported("length")
        assert torch.equal(k[pages1], k0[pages1])
        assert torch.equal(k[pages0], good[pages0])
    for bad in (100, 2 ** 31 - 1):
        for side in ("from", "to"):
            f = frm.copy()
            t = np.tile(np.arange(45, dtype=np.int32), (2, 2, 1))
            (f if side == "from" else t)[0, 1, 5] = bad
            k = run(frm=f, to=t)
            reported("row")
            page0 = int(table[0, 0])
            assert torch.equal(k[page0, 5, 1], k0[page0, 5, 1])
            k[page0, 5, 1] = good[page0, 5, 1]
            assert torch.equal(k, good)
    t = table.copy()
    t[1, 2] = total
    k = run(table=t)
    reported("page")
    assert torch.equal(k[int(table[1, 2])], k0[int(table[1, 2])])
    assert torch.equal(k[pages1[:2]], good[pages1[:2]])
    c.close()


def test_reposition_far_and_replayed(sf):
    """Differences up to the largest, captured on a side stream and replayed with other positions and lengths; turned
    back, a key is what it was but for two roundings."""
    far, page, hd = 4194304, 16, 64
    rng = np.random.default_rng(3)
    c = sf.PagedCache(n_q_heads=2, n_kv_heads=1, head_dim=hd, dtype="f32", page_size=page, max_seqs=2, max_len=40,
                      max_pos=far, rotary_dim=16)
    table, total = make_pages(rng, [40, 40], page)
    first = pool(rng, total, page, 1, hd, "f32")
    k, t, lens = first.clone(), i32(table), i32([40, 40])
    frm, to = (torch.zeros((2, 1, 40), dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.reposition(k, t, lens, frm, pos_to=to)
    freq = oc.frequencies(16, 10000.0)
    for n in ([40, 40], [40, 0], [1, 33]):
        f, x = rng.integers(0, far, (2, 2, 1, 40))
        f[:, :, 0], x[:, :, 0] = 0, far - 1                          # the largest difference
        for a, b in ((frm, f), (to, x)):
            a.copy_(i32(b))
        lens.copy_(i32(n))
        k.copy_(first)
        g.replay()
        c.sync()
        want = f64(first).reshape(-1, hd)
        tol = np.zeros_like(want)
        for s in range(2):
            j = np.arange(n[s])
            slot = table[s, j // page] * page + j % page
            old = want[slot]
            want[slot] = oc.turn(old[:, None], (x - f)[s, 0, j][:, None], freq, "half")[:, 0]
            tol[slot, :16] = (8 * U * pair_sums(old, 16, "half") * (1 + U) + U * np.abs(want[slot]))[:, :16]
        got = f64(k).reshape(-1, hd)
        assert np.all(np.abs(got - want) <= tol)
        frm.copy_(i32(x))
        to.copy_(i32(f))
        g.replay()
        c.sync()
        # back: the first error carried over (a rotation keeps lengths: of a and b together), the same again
        back = np.abs(f64(k) - f64(first)).reshape(-1, hd)
        sums = pair_sums(f64(first).reshape(-1, hd), 16, "half")[:, :16]
        assert np.all(back[:, :16] <= 4 * 9 * U * sums) and not back[:, 16:].any()
    c.close()


def test_evicted_context_becomes_a_prefix(sf):
    """append, attend with weights, evict into dense pages, reposition: keys rotated at 0..budget-1, which the
    verification pass reads; the pass's own oracle on those keys agrees with it."""
    n, budget, page = 96, 64, 16
    cfg = synth.small_config(name="evicted", n_layers=1, d_model=256, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ffn=320,
                             dtype="f32", block_len=32, prefix_len=budget, n_drafts=2)
    R = cfg.n_requests
    wl = synth.make_workload(cfg, seed=4, device="cuda:0")
    rng = np.random.default_rng(8)
    c = sf.PagedCache(n_q_heads=4, n_kv_heads=2, head_dim=64, dtype="f32", page_size=page, max_seqs=R, max_len=n,
                      track_weights=True)
    table, total = make_pages(rng, [n] * R, page)
    k, v = (torch.zeros((total, page, 2, 64), device="cuda") for _ in range(2))
    qkv = torch.randn((R * n, 8, 64), device="cuda")
    seq, index = np.repeat(np.arange(R), n), np.tile(np.arange(n), R)
    c.append(qkv, i32(index), i32(table), k, v, seq=i32(seq))
    w = torch.zeros((R, 2, n), device="cuda")
    c.attend(torch.randn((R, 4, 64), device="cuda"), k, v, i32(table), i32([n] * R), weights=w)
    pk, pv = (torch.zeros((1, R, budget, 2, 64), device="cuda") for _ in range(2))
    dense = np.arange(R * budget // page, dtype=np.int32).reshape(R, -1)
    lens, kept = c.evict(k, v, i32(table), i32([n] * R), w, budget, n_first=4, n_recent=8, k_out=pk.view(-1, page, 2, 64),
                         v_out=pv.view(-1, page, 2, 64), table_out=i32(dense))
    c.reposition(pk.view(-1, page, 2, 64), i32(dense), lens, kept)
    c.sync()
    x, kept = f64(qkv).reshape(R, n, 8, 64), kept.cpu().numpy()
    for r in range(R):
        for h in range(2):
            raw = x[r, kept[r, h], 4 + h]
            want = oc.rotate(raw[:, None], np.arange(budget), 10000.0)[:, 0]
            # two rotations of fp32: each 4 u of |a| + |b|, and a rounding
            tol = 16 * U * pair_sums(raw, 64, "half") + 2 * U * np.abs(want)
            assert np.all(np.abs(f64(pk[0, r, :, h]) - want) <= tol)
            assert np.array_equal(f64(pv[0, r, :, h]), x[r, kept[r, h], 6 + h])
    ctx = sf.from_config(cfg, wl.weights)
    out, *_ = ctx.verify(wl.hidden, wl.parents, pk, pv, 0.0)
    ctx.sync()
    W = [oracle.layer_weights_f64(l) for l in wl.weights]
    ref = oracle.verify_pass(f64(wl.hidden), wl.parents, 0.0, lambda l: W[l], f64(pk), f64(pv), cfg)["out"]
    got = f64(out).reshape(-1, cfg.d_model)
    ref = ref.reshape(got.shape)
    # the pass's own bound for fp32 (tests/parity.py)
    assert np.max(np.abs(got - ref).max(1) / np.maximum(np.abs(ref).max(1), 1e-6)) <= 1e-4
    ctx.close()
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_keys_that_keep_their_position_keep_their_bits(sf, dtype, layout):
    """No rotation by nothing: not the rounding of a magnitude and its reciprocal, no NaN beside an infinite value; the
    keys that do move are turned as ever."""
    nkv, hd, page, n, magnitude = 2, 64, 16, 200, 1.3
    rng = np.random.default_rng(8)
    table, total = make_pages(rng, [n], page)
    c = sf.PagedCache(n_q_heads=4, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=1, max_len=n,
                      max_pos=5000, rotary_dim=48, rotary_layout=layout, rotary_magnitude=magnitude)
    k = pool(rng, total, page, nkv, hd, dtype)
    frm = np.tile(np.arange(n, dtype=np.int32), (1, nkv, 1))
    moved = rng.random((nkv, n)) < 0.3
    frm[0][moved] += rng.integers(1, 4000, int(moved.sum())).astype(np.int32)
    slot = table[0, np.arange(n) // page] * page + np.arange(n) % page
    flat = k.view(-1, nkv, hd)
    for h in range(nkv):
        for x, value in zip(np.flatnonzero(~moved[h])[:2], (np.inf, -0.0)):
            flat[int(slot[x]), h, 5] = value
    before, first = f64(k).reshape(-1, nkv, hd), k.clone()
    for pos_to in (None, i32(np.tile(np.arange(n, dtype=np.int32), (1, nkv, 1)))):
        k.copy_(first)
        c.reposition(k, i32(table), i32([n]), i32(frm), pos_to=pos_to)
        c.sync()
        got, bits, same = f64(k).reshape(-1, nkv, hd), torch.int16 if dtype == "bf16" else torch.int32, first.clone()
        for h in range(nkv):
            at = slot[moved[h]]
            x = before[at, h]
            want = oc.turn(x[:, None], (np.arange(n)[moved[h]] - frm[0, h][moved[h]])[:, None], oc.frequencies(48, 10000.0),
                           layout)[:, 0]
            tol = 8 * U * pair_sums(x, 48, layout) * (1 + E[dtype]) + E[dtype] * np.abs(want)
            assert np.all(np.abs(got[at, h] - want) <= tol)
            same.view(-1, nkv, hd)[torch.as_tensor(at), h] = flat[torch.as_tensor(at), h]
        assert torch.equal(k.view(bits), same.view(bits))
    c.close()
