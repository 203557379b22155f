"""The paged-cache operators over random batches (needs a GB300): how the work
is cut over the GPU depends on the batch, so every way of cutting is met here
(a block per segment, equal parts of a line, a warp per short segment, joins in
place and by a kernel, clusters, narrow and wide selection blocks), the largest
objects, and the longest sequences.

References are float64 torch on the GPU, sequence by sequence; tolerances are
those derived in test_gpu_cache.py, with each bound taken per sequence and head
(its largest score error) rather than per key."""
import numpy as np
import pytest
import torch

from test_gpu_cache import DT, E, U, i32, make_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


def gather(pages, table_row, n, page):
    idx = np.arange(n)
    slot = torch.from_numpy(table_row[idx // page].astype(np.int64) * page + idx % page).cuda()
    return pages.view(-1, *pages.shape[2:])[slot]


def check_sequence(q, k, v, out, w, w_in, scale, dtype):
    """One sequence: q [nq, hd], k / v [n, nkv, hd], out [nq, hd], w [nkv, n] or None."""
    nq, nkv, n, hd = q.shape[0], k.shape[1], k.shape[0], q.shape[1]
    G, e = nq // nkv, E[dtype]
    q, k, v, out = (t.double() for t in (q, k, v, out))
    qg = q.view(nkv, G, hd)
    s = torch.einsum("cgd,ncd->cgn", qg, k) * scale
    p = torch.softmax(s, -1)
    ref = torch.einsum("cgn,ncd->cgd", p, v)
    d = (hd + 4) * 2 * U * abs(scale) * torch.einsum("cgd,ncd->cgn", qg.abs(), k.abs()).amax(-1)   # [c, g]
    r = 2 * d + 4 * (n + 64) * U + 8 * U + 2.0 ** -16
    tol = r[..., None] * torch.einsum("cgn,ncd->cgd", p, v.abs()) * (1 + e) + e * ref.abs()
    err = (out.view(nkv, G, hd) - ref).abs()
    assert (err <= tol).all(), ((err - tol).max().item(), n)
    if w is not None:
        full = w_in.double() + p.sum(1)
        werr = (w.double() - full).abs()
        wtol = (r[..., None] * p).sum(1) + (G + 1) * U * full.abs()
        assert (werr <= wtol).all(), ((werr - wtol).max().item(), n)


def random_lens(rng, kind, S, top):
    if kind == "even":
        lens = np.full(S, top)
    elif kind == "short":
        lens = rng.integers(0, 65, S)
    elif kind == "one long":
        lens = rng.integers(0, 50, S)
        lens[rng.integers(S)] = top
    elif kind == "mostly empty":
        lens = rng.integers(1, top + 1, S) * (rng.random(S) < 0.1)
    else:
        lens = rng.integers(0, top + 1, S)
    return [int(x) for x in lens]


HEADS = [(4, 2, 64), (12, 2, 128), (28, 4, 128), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (10, 5, 128),
         (24, 1, 64), (1, 1, 64)]
KINDS = ["even", "short", "one long", "mostly empty", "any"]


@pytest.mark.parametrize("seed", range(40))
def test_attend_random_batches(sf, seed):
    rng = np.random.default_rng([seed, 4242])
    nq, nkv, hd = heads = HEADS[seed % len(HEADS)]
    kind = KINDS[(seed // 2) % len(KINDS)]
    dtype = "f32" if seed % 4 == 3 else "bf16"
    page = int(rng.choice([1, 3, 16, 17, 32, 64, 250]))
    S = int(np.exp(rng.uniform(0, np.log(400))))
    top = int(np.exp(rng.uniform(np.log(30), np.log(min(30000, 1.5e8 / (S * nkv * hd))))))
    lens = random_lens(rng, kind, S, top)
    table, total = make_pages(rng, lens, page, cols=-(-max(top, 64) // page) + int(rng.integers(0, 3)))
    g = torch.Generator("cuda").manual_seed(seed)
    k, v = (torch.randn((total, page, nkv, hd), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = (2 * torch.randn((S, nq, hd), generator=g, device="cuda")).to(DT[dtype])
    track = seed % 3 != 0
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=S + 3,
                      max_len=max(top, 64) + 5, track_weights=track)
    w = torch.rand((S, nkv, max(top, 64) + 7), generator=g, device="cuda") if track else None
    w_out = torch.full_like(w, -1.0) if track else None
    for _ in range(2):                              # the workspace is left as it was found
        out = c.attend(q, k, v, i32(table), i32(lens), weights=w, weights_out=w_out)
    c.sync()
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any()
        else:
            check_sequence(q[s], gather(k, table[s], n, page), gather(v, table[s], n, page), out[s],
                           w_out[s, :, :n] if track else None, w[s, :, :n] if track else None, hd ** -0.5, dtype)
        if track:
            assert torch.all(w_out[s, :, n:] == -1.0)
    c.close()


@pytest.mark.parametrize("heads,dtype", [((2, 1, 64), "bf16"), ((12, 1, 128), "bf16"), ((2, 1, 64), "f32")])
def test_attend_longest_sequence(sf, heads, dtype):
    """262,144 positions, the most an object takes."""
    nq, nkv, hd = heads
    n, page = 262144, 64
    rng = np.random.default_rng(7)
    table, total = make_pages(rng, [n, 5], page)
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((total, page, nkv, hd), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = (2 * torch.randn((2, nq, hd), generator=g, device="cuda")).to(DT[dtype])
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=2, max_len=n,
                      max_pos=16, track_weights=True)
    w = torch.zeros((2, nkv, n), device="cuda")
    out = c.attend(q, k, v, i32(table), i32([n, 5]), weights=w)
    c.sync()
    for s, m in ((0, n), (1, 5)):
        check_sequence(q[s], gather(k, table[s], m, page), gather(v, table[s], m, page), out[s], w[s, :, :m],
                       torch.zeros_like(w[s, :, :m]), hd ** -0.5, dtype)
    c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_most_sequences(sf, dtype):
    """4,096 sequences, the most an object takes."""
    heads, page, S = (2, 2, 128), 8, 4096
    rng = np.random.default_rng(9)
    lens = random_lens(rng, "any", S, 40)
    lens[4095], lens[17] = 700, 0
    table, total = make_pages(rng, lens, page)
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn((total, page, 2, 128), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = torch.randn((S, 2, 128), generator=g, device="cuda").to(DT[dtype])
    c = sf.PagedCache(n_q_heads=2, n_kv_heads=2, head_dim=128, dtype=dtype, page_size=page, max_seqs=S, max_len=700,
                      track_weights=True)
    w = torch.zeros((S, 2, 700), device="cuda")
    out = c.attend(q, k, v, i32(table), i32(lens), weights=w)
    c.sync()
    for s in list(range(0, S, 37)) + [4095]:
        if lens[s]:
            check_sequence(q[s], gather(k, table[s], lens[s], page), gather(v, table[s], lens[s], page), out[s],
                           w[s, :, :lens[s]], torch.zeros_like(w[s, :, :lens[s]]), 128 ** -0.5, dtype)
        else:
            assert not out[s].any()
    c.close()


# ---------------------------------------------------------------- eviction

def reference_choice(w, n, budget, n_first, n_recent):
    """Kept positions by a sort: heaviest first, NaN last, ties to the lower index."""
    if n <= budget:
        return np.arange(n)
    rest = np.arange(n_first, n - n_recent)
    x = w[rest].astype(np.float64) + 0.0
    order = np.lexsort((rest, -np.where(np.isnan(x), 0, x), np.isnan(x)))
    best = rest[order[:budget - n_first - n_recent]]
    return np.sort(np.concatenate([np.arange(n_first), best, np.arange(n - n_recent, n)]))


def evict_weights(rng, shape, kind):
    if kind == "spread":
        w = np.exp(3 * rng.standard_normal(shape))
        w[rng.random(shape) < 0.2] = 0
    elif kind == "few values":
        w = rng.integers(0, 5, shape) / 4.0
    elif kind == "equal":
        w = np.full(shape, rng.choice([0.0, 0.25, -1.0]))
    elif kind == "close":                            # all in one first bin
        w = 1.0 + rng.random(shape) * 1e-2
    elif kind == "few above zero":
        w = np.where(rng.random(shape) < 0.02, rng.random(shape), 0.0)
    else:
        w = rng.standard_normal(shape) * 10.0 ** rng.integers(-44, 38, shape)
        for x in (np.nan, np.inf, -np.inf, 0.0, -0.0):
            w[rng.random(shape) < 0.03] = x
    return w.astype(np.float32)


WEIGHTS = ["spread", "few values", "equal", "close", "few above zero", "any"]


def run_evict(sf, seed, heads, dtype, page, lens, budget, n_first, n_recent, kind, max_len=None):
    nq, nkv, hd = heads
    rng = np.random.default_rng([seed, 99])
    S, top = len(lens), max(1, max(lens))
    table, total = make_pages(rng, lens, page)
    g = torch.Generator("cuda").manual_seed(seed)
    k, v = (torch.randn((total, page, nkv, hd), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    # weights cover what the object and the table could address
    wn = evict_weights(rng, (S, nkv, max(top, min(max_len or 0, table.shape[1] * page)) + 3), kind)
    w = torch.from_numpy(wn).cuda()
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype=dtype, page_size=page, max_seqs=S,
                      max_len=max_len or max(top, budget), max_pos=1)
    kept_ref = [[reference_choice(wn[s, h, :n], n, budget, n_first, n_recent) for h in range(nkv)]
                for s, n in enumerate(lens)]
    out_lens = [min(n, budget) for n in lens]
    table_out, total_out = make_pages(rng, out_lens, page, cols=-(-budget // page) + 1)
    for place in ("other pages", "in place"):
        if place == "other pages":
            k_out, v_out = (torch.full((total_out, page, nkv, hd), 3.0, device="cuda", dtype=DT[dtype])
                            for _ in range(2))
            w_out, t_out, ln = torch.full_like(w, 5.0), table_out, i32(lens)
            lens_out, kept = c.evict(k, v, i32(table), ln, w, budget, n_first=n_first, n_recent=n_recent, k_out=k_out,
                                     v_out=v_out, table_out=i32(t_out), weights_out=w_out)
            want_tail = 5.0
        else:
            k_out, v_out, w_out, t_out, ln = k.clone(), v.clone(), w.clone(), table, i32(lens)
            lens_out, kept = c.evict(k_out, v_out, i32(table), ln, w_out, budget, n_first=n_first, n_recent=n_recent,
                                     lens_out=ln)
        c.sync()
        assert lens_out.tolist() == out_lens
        kn, wo = kept.cpu().numpy(), w_out.cpu().numpy()
        for s, n in enumerate(lens):
            m = out_lens[s]
            src_k, src_v = gather(k, table[s], n, page), gather(v, table[s], n, page)
            got_k, got_v = gather(k_out, t_out[s], m, page), gather(v_out, t_out[s], m, page)
            for h in range(nkv):
                ids = kept_ref[s][h]
                assert np.array_equal(kn[s, h, :m], ids) and np.all(kn[s, h, m:] == -1), (s, h)
                assert np.array_equal(wo[s, h, :m], wn[s, h, ids], equal_nan=True)
                assert not wo[s, h, m:n].any()
                if place == "other pages":
                    assert np.all(wo[s, h, n:] == want_tail)
                t = torch.from_numpy(ids).cuda()
                assert torch.equal(got_k[:, h], src_k[t, h]) and torch.equal(got_v[:, h], src_v[t, h])
    c.close()


@pytest.mark.parametrize("seed", range(36))
def test_evict_random_batches(sf, seed):
    rng = np.random.default_rng([seed, 2024])
    heads = HEADS[seed % len(HEADS)]
    nkv, hd = heads[1:]
    S = int(np.exp(rng.uniform(0, np.log(60))))
    top = int(np.exp(rng.uniform(np.log(2), np.log(min(20000, 2e7 / (S * nkv * hd)) + 2))))
    lens = random_lens(rng, ["any", "even", "one long", "short"][seed % 4], S, top)
    budget = int(rng.integers(1, max(lens) + 2))
    n_first = int(rng.integers(0, budget + 1)) if seed % 2 else 0
    n_recent = int(rng.integers(0, budget - n_first + 1)) if seed % 3 else 0
    run_evict(sf, seed, heads, "f32" if seed % 5 == 4 else "bf16", int(rng.choice([1, 7, 16, 32, 100])), lens, budget,
              n_first, n_recent, WEIGHTS[seed % len(WEIGHTS)])


@pytest.mark.parametrize("kind", WEIGHTS)
@pytest.mark.parametrize("lens,budget,max_len", [([32768], 5000, None), ([32769, 100], 32768, None),
                                                 ([70001], 65536, None), ([262144], 100000, None),
                                                 ([9000, 8999, 300], 4000, 262144), ([16384] * 40, 257, None),
                                                 ([300, 40, 271, 269, 270], 20, 262144), ([16384] * 3, 14, None)])
def test_evict_long_rows(sf, lens, budget, max_len, kind):
    """Rows at the limits of one block and of a cluster, and short rows of an object for long ones."""
    run_evict(sf, 5, (1, 1, 64), "bf16", 64, lens, budget, 3, 11, kind, max_len)


def test_evict_crowd_of_short_rows(sf):
    """More (sequence, head) pairs than resident blocks."""
    rng = np.random.default_rng(1)
    run_evict(sf, 6, (8, 8, 64), "f32", 4, random_lens(rng, "short", 120, 64), 20, 2, 3, "few values")


# ---------------------------------------------------------------- pools beyond 32-bit offsets

def test_pools_beyond_32_bit_offsets(sf):
    """Pools of 2.2 * 10^9 elements (4.3 GB each): a sequence on their last pages
    gets the bits that it gets on a small pool's."""
    nq, nkv, hd, page, n_pages = 8, 8, 128, 64, 33000
    assert n_pages * page * nkv * hd > 2 ** 31
    rng = np.random.default_rng(3)
    lens, new = [500, 90], [40, 3]
    need = [-(-n // page) for n in lens]
    small = np.full((2, max(need)), 2 ** 30, np.int32)
    big = small.copy()
    small[0, :need[0]], small[1, :need[1]] = np.arange(need[0]), need[0] + np.arange(need[1])
    big[0, :need[0]] = n_pages - 1 - np.arange(need[0]) * 2
    big[1, :need[1]] = n_pages - 40 - np.arange(need[1])
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype="bf16", page_size=page, max_seqs=2, max_len=500,
                      track_weights=True)
    index = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    seq = i32(np.repeat([0, 1], new))
    g = torch.Generator("cuda").manual_seed(1)
    rows = torch.randn((sum(new), nq + 2 * nkv, hd), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((2, nq, hd), generator=g, device="cuda").to(torch.bfloat16)
    k0, v0 = (torch.randn((sum(need), page, nkv, hd), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    got = []
    for table, total in ((small, sum(need)), (big, n_pages)):
        k, v = (torch.zeros((total, page, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for s in range(2):
            where = torch.from_numpy(table[s, :need[s]].astype(np.int64)).cuda()
            first = torch.from_numpy(small[s, :need[s]].astype(np.int64)).cuda()
            k[where], v[where] = k0[first], v0[first]
        t, w = i32(table), torch.zeros((2, nkv, 512), device="cuda")
        qr = c.append(rows, i32(index), t, k, v, seq=seq)
        out = c.attend(q, k, v, t, i32(lens), weights=w)
        w2 = torch.zeros_like(w)
        # to a small pool, then in place
        t_out = i32(np.array([[0, 1], [2, 3]]))
        k2, v2 = (torch.zeros((4, page, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ln, kept = c.evict(k, v, t, i32(lens), w, 100, n_recent=7, k_out=k2, v_out=v2, table_out=t_out, weights_out=w2)
        ln2, kept2 = c.evict(k, v, t, i32(lens), w, 100, n_recent=7)
        c.sync()
        rows_k = [gather(k, table[s], int(ln2[s]), page) for s in range(2)]
        got.append([qr, out, w, w2, ln, kept, kept2, k2, v2, *rows_k])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # the other way round: out to the last pages of the large pools
    k, v = (torch.zeros((n_pages, page, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    t_out = np.array([[n_pages - 1, n_pages - 2], [n_pages - 3, n_pages - 4]], np.int32)
    ln, kept3 = c.evict(k0.clone(), v0.clone(), i32(small), i32(lens), torch.rand((2, nkv, 512), generator=g, device="cuda"),
                        100, k_out=k, v_out=v, table_out=i32(t_out))
    c.sync()
    for s in range(2):
        src, dst = gather(k0, small[s], lens[s], page), gather(k, t_out[s], int(ln[s]), page)
        for h in range(nkv):
            assert torch.equal(dst[:, h], src[kept3[s, h, :int(ln[s])].long(), h])
    c.close()
