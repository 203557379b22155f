"""How many bits of a softmax weight the bf16 forms of attend_rows and
attend_shared keep: 2^-16 (the sum of two bf16 numbers) for tiles of up to 128
query vectors, and for larger ones in calls of little work.

The tolerance is that of test_gpu_cache_rows.py with 2^-16 in the place of
2^-8 (u = 2^-24, e = 2^-8 the half step of the output):
    d = (HD + 4) 2u sum_d |q_d k_d| |scale|
    r = 2 d + 2 (len + 64) 2u + 8u + 2^-16
    out:  r sum_j p_j |v_j| (1 + e) + e |ref|
The output's own rounding, e |ref|, is as large as what a weight rounded to
bf16 costs, but it is small where the weighted values cancel, which some of
thousands of random outputs do.  That the bound tells the two apart on these
inputs is shown here with the plain form, on the CPU."""
import numpy as np
import pytest
import torch

from test_gpu_cache import i32, make_pages, sf  # noqa: F401

U, E = 2.0 ** -24, 2.0 ** -8


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def inputs(heads, lens, rows, page, seed, apart=0):
    """q [sum(rows), nq, hd], pools and table in bf16 (scores about 0.5 of spread).  apart: only so many keys of a
    sequence, at random places, have weights that count; the others' scores are some 12 lower."""
    nq, nkv, hd = heads
    rng = np.random.default_rng([seed, hd, sum(lens)])
    table, total = make_pages(rng, lens, page)
    bf = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    q = rng.standard_normal((sum(rows), nq, hd)) * 0.5
    k, v = (rng.standard_normal((total, page, nkv, hd)) for _ in range(2))
    if apart:
        q[..., 0] = 8.0
        k[..., 0] = -12.0 / 8.0 * hd ** 0.5
        for s, n in enumerate(lens):
            for j in rng.choice(n, min(n, apart), replace=False):
                k[table[s, j // page], j % page, :, 0] = 0.0
    return bf(q), bf(k), bf(v), table


def places(table, s, n, page):
    j = np.arange(n)
    return table[s, j // page].astype(np.int64) * page + j % page


def worst(out, q, k, v, slots, w=2.0 ** -16):
    """Largest error of rows out [R, nq, hd] over the positions `slots` in units of the tolerance."""
    R, nq, hd = q.shape
    nkv, n, most = k.shape[2], len(slots), 0.0
    G, scale, at = nq // nkv, hd ** -0.5, torch.as_tensor(slots, device=q.device)
    for c in range(nkv):
        h = slice(c * G, (c + 1) * G)
        kk, vv = (t.view(-1, nkv, hd)[at, c].double() for t in (k, v))
        x = q[:, h].double().reshape(R * G, hd)
        p = torch.softmax(x @ kk.T * scale, 1)
        d = (hd + 4) * 2 * U * scale * (x.abs() @ kk.abs().T).amax(1)
        r = 2 * d + 4 * (n + 64) * U + 8 * U + w
        ref = p @ vv
        tol = r[:, None] * (p @ vv.abs()) * (1 + E) + E * ref.abs()
        most = max(most, float(((out[:, h].double().reshape(R * G, hd) - ref).abs() / tol).max()))
    return most


def plain(q, k, v, slots, numbers):
    """The operator in fp32 with every weight as the sum of `numbers` bf16 numbers."""
    R, nq, hd = q.shape
    nkv = k.shape[2]
    G, out = nq // nkv, torch.empty(q.shape, dtype=torch.bfloat16)
    for c in range(nkv):
        h = slice(c * G, (c + 1) * G)
        kk, vv = (t.view(-1, nkv, hd)[slots, c].float() for t in (k, v))
        s = q[:, h].float() @ kk.T * hd ** -0.5
        p = torch.exp(s - s.amax(-1, keepdim=True))
        kept = torch.zeros_like(p)
        for _ in range(numbers):
            kept += (p - kept).to(torch.bfloat16).float()
        out[:, h] = (kept @ vv / p.sum(-1, keepdim=True)).to(torch.bfloat16)
    return out


# heads, page, rows, lens, keys that count (0: all).  Up to 128 vectors (rows times heads of a KV head) of a sequence.
NARROW = [
    ((4, 2, 64), 5, [64, 3, 1], [2, 7, 20], 0),
    ((12, 2, 128), 16, [20, 21, 7], [9, 20, 3], 0),
    ((12, 2, 128), 16, [21, 5], [300, 700], 6),
    ((40, 8, 128), 32, [25, 9], [129, 256], 5),
    ((8, 8, 64), 7, [128], [1000], 4),
]


# More vectors together, two blocks of 256 of them and 128 keys at most for each SM.
SMALL = [
    ((12, 2, 128), 32, [32], [512], 5),
    ((40, 8, 128), 32, [32], [20], 0),
    ((40, 8, 128), 16, [52, 26], [700, 9], 6),
    ((4, 2, 64), 5, [100, 65, 129], [17, 257, 5], 6),
    ((16, 1, 128), 100, [40], [2000], 4),
]


@pytest.mark.parametrize("heads,page,rows,lens,apart", NARROW + SMALL)
def test_the_bound_tells_one_bf16_number_from_two(heads, page, rows, lens, apart):
    q, k, v, table = inputs(heads, lens, rows, page, 1, apart)
    st, one, two = offsets(rows), [], []
    for s, n in enumerate(lens):
        x, slots = q[st[s]:st[s + 1]], places(table, s, n, page)
        one.append(worst(plain(x, k, v, slots, 1), x, k, v, slots))
        two.append(worst(plain(x, k, v, slots, 2), x, k, v, slots))
    assert max(two) <= 1.0 and max(one) > 1.5, (one, two)


def rows_of(sf, q, k, v, table, lens, rows, page):
    nq, nkv, hd = q.shape[1], k.shape[2], k.shape[3]
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype="bf16", page_size=page, max_seqs=len(lens),
                      max_len=max(lens), max_rows=q.shape[0])
    out = c.attend_rows(q, k, v, i32(table), i32(lens), i32(offsets(rows)))
    c.sync()
    c.close()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("heads,page,rows,lens,apart", NARROW + SMALL)
def test_rows_keep_two(sf, heads, page, rows, lens, apart):  # noqa: F811
    q, k, v, table = inputs(heads, lens, rows, page, 1, apart)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    out, st = rows_of(sf, q, k, v, table, lens, rows, page), offsets(rows)
    for s, n in enumerate(lens):
        at = slice(int(st[s]), int(st[s + 1]))
        far = worst(out[at], q[at], k, v, places(table, s, n, page))
        assert far <= 1.0, (s, far)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,members,prefix,tail,apart", [((12, 2, 128), 21, 9, 3, 0), ((40, 8, 128), 25, 300, 70, 6),
                                                             ((4, 2, 64), 64, 700, 1, 5), ((32, 8, 128), 61, 400, 9, 6)])
def test_shared_prefixes_keep_two(sf, heads, members, prefix, tail, apart):  # noqa: F811
    nq, nkv, hd = heads
    page, lens = 16, [tail] * members + [prefix]
    q, k, v, table = inputs(heads, lens, [1] * members + [0], page, 2, apart)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    c = sf.PagedCache(n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, dtype="bf16", page_size=page, max_seqs=members,
                      max_len=max(lens), max_rows=members)
    out = c.attend_shared(q, k, v, i32(table[:-1]), i32(lens[:-1]), i32(table[-1:]), i32(lens[-1:]), i32([0, members]))
    c.sync()
    c.close()
    for s in range(members):
        slots = np.r_[places(table, members, prefix, page), places(table, s, tail, page)]
        far = worst(out[s:s + 1], q[s:s + 1], k, v, slots)
        assert far <= 1.0, (s, far)
