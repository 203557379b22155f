"""Blocks of rows, shared prefixes and rotary forms of the paged cache without
a GPU: the oracle's pins, scaled frequencies, how tiles of rows are split over
thread blocks (csrc/sf_cache_index.h, compiled here as plain C++), and refusals
of the C ABI and of the binding."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import cache as oc
from test_cache_host import _let_through, _object, _reached_device_check, _shapes, bound, sf  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---------------------------------------------------------------- oracle

def test_oracle_turns():
    rng = np.random.default_rng(0)
    x, steps = rng.standard_normal((5, 3, 64)), np.array([0, 1, -77, 4095, 131071])
    f = oc.frequencies(64, 10000.0)
    np.testing.assert_allclose(oc.turn(x, steps[:, None], f), oc.rotate(x, steps, 10000.0), atol=1e-9)
    # neighbours: the same pairs in another order; part of a head: the rest as it is
    mixed = np.stack([x[..., :32], x[..., 32:]], -1).reshape(x.shape)
    got = oc.turn(mixed, steps[:, None], f, "interleaved")
    np.testing.assert_allclose(np.concatenate([got[..., 0::2], got[..., 1::2]], -1), oc.rotate(x, steps, 10000.0), atol=1e-9)
    part = oc.turn(x, steps[:, None], oc.frequencies(16, 10000.0), "half", 2.0)
    assert np.array_equal(part[..., 16:], x[..., 16:])
    np.testing.assert_allclose(part[..., :16], 2 * oc.rotate(x[..., :16], steps, 10000.0), atol=1e-9)
    # two turns are one
    back = oc.turn(oc.turn(x, steps[:, None], f), -steps[:, None], f)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_oracle_rows_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((7, 6, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    out, lse, w = oc.attend_rows(q, k, v, 0.2)
    kk, vv = (torch.from_numpy(t).permute(1, 0, 2).repeat_interleave(3, 0) for t in (k, v))
    qq = torch.from_numpy(q).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, scale=0.2).transpose(0, 1).numpy()
    np.testing.assert_allclose(out, ref, rtol=1e-10)
    np.testing.assert_allclose(lse, torch.logsumexp(qq @ kk.transpose(1, 2) * 0.2, -1).T.numpy(), rtol=1e-12)
    np.testing.assert_allclose(w.sum(-1), 1.0, rtol=1e-12)
    one, _ = oc.attend_one(q[3], k, v, 0.2)
    np.testing.assert_allclose(out[3], one, rtol=1e-12)
    none, lse, _ = oc.attend_rows(q, k[:0], v[:0], 0.2)
    assert not none.any() and np.all(lse == -np.inf)


# ---------------------------------------------------------------- frequencies

def test_frequencies(sf):
    f, m = sf.rotary_frequencies(64)
    assert m == 1.0 and len(f) == 32
    np.testing.assert_allclose(f, oc.frequencies(64, 10000.0), rtol=1e-14)
    np.testing.assert_allclose(sf.rotary_frequencies(64, 500.0, scaling="linear", factor=4)[0],
                               oc.frequencies(64, 500.0, 4.0), rtol=1e-14)
    # ntk: the fastest pair stays, the slowest is stretched by the factor
    n, m = sf.rotary_frequencies(64, scaling="ntk", factor=8.0)
    assert m == 1.0 and n[0] == 1.0 and math.isclose(n[-1], f[-1] / 8, rel_tol=1e-12)
    assert all(a <= b for a, b in zip(n, f))


def test_frequencies_bands_and_yarn_by_hand(sf):
    L, factor = 8192, 8.0
    f = oc.frequencies(128, 500000.0)
    turns = L * f / (2 * math.pi)
    b, m = sf.rotary_frequencies(128, 500000.0, scaling="bands", factor=factor, original_len=L)
    assert m == 1.0
    for x, y, t in zip(b, f, turns):
        if t >= 4:
            assert math.isclose(x, y, rel_tol=1e-13)
        elif t <= 1:
            assert math.isclose(x, y / factor, rel_tol=1e-12)
        else:
            g = (t - 1) / 3
            assert math.isclose(x, (1 - g) * y / factor + g * y, rel_tol=1e-12)
    assert (turns > 4).any() and (turns < 1).any() and ((turns > 1) & (turns < 4)).any()
    f = oc.frequencies(128, 10000.0)
    y, m = sf.rotary_frequencies(128, scaling="yarn", factor=4.0, original_len=4096)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    # pair of 32 turns: 64 ln(4096 / 64 pi) / ln 10000 = 20.9..; of one turn: 64 ln(4096 / 2 pi) / ln 10000 = 45.03
    assert np.allclose(y[:21], f[:21], rtol=1e-13) and np.allclose(y[46:], f[46:] / 4, rtol=1e-13)
    g = (30 - 20) / (46 - 20)
    assert math.isclose(y[30], f[30] / 4 * g + f[30] * (1 - g), rel_tol=1e-12)
    assert sf.rotary_frequencies(64, scaling="yarn", factor=1.0, original_len=4096)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(dim=0), dict(dim=7), dict(theta=0.0), dict(theta=float("nan")), dict(factor=0.0),
                                dict(factor=float("inf")), dict(scaling="cubic"), dict(scaling="yarn"),
                                dict(scaling="bands", original_len=0), dict(dim=2, scaling="ntk", factor=2.0),
                                dict(scaling="yarn", original_len=99, fast=1.0, slow=2.0),
                                dict(scaling="yarn", original_len=99, theta=1.0),
                                dict(scaling="bands", original_len=99, low=4.0, high=1.0)])
def test_frequencies_refuse(sf, kw):
    with pytest.raises(ValueError):
        sf.rotary_frequencies(**dict(dict(dim=64), **kw))


# ---------------------------------------------------------------- split

@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src = d / "rows.cpp"
    src.write_text("""
#include <vector>
#include "sf_cache_index.h"
using namespace sf;
struct Part { int cta, s, kvh, v0, nv, w, nb, b0, b1, first, last, slot; };
extern "C" {
// Parts that every thread block takes, in its order, as the kernels walk; ~n where out is too short.
int walk(const int* rows, const int* lens, int S, int group, int nkv, int half, int pair, int block, int fixed,
         int cost1, int cost2, int ctas, int least, Part* out, int room, long long* per_out) {
  const RowsShape sh{group, nkv, half, pair, block, fixed, {cost1, cost2}};
  std::vector<long long> first(S + 1, 0);
  for (int s = 0; s < S; ++s) first[s + 1] = first[s] + nkv * row_units(sh, rows[s], lens[s]);
  const long long total = first[S], per = units_per_block(total, ctas, least);
  *per_out = per;
  int n = 0;
  for (int c = 0; c < ctas; ++c) {
    long long u = per * c, end = u + per < total ? u + per : total;
    if (u >= end) continue;
    int s = 0;
    while (first[s + 1] <= u) ++s;
    RowsTiles t;
    t.start(sh, rows[s], lens[s], first[s], u);
    while (t.at < end) {
      if (!t.more(sh)) {
        do ++s; while (first[s + 1] == first[s]);
        t.start(sh, rows[s], lens[s], t.at, t.at);
      }
      const RowsPart p = t.take(sh, end);
      if (p.b0 < p.b1) {
        if (n == room) return ~n;
        out[n++] = Part{c, s, p.kvh, p.v0, p.nv, p.w, p.nb, p.b0, p.b1, (int)(p.u0 / per), rows_last_cta(p, per),
                        rows_slot(c, p.b0 == 0)};
      }
    }
  }
  return n;
}
long long units(int rows, int len, int group, int nkv, int half, int pair, int block, int fixed, int cost1, int cost2) {
  return row_units(RowsShape{group, nkv, half, pair, block, fixed, {cost1, cost2}}, rows, len);
}
}
""")
    so = d / "rows.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sparse_reuse_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    x = ctypes.CDLL(str(so))
    x.units.restype = ctypes.c_longlong
    return x


FIELDS = ["cta", "s", "kvh", "v0", "nv", "w", "nb", "b0", "b1", "first", "last", "slot"]


@pytest.mark.parametrize("seed", range(60))
def test_split_of_rows(lib, seed):
    """Every block of every tile is taken once; a tile's vectors are all of its rows'; a cut tile's thread blocks are
    first..last, each with a part; no two cut tiles share a slot or a first thread block."""
    rng = np.random.default_rng(seed)
    half, pair, block, fixed, costs = [(128, 2, 128, 24, (5, 6)), (64, 1, 64, 1, (1, 1)), (16, 1, 64, 0, (1, 1)),
                                       (128, 2, 128, 0, (1, 2))][seed % 4]
    S, nkv, group = int(rng.integers(1, 30)), int(rng.integers(1, 9)), int(rng.choice([1, 4, 5, 6, 16, 21]))
    ctas, least = int(rng.choice([1, 7, 152])), int(rng.choice([3, 8, 12]))
    rows = (rng.integers(0, int(rng.choice([2, 40, 700])), S) * (rng.random(S) < 0.8)).astype(np.int32)
    lens = (rng.integers(0, int(rng.choice([2, 300, 9000])), S) * (rng.random(S) < 0.8)).astype(np.int32)
    room = 400000
    out, per = np.zeros((room, len(FIELDS)), np.int32), ctypes.c_longlong()
    n = lib.walk(rows.ctypes.data_as(ctypes.c_void_p), lens.ctypes.data_as(ctypes.c_void_p), S, group, nkv, half, pair,
                 block, fixed, *costs, ctas, least, out.ctypes.data_as(ctypes.c_void_p), room, ctypes.byref(per))
    assert n >= 0
    tiles, loads = {}, np.zeros(ctas, np.int64)
    for row in out[:n]:
        p = dict(zip(FIELDS, row.tolist()))
        tiles.setdefault((p["s"], p["kvh"], p["v0"]), []).append(p)
        loads[p["cta"]] += (p["b1"] - p["b0"]) * costs[p["w"] - 1]
    slots, firsts, seen = set(), set(), {}
    for (s, kvh, v0), parts in tiles.items():
        assert v0 % (half * pair) == 0 and 0 <= kvh < nkv
        seen.setdefault((s, kvh), []).append((v0, parts[0]["nv"]))
        nb = -(-int(lens[s]) // block)
        at = 0
        for i, p in enumerate(parts):
            assert p["nb"] == nb and p["b0"] == at and p["cta"] == parts[0]["first"] + i
            assert p["w"] == -(-p["nv"] // half) <= pair
            at = p["b1"]
        assert at == nb and parts[-1]["cta"] == parts[0]["last"]
        if len(parts) > 1:
            assert parts[0]["first"] not in firsts
            firsts.add(parts[0]["first"])
            for p in parts:
                assert 0 <= p["slot"] < 2 * ctas and p["slot"] not in slots
                slots.add(p["slot"])
    want = {(s, h) for s in range(S) for h in range(nkv) if rows[s] and lens[s]}
    assert set(seen) == want
    for (s, _), t in seen.items():
        t.sort()
        assert t[0][0] == 0 and all(a + b == c for (a, b), (c, _) in zip(t, t[1:]))
        assert sum(b for _, b in t) == rows[s] * group
    shape = (group, nkv, half, pair, block, fixed, *costs)
    total = sum(lib.units(int(r), int(x), *shape) * nkv for r, x in zip(rows, lens))
    assert loads.sum() == total - fixed * len(tiles)
    # even shares: within a block either way
    assert n == 0 or (loads.max() <= per.value + max(costs) - 1 and per.value == max(least, -(-total // ctas)))


def test_largest_units(lib):
    assert lib.units(1048576, 262144, 1024, 1, 128, 2, 128, 8, 2, 3) == 2 ** 30 // 256 * (8 + 3 * 2048)
    assert lib.units(0, 5, 4, 2, 128, 2, 128, 8, 2, 3) == lib.units(5, 0, 4, 2, 128, 2, 128, 8, 2, 3) == 0
    assert lib.units(97, 300, 4, 2, 128, 2, 128, 8, 2, 3) == (8 + 9) + (8 + 9)     # 388 vectors: two tiles of two halves
    assert lib.units(96, 300, 4, 2, 128, 2, 128, 8, 2, 3) == (8 + 9) + (8 + 6)


# ---------------------------------------------------------------- refusals

def _options(sf, **kw):
    base = dict(rotary_layout=0, rotary_dim=0, inv_freq=None, rotary_magnitude=0.0, max_rows=64)
    base.update(kw)
    if base["inv_freq"] is not None:
        base["inv_freq"] = (ctypes.c_double * len(base["inv_freq"]))(*base["inv_freq"])
    return sf.SfCacheOptions(*[base[f] for f, _ in sf.SfCacheOptions._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_layout=2), 1), (dict(rotary_layout=-1), 1), (dict(rotary_dim=-16), 1), (dict(rotary_magnitude=-1.0), 1),
    (dict(rotary_magnitude=float("nan")), 1), (dict(rotary_magnitude=float("inf")), 1), (dict(rotary_magnitude=1e-40), 1),
    (dict(rotary_magnitude=1e39), 1), (dict(max_rows=-1), 1), (dict(inv_freq=[1.0] * 31 + [float("nan")]), 1),
    (dict(rotary_dim=16, inv_freq=[float("inf")] + [1.0] * 7), 1), (dict(rotary_dim=8), 4), (dict(rotary_dim=24), 4),
    (dict(rotary_dim=80), 4), (dict(max_rows=1048577), 4)])
def test_create_refuses_bad_options_before_any_device_work(sf, kw, status):
    c = ctypes.c_void_p(1)
    o = _options(sf, **kw)
    assert sf.lib.sf_cache_create_with(ctypes.byref(_shapes(sf)), ctypes.byref(o), ctypes.byref(c)) == status
    assert not c.value
    # the shapes are looked at as ever
    assert sf.lib.sf_cache_create_with(ctypes.byref(_shapes(sf, head_dim=96)), None, ctypes.byref(c)) == 4


def _rows_object(sf, max_rows=64, **kw):
    """An object of which only shapes and options are filled in."""
    buf = _object(sf, **kw)
    o = _options(sf, max_rows=max_rows)
    at = (ctypes.sizeof(sf.SfCacheShapes) + 7) // 8 * 8
    ctypes.memmove(ctypes.addressof(buf) + at, ctypes.byref(o), ctypes.sizeof(o))
    return buf


ROWS = dict(q=16, ld_q=256, T=8, k=16, v=32, n_pages=9, page_table=16, S=4, cols=4, ld_table=4, lens=16, starts=16,
            scale=0.1, out=65536, ld_out=256, lse=262144)
SHARED = dict(q=16, ld_q=256, k=16, v=32, n_pages=9, page_table=16, S=4, cols=4, ld_table=4, lens=16, ptable=16, G=2,
              pcols=4, ld_ptable=4, plens=16, starts=16, scale=0.1, out=65536, ld_out=256, lse=262144)
TURN = dict(k=16, n_pages=9, page_table=16, S=4, cols=4, ld_table=4, lens=16, frm=16, to=16, ld_pos=64)


@pytest.mark.parametrize("call,base,kw,status,text", [
    ("attend_rows", ROWS, dict(q=8), 1, "q/out"), ("attend_rows", ROWS, dict(q=None), 1, "q/out"),
    ("attend_rows", ROWS, dict(ld_q=252), 1, "q/out"), ("attend_rows", ROWS, dict(ld_out=255), 1, "q/out"),
    ("attend_rows", ROWS, dict(T=-1), 1, "-1 rows"), ("attend_rows", ROWS, dict(T=65), 2, "65 rows"),
    ("attend_rows", ROWS, dict(scale=float("inf")), 1, "scale"), ("attend_rows", ROWS, dict(scale=3e38), 1, "scale"),
    ("attend_rows", ROWS, dict(out=16), 1, "out overlaps q"), ("attend_rows", ROWS, dict(out=16 + 512 * 7), 1, "out overlaps q"),
    ("attend_rows", ROWS, dict(lse=16), 1, "lse overlaps"), ("attend_rows", ROWS, dict(lse=65536 + 4), 1, "lse overlaps"),
    ("attend_rows", ROWS, dict(lse=262146), 1, "lse misaligned"), ("attend_rows", ROWS, dict(starts=None), 1, "starts"),
    ("attend_rows", ROWS, dict(starts=18), 1, "starts"), ("attend_rows", ROWS, dict(lens=None), 1, "lens"),
    ("attend_rows", ROWS, dict(k=None), 1, "pool"), ("attend_rows", ROWS, dict(S=5), 2, "S=5"),
    ("attend_rows", ROWS, dict(S=-1), 1, "S=-1"), ("attend_rows", ROWS, dict(cols=0), 1, "table_cols"),
    ("attend_shared", SHARED, dict(q=8), 1, "q/out"), ("attend_shared", SHARED, dict(S=5), 2, "S=5"),
    ("attend_shared", SHARED, dict(S=-1), 1, "-1 rows"), ("attend_shared", SHARED, dict(G=0), 1, "G=0"),
    ("attend_shared", SHARED, dict(G=65537), 2, "G=65537"), ("attend_shared", SHARED, dict(ptable=None), 1, "table"),
    ("attend_shared", SHARED, dict(pcols=0), 1, "table_cols"), ("attend_shared", SHARED, dict(ld_ptable=3), 1, "ld_table"),
    ("attend_shared", SHARED, dict(plens=None), 1, "prefix_lens"), ("attend_shared", SHARED, dict(starts=None), 1, "starts"),
    ("attend_shared", SHARED, dict(plens=18), 1, "prefix_lens"), ("attend_shared", SHARED, dict(out=16), 1, "out overlaps q"),
    ("attend_shared", SHARED, dict(scale=float("nan")), 1, "scale"), ("attend_shared", SHARED, dict(lse=24), 1, "lse overlaps"),
    ("reposition", TURN, dict(k=None), 1, "pool"), ("reposition", TURN, dict(k=24), 1, "pool"),
    ("reposition", TURN, dict(lens=None), 1, "lens"), ("reposition", TURN, dict(frm=None), 1, "pos_from"),
    ("reposition", TURN, dict(to=18), 1, "pos_to"), ("reposition", TURN, dict(ld_pos=0), 1, "ld_pos"),
    ("reposition", TURN, dict(S=5), 2, "S=5"), ("reposition", TURN, dict(n_pages=0), 1, "n_pages"),
    ("reposition", TURN, dict(page_table=17), 1, "table"),
])
def test_calls_refuse_bad_arguments(sf, call, base, kw, status, text):
    obj = _rows_object(sf)
    fn = getattr(sf.lib, f"sf_cache_{call}")
    assert fn(obj, None, *dict(base, **kw).values()) == status
    said = sf.lib.sf_cache_last_error(obj).decode()
    assert text in said, said
    assert fn(None, None, *base.values()) == sf.SF_ERR_INVALID_ARG


@pytest.mark.parametrize("call,base", [("attend_rows", ROWS), ("attend_shared", SHARED)])
def test_rows_need_an_object_for_them(sf, call, base):
    obj = _rows_object(sf, max_rows=0)
    assert getattr(sf.lib, f"sf_cache_{call}")(obj, None, *base.values()) == sf.SF_ERR_INVALID_ARG
    assert "max_rows" in sf.lib.sf_cache_last_error(obj).decode()


# ---------------------------------------------------------------- binding

@pytest.fixture
def rows_bound(sf, bound):
    obj = _rows_object(sf)
    bound.keep = obj
    bound._bind(ctypes.addressof(obj), -1)
    return bound


def _tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(q=torch.zeros(5, 4, 64, dtype=bf), k=torch.zeros(9, 16, 2, 64, dtype=bf), v=torch.zeros(9, 16, 2, 64, dtype=bf),
                table=torch.zeros(3, 4, dtype=i32), lens=torch.zeros(3, dtype=i32), starts=torch.zeros(4, dtype=i32),
                ptable=torch.zeros(2, 7, dtype=i32), plens=torch.zeros(2, dtype=i32), groups=torch.zeros(3, dtype=i32),
                frm=torch.zeros(3, 2, 20, dtype=i32))


def test_binding_lets_rows_through(rows_bound, sf):
    c, t = rows_bound, _tensors()
    wide = torch.zeros(5, 512, dtype=torch.bfloat16)
    for call in (lambda: c.attend_rows(t["q"], t["k"], t["v"], t["table"], t["lens"], t["starts"]),
                 lambda: c.attend_rows(wide[:, :256], t["k"], t["v"], t["table"][:, :3], t["lens"], t["starts"],
                                       out=wide[:, 256:], lse=torch.zeros(5, 4), scale=1),
                 lambda: c.attend_shared(t["q"][:3], t["k"], t["v"], t["table"], t["lens"], t["ptable"], t["plens"],
                                         t["groups"], lse=torch.zeros(3, 4)),
                 lambda: c.reposition(t["k"], t["table"], t["lens"], t["frm"]),
                 lambda: c.reposition(t["k"], t["table"], t["lens"], t["frm"], pos_to=t["frm"])):
        _let_through(sf, call)
        assert _reached_device_check(c, sf)


def test_binding_refuses_rows(rows_bound, sf):
    c, t = rows_bound, _tensors()
    good = dict(q=t["q"], k_pages=t["k"], v_pages=t["v"], table=t["table"], lens=t["lens"], starts=t["starts"])
    for kw in (dict(q=t["q"].float()), dict(q=t["q"][:, :3]), dict(out=t["q"][:4]), dict(lse=torch.zeros(5, 3)),
               dict(lse=torch.zeros(4, 4)), dict(lse=torch.zeros(5, 4, dtype=torch.float64)), dict(lse=torch.zeros(5, 8)[:, ::2]),
               dict(starts=t["starts"][:3]), dict(starts=t["starts"].long()), dict(lens=t["lens"][:2]), dict(table=t["table"][0]),
               dict(k_pages=t["k"].float()), dict(starts=[0, 1, 2, 3])):
        with pytest.raises(ValueError):
            c.attend_rows(**dict(good, **kw))
    with pytest.raises(TypeError):
        c.attend_rows(**good, scale="x")
    good = dict(q=t["q"][:3], k_pages=t["k"], v_pages=t["v"], table=t["table"], lens=t["lens"], prefix_table=t["ptable"],
                prefix_lens=t["plens"], starts=t["groups"])
    for kw in (dict(q=t["q"]), dict(out=t["q"]), dict(starts=t["groups"][:2]), dict(prefix_lens=t["plens"][:1]),
               dict(prefix_table=t["ptable"].long()), dict(prefix_table=t["ptable"].t()), dict(lse=torch.zeros(2, 4))):
        with pytest.raises(ValueError):
            c.attend_shared(**dict(good, **kw))
    for kw in (dict(pos_from=t["frm"][:2]), dict(pos_from=t["frm"].long()), dict(pos_from=t["frm"][:, :1]),
               dict(pos_to=t["frm"][..., :19]), dict(pos_from=t["frm"][..., ::2]), dict(k_pages=t["k"][0]), dict(lens=t["lens"][:1])):
        with pytest.raises(ValueError):
            c.reposition(**dict(dict(k_pages=t["k"], table=t["table"], lens=t["lens"], pos_from=t["frm"]), **kw))
    assert not _reached_device_check(c, sf)


def test_binding_refuses_bad_rotary_options(sf):
    base = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, dtype="bf16", page_size=16, max_seqs=1, max_len=16)
    for kw in (dict(rotary_layout="halves"), dict(rotary_dim=0), dict(rotary_magnitude=0.0), dict(inv_freq=[1.0] * 31),
               dict(rotary_magnitude=float("nan")), dict(rotary_dim=32, inv_freq=[1.0] * 32), dict(rotary_dim=-16)):
        with pytest.raises(ValueError):
            sf.PagedCache(**base, **kw)
    for kw, status in ((dict(rotary_dim=40), 4), (dict(max_rows=-1), 1), (dict(inv_freq=[float("inf")] * 32), 1)):
        with pytest.raises(sf.SpecFoldError) as e:
            sf.PagedCache(**base, **kw)
        assert e.value.status == status
