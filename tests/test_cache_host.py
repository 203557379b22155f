"""Paged cache without a GPU: the oracle's pins, the index arithmetic the
kernels share (compiled here as plain C++), refusals of the C ABI and of the
binding, and how the binding passes strided tensors on."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sf():
    from sparse_reuse_gb300 import build
    build.build()
    import sparse_reuse_gb300 as m
    return m


# ---------------------------------------------------------------- oracle

def test_oracle_rotation_is_the_pass_rotation():
    """The cache rotates as the verification pass does (the same function of
    position), with 30-digit pins behind oracle.rope's golden values."""
    x = np.random.default_rng(0).standard_normal((5, 3, 64))
    pos = np.array([0, 1, 77, 4095, 131071])
    want = oracle.rope(x, pos, 10000.0)
    np.testing.assert_allclose(oc.rotate(x, pos, 10000.0), want, atol=1e-9)


def test_oracle_norm_and_attention_against_torch():
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((4, 3, 64)), rng.standard_normal(64)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(g), 1e-6).numpy()
    np.testing.assert_allclose(oc.head_norm(x, g, 1e-6), want, rtol=1e-12)
    q, k, v = rng.standard_normal((6, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    out, w = oc.attend_one(q, k, v, 0.125)
    kk, vv = (torch.from_numpy(t).permute(1, 0, 2).repeat_interleave(3, 0) for t in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q)[:, None], kk, vv)[:, 0].numpy()
    np.testing.assert_allclose(out, ref, rtol=1e-10)
    np.testing.assert_allclose(w.sum(1), 1.0, rtol=1e-12)


def test_oracle_choice_by_hand():
    w = [5.0, 1.0, 3.0, 3.0, float("nan"), -0.0, 0.0, 3.0, 2.0, 9.0]
    assert oc.choose(w, 10, 10, 0, 0) == list(range(10))
    assert oc.choose(w, 10, 4, 0, 0) == [0, 2, 3, 9]            # ties of 3.0: lower indexes
    assert oc.choose(w, 10, 4, 0, 2) == [0, 2, 8, 9]
    assert oc.choose(w, 10, 9, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8, 9]   # NaN goes first
    assert oc.choose(w, 10, 8, 1, 0) == [0, 1, 2, 3, 5, 7, 8, 9]      # -0 and 0 tie: index 5
    assert oc.choose(w, 10, 3, 1, 2) == [0, 8, 9]
    assert oc.choose([-np.inf, np.nan, np.inf, 0.0], 4, 3, 0, 0) == [0, 2, 3]


# ---------------------------------------------------------------- index arithmetic of the kernels

@pytest.fixture(scope="module")
def index_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    src = d / "shim.cpp"
    src.write_text("""
#include "sf_cache_index.h"
extern "C" {
long long slot(const int* pages, long long ld, int cols, int page, long long n_pages, int s, int j) {
  return sf::page_slot(sf::make_page_table(pages, ld, cols, page, n_pages), s, j);
}
unsigned slot32(const int* pages, long long ld, int cols, int page, long long n_pages, int s, int j) {
  const sf::PageTable t = sf::make_page_table(pages, ld, cols, page, n_pages);
  return sf::entry_slot32(t, sf::page_entry(t, s, j), j);
}
int quotients(int page) {  // positions whose page is not their quotient
  const sf::PageTable t = sf::make_page_table(nullptr, 0, 0, page, 0);
  int wrong = 0;
  for (int j = 0; j < sf::kMaxLen; ++j) wrong += sf::page_of(t, j) != j / page;
  return wrong;
}
long long limit(int max_len, int cols, int page) { return sf::length_limit(max_len, cols, page); }
long long per(long long u, int blocks, int least) { return sf::units_per_block(u, blocks, least); }
int tiles(int n) { return sf::tiles_of(n); }
void cut(long long first, int tiles, long long per, int* b0, int* b1) {
  *b0 = sf::first_block(first, per);
  *b1 = sf::last_block(first, tiles, per);
}
int part(int block, long long first, long long per) { return sf::part_slot(block, first, per); }
int len(int n, long long lim, int* bad) { bool b; int r = sf::checked_len(n, lim, &b); *bad = b; return r; }
}
""")
    so = d / "shim.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sparse_reuse_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.slot.restype = ctypes.c_longlong
    lib.slot.argtypes = [ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_longlong,
                         ctypes.c_int, ctypes.c_int]
    lib.slot32.argtypes = lib.slot.argtypes
    lib.slot32.restype = ctypes.c_uint
    lib.limit.restype = lib.per.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("page", [1, 7, 16, 24, 128])
def test_slots_and_bad_pages(index_lib, page):
    rng = np.random.default_rng(page)
    table = rng.integers(0, 50, (3, 9)).astype(np.int32)
    table[0, 2], table[1, 3] = -1, 50              # outside a pool of 50 pages
    wide = np.full((3, 12), 10 ** 6, np.int32)     # a strided table: columns 9.. are not the sequence's
    wide[:, :9] = table
    for s in range(3):
        for j in list(range(-2, 9 * page + 3)) + [2 ** 31 - 1]:
            got = index_lib.slot(wide.ctypes.data, 12, 9, page, 50, s, j)
            c = j // page
            ok = 0 <= j < 9 * page and 0 <= table[s, c] < 50
            assert got == (int(table[s, c]) * page + j % page if ok else -1), (s, j)
            if j >= 0:
                assert index_lib.slot32(wide.ctypes.data, 12, 9, page, 50, s, j) == got % 2 ** 32


def test_page_of_every_position(index_lib):
    rng = np.random.default_rng(0)
    for page in [1, 2, 3, 5, 7, 16, 24, 100, 4095, 4097, 65521, 65535, 65536] + rng.integers(1, 65537, 60).tolist():
        assert index_lib.quotients(int(page)) == 0, page


def test_slots_beyond_32_bits(index_lib):
    table = np.array([[2 ** 31 - 1]], np.int32)
    assert index_lib.slot(table.ctypes.data, 1, 1, 65536, 2 ** 31, 0, 65535) == (2 ** 31 - 1) * 65536 + 65535
    assert index_lib.slot32(table.ctypes.data, 1, 1, 1, 2 ** 32 - 2, 0, 0) == 2 ** 31 - 1
    table[0, 0] = -1
    assert index_lib.slot32(table.ctypes.data, 1, 1, 1, 2 ** 32 - 2, 0, 0) == 2 ** 32 - 1


def test_length_limits(index_lib):
    bad = ctypes.c_int()
    assert index_lib.limit(1000, 7, 100) == 700 and index_lib.limit(600, 7, 100) == 600
    assert index_lib.limit(262144, 2 ** 20, 65536) == 262144
    for n, want, b in ((0, 0, 0), (700, 700, 0), (701, 0, 1), (-1, 0, 1), (-2 ** 31, 0, 1)):
        assert index_lib.len(n, ctypes.c_longlong(700), ctypes.byref(bad)) == want and bad.value == b


@pytest.mark.parametrize("seed", range(40))
def test_split_of_a_batch(index_lib, seed):
    """Every unit belongs to one block; a cut segment's blocks are first..last;
    no two cut segments share a partial slot or an arrival counter, whatever the
    batch; sizes beyond 32 bits of units."""
    ll = ctypes.c_longlong
    rng = np.random.default_rng(seed)
    S, H, blocks, least = int(rng.integers(1, 40)), int(rng.integers(1, 9)), int(rng.integers(1, 153)), 16
    top = int(rng.choice([5, 40, 2000, 262144]))
    lens = rng.integers(0, top + 1, S) * (rng.random(S) < 0.8)
    tiles = [index_lib.tiles(int(n)) for n in lens]
    assert tiles == [-(-int(n) // 16) for n in lens]
    units = sum(tiles) * H
    per = index_lib.per(ll(units), blocks, least)
    assert per >= least and per * blocks >= units and (per == least or (per - 1) * blocks < units)
    at, slots, counters = 0, set(), set()
    for t in tiles:
        for _ in range(H):
            if t:
                b0, b1 = ctypes.c_int(), ctypes.c_int()
                index_lib.cut(ll(at), t, ll(per), ctypes.byref(b0), ctypes.byref(b1))
                b0, b1 = b0.value, b1.value
                assert b0 == at // per and b1 == (at + t - 1) // per < blocks
                if b0 != b1:
                    assert b0 not in counters
                    counters.add(b0)
                    for b in range(b0, b1 + 1):
                        p = index_lib.part(b, ll(at), ll(per))
                        assert 0 <= p < 2 * blocks and p not in slots
                        slots.add(p)
            at += t
    assert index_lib.per(ll(2 ** 40), 152, least) == -(-2 ** 40 // 152)


# ---------------------------------------------------------------- refusals

def _shapes(sf, **kw):
    base = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, dtype=sf.SF_BF16, page_size=16, max_seqs=4, max_len=64,
                max_pos=128, rms_eps=1e-6, rope_theta=1e4, track_weights=1)
    base.update(kw)
    return sf.SfCacheShapes(*[base[f] for f, _ in sf.SfCacheShapes._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(n_q_heads=0), 1), (dict(dtype=2), 1), (dict(page_size=0), 1), (dict(max_len=-1), 1), (dict(max_pos=0), 1),
    (dict(rms_eps=-1.0), 1), (dict(rms_eps=float("nan")), 1), (dict(rope_theta=0.0), 1),
    (dict(rope_theta=float("inf")), 1), (dict(head_dim=96), 4), (dict(n_q_heads=5), 4), (dict(max_seqs=4097), 4),
    (dict(max_len=262145), 4), (dict(page_size=65537), 4), (dict(max_pos=4194305), 4), (dict(n_q_heads=2048), 4)])
def test_create_refuses_bad_shapes_before_any_device_work(sf, kw, status):
    c = ctypes.c_void_p(1)
    assert sf.lib.sf_cache_create(ctypes.byref(_shapes(sf, **kw)), ctypes.byref(c)) == status and not c.value
    assert sf.lib.sf_cache_create(None, ctypes.byref(c)) == sf.SF_ERR_INVALID_ARG
    assert sf.lib.sf_cache_create(ctypes.byref(_shapes(sf)), None) == sf.SF_ERR_INVALID_ARG


def _object(sf, **kw):
    """An object of which only the shapes (its first member) are filled in:
    enough for the argument checks, which come before everything else."""
    buf = ctypes.create_string_buffer(4096)
    shapes = _shapes(sf, **kw)
    ctypes.memmove(buf, ctypes.byref(shapes), ctypes.sizeof(shapes))
    return buf


APPEND = dict(qkv=16, ld_qkv=512, T=3, q_gain=16, k_gain=16, index=16, pos=16, seq=16, page_table=16, S=4, cols=4,
              ld_table=4, k=16, v=32, n_pages=9, q_out=16, ld_q=256)
ATTEND = dict(q=16, ld_q=256, k=16, v=32, n_pages=9, page_table=16, S=4, cols=4, ld_table=4, lens=16, scale=0.1,
              out=16, ld_out=256, w_in=16, w_out=16, ld_w=64)
EVICT = dict(k=16, v=32, n_pages=9, page_table=16, S=4, cols=4, ld_table=4, lens=16, w=16, ld_w=64, budget=32,
             n_first=4, n_recent=8, k_out=48, v_out=64, n_pages_out=9, table_out=20, cols_out=4, ld_out=4, w_out=16,
             lens_out=16, kept=16)


@pytest.mark.parametrize("call,base,kw,status,text", [
    ("append", APPEND, dict(qkv=None), 1, "qkv"), ("append", APPEND, dict(qkv=24), 1, "qkv"),
    ("append", APPEND, dict(ld_qkv=511), 1, "qkv"), ("append", APPEND, dict(ld_qkv=516), 1, "qkv"),
    ("append", APPEND, dict(ld_qkv=-512), 1, "qkv"), ("append", APPEND, dict(q_out=8), 1, "q_out"),
    ("append", APPEND, dict(ld_q=248), 1, "q_out"), ("append", APPEND, dict(index=None), 1, "index"),
    ("append", APPEND, dict(index=18), 1, "index"), ("append", APPEND, dict(q_gain=20), 1, "gain"),
    ("append", APPEND, dict(T=-1), 1, "T=-1"), ("append", APPEND, dict(k=None), 1, "pool"),
    ("append", APPEND, dict(v=40), 1, "pool"), ("append", APPEND, dict(page_table=17), 1, "table"),
    ("append", APPEND, dict(cols=0), 1, "table_cols"), ("append", APPEND, dict(ld_table=3), 1, "ld_table"),
    ("append", APPEND, dict(n_pages=0), 1, "n_pages"), ("append", APPEND, dict(S=5), 2, "S=5"),
    ("append", APPEND, dict(seq=None, T=5), 2, "T=5"), ("append", APPEND, dict(T=1048577), 2, "T=1048577"),
    ("append", APPEND, dict(k=32), 1, "one pool"),
    ("attend", ATTEND, dict(q=8), 1, "q/out"), ("attend", ATTEND, dict(ld_out=255), 1, "q/out"),
    ("attend", ATTEND, dict(lens=None), 1, "lens"), ("attend", ATTEND, dict(scale=float("nan")), 1, "scale"),
    ("attend", ATTEND, dict(w_out=None), 1, "weights_in"), ("attend", ATTEND, dict(ld_w=63), 2, "ld_w"),
    ("attend", ATTEND, dict(w_in=18), 1, "weights"), ("attend", ATTEND, dict(S=-1), 1, "S=-1"),
    ("evict", EVICT, dict(budget=0), 1, "budget"), ("evict", EVICT, dict(n_first=-1), 1, "n_first"),
    ("evict", EVICT, dict(n_first=20, n_recent=13), 1, "n_recent"), ("evict", EVICT, dict(budget=65), 2, "budget"),
    ("evict", EVICT, dict(cols_out=1), 2, "output table"), ("evict", EVICT, dict(ld_w=60), 2, "ld_w"),
    ("evict", EVICT, dict(k_out=16), 1, "in part"), ("evict", EVICT, dict(table_out=16), 1, "in part"),
    ("evict", EVICT, dict(k_out=16, v_out=32, table_out=16, ld_out=5), 1, "in part"),
    ("evict", EVICT, dict(v_out=48), 1, ""), ("evict", EVICT, dict(kept=None), 1, "kept"),
    ("evict", EVICT, dict(w=None), 1, "weights"), ("evict", EVICT, dict(n_first=2 ** 31 - 1, n_recent=2), 1, "n_first"),
])
def test_calls_refuse_bad_arguments(sf, call, base, kw, status, text):
    obj = _object(sf)
    fn = getattr(sf.lib, f"sf_cache_{call}")
    assert fn(obj, None, *dict(base, **kw).values()) == status
    said = sf.lib.sf_cache_last_error(obj).decode()
    assert text in said, said
    assert fn(None, None, *base.values()) == sf.SF_ERR_INVALID_ARG


def test_weights_need_an_object_that_tracks_them(sf):
    obj = _object(sf, track_weights=0)
    assert sf.lib.sf_cache_attend(obj, None, *ATTEND.values()) == sf.SF_ERR_INVALID_ARG
    assert "track_weights" in sf.lib.sf_cache_last_error(obj).decode()


def test_binding_refuses_unknown_types(sf):
    for dtype in ("fp16", torch.float16, None, 2):
        with pytest.raises(ValueError):
            sf.PagedCache(n_q_heads=4, n_kv_heads=2, head_dim=64, dtype=dtype, page_size=16, max_seqs=1, max_len=16)


def test_null_objects(sf):
    assert sf.lib.sf_cache_sync_status(None, None) == sf.SF_ERR_INVALID_ARG
    assert sf.lib.sf_cache_destroy(None) == sf.SF_ERR_INVALID_ARG
    assert sf.lib.sf_cache_last_error(None) == b""


# ---------------------------------------------------------------- binding

@pytest.fixture
def bound(sf):
    """A PagedCache over an object of which only the shapes are filled in, with
    its checks set to CPU tensors: a call that they let through stops at the
    library's last check (no such device), one that they refuse raises."""
    c = sf.PagedCache.__new__(sf.PagedCache)
    obj = _object(sf)
    c.keep, c.cache, c.device, c.dtype, c.shapes = obj, None, torch.device("cpu"), torch.bfloat16, _shapes(sf)
    c._bind(ctypes.addressof(obj), -1)
    return c


def _let_through(sf, call):
    with pytest.raises(sf.SpecFoldError) as e:
        call()
    assert e.value.status == sf.SF_ERR_INVALID_ARG
    return e


def _reached_device_check(c, sf):
    return "lives on device" in sf.lib.sf_cache_last_error(c.keep).decode()


def _tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(qkv=torch.zeros(3, 8, 64, dtype=bf), index=torch.zeros(3, dtype=i32),
                table=torch.zeros(3, 4, dtype=i32), k=torch.zeros(9, 16, 2, 64, dtype=bf),
                v=torch.zeros(9, 16, 2, 64, dtype=bf), lens=torch.zeros(3, dtype=i32), q=torch.zeros(3, 4, 64, dtype=bf),
                w=torch.zeros(3, 2, 64))


def test_binding_lets_strided_rows_through(bound, sf):
    c, t = bound, _tensors()
    packed = torch.zeros(3, 704, dtype=torch.bfloat16)          # rows of a wider projection output
    qkv, table = packed[:, :512], torch.zeros(3, 11, dtype=torch.int32)[:, 2:6]
    calls = [lambda: c.append(qkv, t["index"], table, t["k"], t["v"], q=qkv[:, :256]),
             lambda: c.append(t["qkv"], t["index"], table, t["k"], t["v"], pos=t["index"], seq=t["index"],
                              q_gain=torch.ones(64)),
             lambda: c.attend(qkv[:, :256], t["k"], t["v"], table, t["lens"], weights=t["w"]),
             lambda: c.attend(t["q"], t["k"], t["v"], table, t["lens"], weights_out=t["w"], scale=2),
             lambda: c.evict(t["k"], t["v"], table, t["lens"], t["w"], 20, n_first=1),
             lambda: c.evict(t["k"], t["v"], table, t["lens"], t["w"], 20, k_out=t["k"].clone(), v_out=t["v"].clone(),
                             table_out=t["table"], weights_out=t["w"].clone(), lens_out=t["lens"])]
    for call in calls:
        _let_through(sf, call)
        assert _reached_device_check(c, sf)
    # what the library itself refuses comes back with its text
    _let_through(sf, lambda: c.append(packed[:, 1:513], t["index"], table, t["k"], t["v"]))
    assert "misaligned" in sf.lib.sf_cache_last_error(c.keep).decode()


@pytest.mark.parametrize("what", ["qkv dtype", "qkv inner", "qkv heads", "qkv dim", "k dtype", "k page", "v shape",
                                  "k stride", "table dtype", "table inner", "table dim", "index dtype", "index size",
                                  "index stride", "gain dtype", "gain size", "q rows", "q heads", "device",
                                  "no tensor"])
def test_binding_refuses_append(bound, sf, what):
    c, t = bound, _tensors()
    kw = {}
    if what == "qkv dtype":
        t["qkv"] = t["qkv"].float()
    elif what == "qkv inner":
        t["qkv"] = torch.zeros(3, 8, 128, dtype=torch.bfloat16)[..., ::2]
    elif what == "qkv heads":
        t["qkv"] = t["qkv"][:, :7]
    elif what == "qkv dim":
        t["qkv"] = t["qkv"][None]
        kw["q"] = t["q"]
    elif what == "k dtype":
        t["k"] = t["k"].float()
    elif what == "k page":
        t["k"] = t["k"][:, :8]
    elif what == "k stride":
        t["k"] = torch.zeros(9, 16, 2, 128, dtype=torch.bfloat16)[..., :64]
    elif what == "v shape":
        t["v"] = t["v"][:8]
    elif what == "table dtype":
        t["table"] = t["table"].long()
    elif what == "table inner":
        t["table"] = torch.zeros(4, 3, dtype=torch.int32).t()
    elif what == "table dim":
        t["table"] = t["table"][0]
    elif what == "index dtype":
        t["index"] = t["index"].long()
    elif what == "index size":
        t["index"] = t["index"][:2]
    elif what == "index stride":
        t["index"] = torch.zeros(6, dtype=torch.int32)[::2]
    elif what == "gain dtype":
        kw["q_gain"] = torch.ones(64, dtype=torch.bfloat16)
    elif what == "gain size":
        kw["k_gain"] = torch.ones(128)
    elif what == "q rows":
        kw["q"] = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    elif what == "q heads":
        kw["q"] = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    elif what == "device":
        kw["pos"] = torch.zeros(3, dtype=torch.int32, device="meta")
    else:
        t["index"] = [0, 1, 2]
    with pytest.raises(ValueError):
        c.append(t["qkv"], t["index"], t["table"], t["k"], t["v"], **kw)
    assert not _reached_device_check(c, sf)


def test_binding_refuses_cpu_tensors_on_a_gpu_object(sf, bound):
    c, t = bound, _tensors()
    c._bind(ctypes.addressof(c.keep), 0)
    with pytest.raises(ValueError, match="on device 0"):
        c.append(t["qkv"], t["index"], t["table"], t["k"], t["v"], q=t["q"])


def test_binding_refuses_attend_and_evict(bound, sf):
    c, t = bound, _tensors()
    for kw in (dict(weights=t["w"].double()), dict(weights=t["w"], weights_out=t["w"][:, :1]),
               dict(weights=t["w"], weights_out=t["w"][..., :63]), dict(out=t["q"][:2]), dict(weights=t["w"][..., ::2]),
               dict(weights=t["w"][0]), dict(out=t["q"].float())):
        with pytest.raises(ValueError):
            c.attend(t["q"], t["k"], t["v"], t["table"], t["lens"], **kw)
    with pytest.raises(ValueError):
        c.attend(t["q"][:2], t["k"], t["v"], t["table"], t["lens"])
    with pytest.raises(TypeError):
        c.attend(t["q"], t["k"], t["v"], t["table"], t["lens"], scale="x")
    for kw in (dict(k_out=t["k"]), dict(k_out=t["k"], v_out=t["v"], table_out=t["table"][:2]),
               dict(lens_out=t["lens"].long()), dict(kept=torch.zeros(3, 2, 19, dtype=torch.int32)),
               dict(weights_out=t["w"][..., :60]), dict(n_first=2 ** 31)):
        with pytest.raises(ValueError):
            c.evict(t["k"], t["v"], t["table"], t["lens"], t["w"], 20, **kw)
    with pytest.raises(TypeError):
        c.evict(t["k"], t["v"], t["table"], t["lens"], t["w"], 20.5, kept=torch.zeros(3, 2, 20, dtype=torch.int32))
    assert not _reached_device_check(c, sf)
