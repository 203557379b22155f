"""attend_rows and attend_shared on calls at the edge of what their
documentation allows (needs a GB300).  Tolerances are test_gpu_cache_rows.py's."""
import numpy as np
import pytest
import torch

from test_gpu_cache import DT, i32, sf  # noqa: F401
from test_gpu_cache_rows import check, check_rows, places, rows_inputs, run_rows, run_shared, shared_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 90, 300])
def test_rows_of_scale_zero_keep_nan_and_infinite_queries(sf, dtype, rows):  # noqa: F811
    """0 times a NaN or infinite score is NaN; finite queries get the values' mean."""
    a = rows_inputs(sf, (4, 2, 64), dtype, 16, [rows, 2], [300, 40])
    a["q"][1, 0, 5] = torch.nan
    a["q"][rows - 1, 3, 63] = torch.inf
    a["q"][rows, 2, 0] = -torch.inf
    bad = torch.zeros(a["q"].shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[rows - 1, 3] = bad[rows, 2] = True
    out, lse = run_rows(a, scale=0.0)
    a["c"].sync()
    live = slice(0, rows + 2)
    assert torch.equal(~torch.isfinite(out[live]).any(-1), bad[live])
    assert torch.equal(torch.isnan(out[live]).all(-1), bad[live]) and torch.equal(torch.isnan(lse[live]), bad[live])
    clean = a["q"].clone()
    clean[bad] = 0.0
    out[bad], lse[bad] = (t[bad] for t in run_rows(dict(a, q=clean), scale=0.0))
    check_rows(dict(a, q=clean), out, lse, dtype, scale=0.0)
    a["c"].close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members", [4, 80])
def test_shared_of_scale_zero_keeps_nan_queries(sf, dtype, members):  # noqa: F811
    """Whether or not a sequence has positions of its own."""
    tails = [7 * (s % 2) for s in range(members)]
    a = shared_inputs(sf, (4, 2, 64), dtype, 16, [members], [100], 0, 0, tails)
    bad = torch.zeros(a["q"].shape[:2], dtype=torch.bool, device="cuda")
    for s, h, x in ((0, 1, torch.nan), (1, 2, torch.nan), (2, 0, torch.inf), (3, 3, -torch.inf)):
        a["q"][s, h, 9] = x
        bad[s, h] = True
    out, lse = run_shared(a, scale=0.0)
    a["c"].sync()
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(lse), bad)
    q = a["q"].clone()
    q[bad] = 0.0
    for s in range(members):
        if not bad[s].any():
            slots = np.r_[places(a["ptable"], 0, 100, 16), places(a["table"], s, tails[s], 16)]
            check(a, s, q[s:s + 1], out[s:s + 1], lse[s:s + 1], slots, 0.0, dtype)
    a["c"].close()


@pytest.mark.parametrize("heads,dtype,n,long", [((40, 8, 128), "bf16", 1024, 8192), ((12, 2, 128), "bf16", 36, 4096),
                                                ((40, 8, 128), "bf16", 128, 700), ((8, 8, 64), "f32", 200, 1000)])
def test_shared_one_long_tail_among_short_ones(sf, heads, dtype, n, long):  # noqa: F811
    tails = [(50 * s + 1) % 51 for s in range(n)]
    tails[n // 3] = long
    a = shared_inputs(sf, heads, dtype, 32, [n - 2], [70], 1, 1, tails)
    out, lse = run_shared(a)
    a["c"].sync()
    pre = places(a["ptable"], 0, 70, 32)
    for s in (0, 1, 2, n // 3 - 1, n // 3, n // 3 + 1, n - 2, n - 1):
        slots = np.r_[pre if 1 <= s < n - 1 else pre[:0], places(a["table"], s, tails[s], 32)]
        check(a, s, a["q"][s:s + 1], out[s:s + 1], lse[s:s + 1], slots, heads[2] ** -0.5, dtype)
    assert torch.isfinite(out).all()
    a["c"].close()


@pytest.mark.parametrize("heads,page,members,prefix,tails", [
    ((4, 2, 64), 16, 3, 50, [5000, 1, 300]),                  # chunks, joined by the last block to arrive
    ((2, 1, 64), 24, 1, 70, [40000]),                         # cut over more blocks than that: the join kernel
    ((12, 2, 128), 7, 2, 130, [30000, 9, 0]),
    ((8, 8, 64), 16, 20, 33, [3000] + [40 * s for s in range(29)]),   # a line of short and cut segments
    ((16, 1, 128), 100, 0, 10, [3000, 0, 2000]),              # a group of none
])
def test_shared_long_tails_in_fp32(sf, heads, page, members, prefix, tails):  # noqa: F811
    """Own positions too many for a warp: planned blocks, as in bf16."""
    behind = len(tails) - members
    a = shared_inputs(sf, heads, "f32", page, [members], [prefix], 0, behind, tails)
    out, lse = run_shared(a)
    a["c"].sync()
    for s, n in enumerate(tails):
        pre = places(a["ptable"], 0, prefix, page)[:prefix if s < members else 0]
        check(a, s, a["q"][s:s + 1], out[s:s + 1], lse[s:s + 1], np.r_[pre, places(a["table"], s, n, page)],
              heads[2] ** -0.5, "f32")
    o2, l2 = run_shared(a)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    a["c"].close()
