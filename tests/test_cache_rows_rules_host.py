"""Rules and refusals around the paged cache's rows and shared prefixes that
need no GPU."""
import ctypes
import os
import subprocess

import pytest

from test_cache_host import sf  # noqa: F401
from test_cache_rows_host import _rows_object

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, so = d / "rules.cpp", d / "rules.so"
    src.write_text("""
#include "sf_cache_index.h"
extern "C" int tail_warps(int longest, long long segments, int most, int sms) {
  return sf::tail_warps(longest, segments, most, sms);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "sparse_reuse_gb300", "csrc"), str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.tail_warps.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


def test_no_warp_gets_a_long_tail(rules):
    """However many sequences there are: the table says how long one of them may be, not how long they are."""
    for sms in (1, 132, 152, 160):
        for segments in (1, 8, 18, 64, 151, 152, 153, 288, 1016, 8192, 32768, 4096 * 1024):
            for longest in list(range(1, 200)) + [256, 512, 3440, 16384]:
                w = rules.tail_warps(longest, segments, 4, sms)
                assert w in (0, 1, 2, 4) and longest <= 48 * w or w == 0
                assert w or longest > 4                    # the shortest always go by warps
    # 1,024 sequences of 8 KV heads that a table of 8,192 positions holds; 4,096 of them and 55,000 positions
    assert rules.tail_warps(512, 8192, 4, 152) == rules.tail_warps(3438, 32768, 4, 152) == 0
    # the branches of one request and of four, a ragged serving batch with up to 701 positions
    assert rules.tail_warps(2, 18, 4, 152) == 1 and rules.tail_warps(2, 288, 4, 152) == 1
    assert rules.tail_warps(44, 1016, 4, 152) == 2


@pytest.mark.parametrize("signal,status", [(0, 0), (1, 0), (13, 0), (14, 1), (-1, 1), (2 ** 31 - 1, 1)])
def test_injected_stalls_are_known_signals(sf, signal, status):  # noqa: F811
    obj = _rows_object(sf)
    assert sf.lib.sf_cache_inject_stall(obj, signal) == status
    assert ("no signal" in sf.lib.sf_cache_last_error(obj).decode()) == (status != 0)
    assert sf.lib.sf_cache_inject_stall(None, signal) == sf.SF_ERR_INVALID_ARG
