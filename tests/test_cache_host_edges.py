"""Paged cache without a GPU, at the edges: refusals of calls that the kernels
could not answer."""
import numpy as np
import pytest

from test_cache_host import APPEND, ATTEND, EVICT, _object, sf  # noqa: F401  (sf is a fixture)


def _says(sf, call, base, **kw):
    """Status and text of a call on an object of which only the shapes are filled in."""
    obj = _object(sf)
    status = getattr(sf.lib, f"sf_cache_{call}")(obj, None, *dict(base, **kw).values())
    return status, sf.lib.sf_cache_last_error(obj).decode()


@pytest.mark.parametrize("scale,fits", [(2.358e38, True), (-2.358e38, True), (1e-45, True), (0.0, True),
                                        (2.36e38, False), (-3.4e38, False), (float("inf"), False)])
def test_scales_that_fp32_cannot_hold_in_log2_units(sf, scale, fits):
    assert (abs(scale) * np.log2(np.e) <= float(np.finfo(np.float32).max)) == fits
    status, text = _says(sf, "attend", ATTEND, q=16, out=1 << 20, scale=scale)
    assert status == sf.SF_ERR_INVALID_ARG           # at the latest there is no device
    assert ("lives on device" in text) == fits and ("scale" in text) != fits


# rows of 512 elements (append: qkv) and 256 (queries and outputs) of bf16, 1,024 and 512 bytes; far apart unless said
FAR = 1 << 20
OVERLAPS = [
    ("append", APPEND, dict(qkv=FAR, q_out=FAR, ld_q=512), None),                      # in place
    ("append", APPEND, dict(qkv=FAR, q_out=FAR, T=1), None),                           # one row: strides do not matter
    ("append", APPEND, dict(qkv=FAR, q_out=FAR), "q_out"),                             # packed over the rows it reads
    ("append", APPEND, dict(qkv=FAR, q_out=FAR + 512, ld_q=512), "q_out"),             # over the keys
    ("append", APPEND, dict(qkv=FAR, ld_qkv=768, q_out=FAR + 1024, ld_q=768), None),   # beside the row
    ("append", APPEND, dict(qkv=FAR, q_out=FAR + 2 * 1024, T=2), None),                # right behind the last row
    ("append", APPEND, dict(qkv=FAR, q_out=FAR + 2 * 1024 - 16, T=2), "q_out"),
    ("append", APPEND, dict(qkv=FAR, q_out=FAR - 3 * 512), None),                      # right before the first
    ("attend", ATTEND, dict(q=FAR, out=FAR), "out"),
    ("attend", ATTEND, dict(q=FAR, out=FAR, S=1), "out"),
    ("attend", ATTEND, dict(q=FAR, out=FAR + 512), "out"),
    ("attend", ATTEND, dict(q=FAR, out=FAR + 4 * 512), None),
    ("attend", ATTEND, dict(q=FAR, out=FAR + 512, ld_q=512, ld_out=512), None),        # columns of one wide array
    ("attend", ATTEND, dict(q=FAR + 512, out=FAR, ld_q=512, ld_out=512), None),
    ("attend", ATTEND, dict(q=FAR, out=FAR + 496, ld_q=512, ld_out=512), "out"),
    ("attend", ATTEND, dict(q=FAR + 16, out=FAR + 512, ld_q=512, ld_out=512), "out"),
    ("attend", ATTEND, dict(q=FAR, w_in=FAR * 2, w_out=FAR * 2 + 4 * 64), "weights_out"),
    ("attend", ATTEND, dict(q=FAR, w_in=FAR * 2, w_out=FAR * 2 + 4 * 2 * 64 * 4), None),
    ("attend", ATTEND, dict(q=FAR, w_in=None, w_out=FAR * 2), None),
    ("evict", EVICT, dict(w=FAR, w_out=FAR), None),
    ("evict", EVICT, dict(w=FAR, w_out=FAR + 4), "weights_out"),
    ("evict", EVICT, dict(w=FAR + 4 * 2 * 64 * 4, w_out=FAR), None),
    ("evict", EVICT, dict(lens=FAR, lens_out=FAR + 4), "lens_out"),
    ("evict", EVICT, dict(lens=FAR, lens_out=FAR + 16), None),
]


@pytest.mark.parametrize("call,base,kw,refused", OVERLAPS)
def test_outputs_that_overlap_inputs_are_refused(sf, call, base, kw, refused):
    """Blocks of a call run in any order: an output over a part of an input that
    another block has still to read would change results from run to run."""
    if call == "append":
        kw = dict(dict(k=1 << 30, v=1 << 31), **kw)
    status, text = _says(sf, call, base, **kw)
    assert status == sf.SF_ERR_INVALID_ARG           # at the latest there is no device
    assert ("lives on device" in text) == (refused is None), text
    assert refused is None or refused in text
