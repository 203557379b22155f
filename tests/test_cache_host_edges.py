"""Paged cache without a GPU, at the edges: refusals of calls that the kernels
could not answer."""
import numpy as np
import pytest

from test_cache_host import ATTEND, _object, sf  # noqa: F401  (sf is a fixture)


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
