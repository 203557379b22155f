"""Rules and refusals around the paged cache's rows and shared prefixes that
need no GPU."""
import pytest

from test_cache_host import sf  # noqa: F401
from test_cache_rows_host import _rows_object


@pytest.mark.parametrize("signal,status", [(0, 0), (1, 0), (13, 0), (14, 1), (-1, 1), (2 ** 31 - 1, 1)])
def test_injected_stalls_are_known_signals(sf, signal, status):  # noqa: F811
    obj = _rows_object(sf)
    assert sf.lib.sf_cache_inject_stall(obj, signal) == status
    assert ("no signal" in sf.lib.sf_cache_last_error(obj).decode()) == (status != 0)
    assert sf.lib.sf_cache_inject_stall(None, signal) == sf.SF_ERR_INVALID_ARG
