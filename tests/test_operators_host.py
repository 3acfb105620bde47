"""Host side of the operators around the cache, on the CPU: checks that need no
device."""
import ctypes

import pytest

from paged_kv_cache_283_gb300 import pa


@pytest.fixture(scope="module")
def lib():
    return pa.lib()


def test_awaiting_no_event_is_refused(lib):
    assert lib.pa_await_event(None, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_await_event(None, ctypes.c_void_p(0x10000)) == pa.PA_ERR_INVALID_ARG
