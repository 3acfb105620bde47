"""More of what the C entry points of the search operators refuse before any launch."""
import ctypes

import pytest

from paged_kv_cache_283_gb300 import pa

F = ctypes.c_void_p(0x10000)
FAR = ctypes.c_void_p(1 << 40)
BAD = pa.PA_ERR_INVALID_ARG


# Every call below fails a check, or ends where it asks for a device: the fake addresses
# never reach a kernel.

@pytest.mark.parametrize("prepare", [False, True])
def test_cross_attention_tables_past_31_bits(prepare):
    """A source's length plus a chunk's 63 keys more: the last tables of 31-bit capacity
    would wrap around where the chunks are counted."""
    def call(mb):
        args = (FAR, F, 1024, F, F, F, mb, F, F, 3, 2, 6, 8, 4, 128, 16, 10, 0.1, F, F, F, 8)
        if prepare:
            return pa.lib().pa_prepare_cross_attention(ctypes.byref(ctypes.c_void_p()), *args)
        return pa.lib().pa_cross_attention(*args, None)

    for mb in ((1 << 27) - 1, (1 << 27) - 2, (1 << 27) - 3, (1 << 27) - 4, 1 << 27):
        assert call(mb) == BAD, mb
