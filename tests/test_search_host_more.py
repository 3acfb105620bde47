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


@pytest.mark.parametrize("prepare", [False, True])
def test_read_cache_outputs_that_meet(prepare):
    """K and V rows that share bytes are refused, also where neither begins with the other:
    which of the two a place would end with is nobody's choice."""
    def call(apart, stride=1024, slots=None, nob=0, T=12):
        ko, vo = (1 << 40, (1 << 40) + apart) if apart >= 0 else ((1 << 40) - apart, 1 << 40)
        args = (1, ko, vo, stride, F, F, F, F, F, 4, None, F, 9, 2, T, slots, nob, 4, 128, 16, 10)
        if prepare:
            return pa.lib().pa_prepare_read_cache(ctypes.byref(ctypes.c_void_p()), *args)
        return pa.lib().pa_read_cache(*args, None)

    # 12 rows of 1024 bytes, 2048 apart
    for apart in (0, 16, 1008, 1040, 2032, 2048, 2064, 4096, 11 * 2048, 11 * 2048 + 1008):
        assert call(apart) == BAD and call(-apart) == BAD, apart
    for apart in (512, 1008, 11 * 1024 + 16):               # and with nothing between them
        assert call(apart, stride=512) == BAD and call(-apart, stride=512) == BAD, apart
    for apart in (16, 3 * 16384 - 16):                      # pools of 3 blocks of 16 KiB
        assert call(apart, slots=F, nob=3) == BAD and call(-apart, slots=F, nob=3) == BAD, apart
