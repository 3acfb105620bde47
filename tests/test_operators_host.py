"""Host side of the operators around the cache, on the CPU: checks that need no
device."""
import ctypes
import heapq

import numpy as np
import pytest

from paged_kv_cache_283_gb300 import pa


@pytest.fixture(scope="module")
def lib():
    return pa.lib()


def test_awaiting_no_event_is_refused(lib):
    assert lib.pa_await_event(None, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_await_event(None, ctypes.c_void_p(0x10000)) == pa.PA_ERR_INVALID_ARG


# The launch-time model of the 4-bit cache's and the changed scores' steps, restated:
# (µs per token of 128 dims, per CTA, per merging CTA, of a merge as its own launch)
COSTS = {"int4": (0.0045, 2.0, 1.0, 5.0), "bf16-biased": (0.022, 4.0, 1.0, 3.0)}
SIZES = [256, 384, 512, 640, 768, 1024, 1280, 1536, 1792, 2048, 4096]
SIZES4 = sorted(SIZES + [2304, 2560, 2816, 3328, 3584, 5120, 8192])


def _ctas(kind, group, d, part):
    """CTAs an SM, and what a token costs beside four of them."""
    if kind == "bf16-biased":
        return (3 if group <= 4 else 1), 1.0
    # steps of four blocks at D = 128: groups of 8, and partitions from 4096 tokens on
    four = d == 64 or (group <= 4 and part < 4096)
    return (4, 1.0) if four else (3, 0.65)


def _time(kind, ctx, hkv, group, d, part, sms, ordered):
    token, cta, merge, apart_us = COSTS[kind]
    ctas, share = _ctas(kind, group, d, part)
    parts = [-(-n // part) for n in ctx]
    apart = max(parts) > 16
    items = []
    for z in range(max(1, *parts)):
        for n, k in zip(ctx, parts):
            if z < max(k, 1):
                tokens = max(0, min(part, n - z * part))
                items.append(token * d / 128 * share * tokens + cta +
                             (merge if k > 1 and not apart else 0.0))
    if ordered:
        items.sort(reverse=True)
    free = [0.0] * (sms * ctas)
    for t in items:
        for _ in range(hkv):
            heapq.heapreplace(free, free[0] + t)
    return max(free) + (apart_us if apart else 0.0)


@pytest.mark.parametrize("kind", ["int4", "bf16-biased"])
@pytest.mark.parametrize("seed", range(5))
def test_partition_size_follows_the_stated_model(kind, seed):
    rng = np.random.default_rng(seed)
    for _ in range(4):
        hkv, group = int(rng.choice([1, 2, 4, 8])), int(rng.choice([2, 4, 8]))
        d, sms = int(rng.choice([64, 128])), int(rng.choice([148, 152]))
        top = int(rng.choice([300, 4000, 50000, 131072]))
        b = int(rng.integers(1, max(2, 200000 // top)))
        ctx = rng.integers(1, top, size=min(b, 200)).tolist()
        ordered = bool(rng.integers(0, 2))
        want, best = 0, 0.0
        for part in SIZES4 if kind == "int4" else SIZES:
            t = _time(kind, ctx, hkv, group, d, part, sms, ordered)
            if want == 0 or t <= best + 1e-9:
                want, best = part, t
            if part >= max(ctx):
                break
        got = pa.splitk_partition_size(ctx, hkv * group, hkv, d, kind, num_sms=sms,
                                       ordered=ordered)
        assert got == want, (kind, hkv, group, d, sms, ordered, len(ctx), max(ctx))


def test_partition_sizes_of_long_4bit_contexts_pass_4096():
    sizes = {pa.splitk_partition_size([131072] * n, 32, 8, 128, "int4", num_sms=152, ordered=True)
             for n in (1, 4, 8, 16)}
    assert all(s in SIZES4 for s in sizes) and max(sizes) >= 4096
