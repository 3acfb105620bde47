"""Cross attention's two orders of work.  With more (tile, sequence) pairs than a CTA
looks through at its start, the units go by sequence, head and tile in place of tile,
sequence and head: many single steps beside one long prompt."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

from test_gpu_cross import Case

pytestmark = pytest.mark.gpu


def _mixed(seed, n, hkv, prompts):
    """n single queries, some of them in place of prompts of up to 512, 8 heads a KV head:
    tiles of 16 queries."""
    rng = np.random.default_rng(seed)
    counts = np.ones(n, dtype=np.int32)
    counts[5], counts[6] = 0, 3
    for at, m in prompts.items():
        counts[at] = m
    sources = rng.choice([0, 1, 15, 64, 65, 130, 700], n)
    sources[list(prompts)] = [700, 1300, 0][:len(prompts)]
    return Case(seed, sources, counts, 8 * hkv, hkv, 64, gap=3)


# 32 tiles of the longest prompt: 512 sequences are 16,384 pairs, the most that go by tile
@pytest.mark.parametrize("n,hkv,prompts", [(512, 1, {77: 512}), (513, 1, {77: 512}),
                                           (520, 2, {200: 512}),
                                           (530, 2, {0: 512, 300: 200, 529: 37})])
def test_both_orders(n, hkv, prompts):
    pa.pa_clear_device_error()
    c = _mixed(n, n, hkv, prompts)
    q, k, v, tables, sources, start = c.on_gpu()
    rows = int(c.counts.sum())
    for ctas in (304, 1, 7, 50, 1000):
        out = torch.full_like(q, 7.0)
        ws = pa.CrossWorkspace(512, 8 * hkv, hkv, 64, ctas=ctas)
        ws.ws_out.fill_(float("nan"))
        ws.ws_ml.fill_(float("nan"))
        seen = []
        for again in range(3):
            out[:rows] = float("nan")
            pa.pa_cross_attention(out, q, k, v, tables, sources, start, 512, c.scale, ws)
            torch.cuda.synchronize()
            assert not ws.counters.any(), (ctas, again)
            assert bool((out[rows:] == 7.0).all())
            seen.append(out[:rows].view(torch.int16).clone())
            assert torch.equal(seen[-1], seen[0]), "a call repeats itself"
        c.check(out, f"{ctas} CTAs")
    assert pa.pa_get_device_error() == 0


def test_many_sequences_by_sequence():
    """More sequences than the pairs that go by tile, of a tile each; then a bad one."""
    pa.pa_clear_device_error()
    rng = np.random.default_rng(64)
    n = 16500
    c = Case(64, rng.choice([0, 1, 17, 64, 70], n), rng.integers(0, 3, n), 1, 1, 64)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, 7.0)
    ws = pa.CrossWorkspace(2, 1, 1, 64)
    for _ in range(2):
        pa.pa_cross_attention(out, q, k, v, tables, sources, start, 2, c.scale, ws)
    torch.cuda.synchronize()
    assert not ws.counters.any() and pa.pa_get_device_error() == 0
    c.check(out)
    at = int(np.flatnonzero((c.counts == 2) & (c.sources > 0))[100])
    lo, hi = c.start[at:at + 2].tolist()
    good = out[lo:hi].clone()
    sources[at] = tables.shape[1] * 16 + 1
    out.fill_(7.0)
    pa.pa_cross_attention(out, q, k, v, tables, sources, start, 2, c.scale, ws)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_CONTEXT_LEN
    pa.pa_clear_device_error()
    assert bool((out[lo:hi] == 7.0).all()) and not ws.counters.any()
    out[lo:hi] = good
    c.check(out)
