"""Host side of the search operators, on the CPU: what the C entry points refuse
before any launch, and their sizes."""
import ctypes

import pytest

from paged_kv_cache_283_gb300 import pa

F = ctypes.c_void_p(0x10000)
FAR = ctypes.c_void_p(1 << 40)
MIS8, MIS2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
BAD, SHAPE, OK = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED_SHAPE, pa.PA_OK


@pytest.fixture(scope="module")
def lib():
    return pa.lib()


# Every call below fails a check or has nothing to do: the fake addresses never
# reach a kernel.

def test_cross_attention_refusals(lib):
    def call(out=FAR, q=F, stride=1024, k=F, v=F, tables=F, mb=4, lens=F, start=F, max_q=3, n=2,
             T=6, hq=8, hkv=4, d=128, bs=16, nb=10, scale=0.1, ws=F, ml=F, counters=F, ctas=8,
             prepare=False):
        args = (out, q, stride, k, v, tables, mb, lens, start, max_q, n, T, hq, hkv, d, bs, nb,
                scale, ws, ml, counters, ctas)
        if prepare:
            h = ctypes.c_void_p(1)
            st = lib.pa_prepare_cross_attention(ctypes.byref(h), *args)
            assert not h.value
            return st
        return lib.pa_cross_attention(*args, None)

    for prepare in (False, True):
        for bad in (dict(out=None), dict(out=MIS8), dict(q=MIS8), dict(k=None), dict(v=MIS8),
                    dict(tables=MIS2), dict(lens=None), dict(start=None), dict(stride=1023),
                    dict(stride=1032 - 4), dict(stride=1016), dict(mb=0), dict(n=-1), dict(T=-1),
                    dict(max_q=-1), dict(hkv=3), dict(hkv=0), dict(nb=0), dict(scale=0.0),
                    dict(scale=-1.0), dict(scale=float("nan")), dict(ws=None), dict(ml=MIS8),
                    dict(counters=None), dict(ctas=0), dict(ctas=(1 << 20) + 1), dict(nb=1 << 27),
                    dict(mb=1 << 28), dict(out=F), dict(out=ctypes.c_void_p(0x10000 + 12288 - 16)),
                    dict(out=F, q=ctypes.c_void_p(0x10000 + 12288 - 16)),
                    dict(out=ctypes.c_void_p(0x10000 + 2 * (5 * 4096 + 1024) - 16),
                         stride=4096)):
            assert call(prepare=prepare, **bad) == BAD, bad
        for shape in (dict(d=96), dict(d=256), dict(bs=32), dict(hq=64), dict(hq=12)):
            assert call(prepare=prepare, stride=1 << 14, **shape) == SHAPE, shape
    for nothing in (dict(n=0), dict(T=0), dict(max_q=0)):
        assert call(out=None, **nothing) == OK
    assert lib.pa_prepare_cross_attention(None, *(F,) * 2, 0, *(F,) * 3, 1, F, F, *(1,) * 8, 0.1,
                                          F, F, F, 1) == BAD


def test_cross_attention_sizes(lib):
    assert lib.pa_cross_attention_ctas(152) == 304 and lib.pa_cross_attention_ctas(0) == 0
    assert lib.pa_cross_attention_rows(4, 4) == 16
    assert lib.pa_cross_attention_rows(1, 1) == 1
    assert lib.pa_cross_attention_rows(31, 4) == 124 and lib.pa_cross_attention_rows(33, 4) == 128
    assert lib.pa_cross_attention_rows(2 ** 31 - 1, 8) == 128
    assert lib.pa_cross_attention_rows(0, 4) == 0
    for d, g, bs, ok in ((64, 1, 16, 1), (128, 8, 16, 1), (128, 16, 16, 0), (128, 3, 16, 0),
                         (80, 1, 16, 0), (64, 1, 32, 0)):
        assert lib.pa_cross_attention_supported(d, g, bs) == ok


def test_read_cache_refusals(lib):
    beside = ctypes.c_void_p((1 << 40) + 1024)

    def call(kind=1, ko=FAR, vo=beside, stride=512, k=F, v=F, ks=F, vs=F, tables=F, mb=4, first=None,
             start=F, rows=9, n=2, T=12, slots=None, nob=0, hkv=4, d=128, bs=16, nb=10,
             prepare=False):
        args = (kind, ko, vo, stride, k, v, ks, vs, tables, mb, first, start, rows, n, T, slots,
                nob, hkv, d, bs, nb)
        if prepare:
            h = ctypes.c_void_p(1)
            st = lib.pa_prepare_read_cache(ctypes.byref(h), *args)
            assert not h.value
            return st
        return lib.pa_read_cache(*args, None)

    for prepare in (False, True):
        for bad in (dict(kind=3), dict(kind=-1), dict(kind=5), dict(ko=None), dict(vo=MIS8),
                    dict(k=None), dict(v=MIS8), dict(ks=None), dict(vs=MIS8), dict(kind=0),
                    dict(kind=4), dict(tables=MIS2), dict(start=None), dict(first=MIS2),
                    dict(stride=511), dict(stride=504), dict(stride=516), dict(mb=0),
                    dict(rows=-1), dict(n=-1), dict(T=-1), dict(hkv=0), dict(nb=0),
                    dict(slots=F), dict(slots=ctypes.c_void_p(0x10004), nob=3), dict(mb=1 << 28),
                    dict(ko=F), dict(vo=FAR), dict(vo=ctypes.c_void_p(0x10000 + 10 * 16 * 512 - 16)),
                    dict(ko=ctypes.c_void_p(0x10000 - 16)),
                    dict(ko=ctypes.c_void_p(0x10000 - 16), slots=F, nob=1)):
            assert call(prepare=prepare, **bad) == BAD, bad
        for shape in (dict(d=96), dict(bs=32), dict(n=70000)):
            assert call(prepare=prepare, **shape) == SHAPE, shape
    for nothing in (dict(n=0), dict(T=0), dict(rows=0)):
        assert call(ko=None, **nothing) == OK
    assert lib.pa_prepare_read_cache(None, 1, F, F, 512, F, F, F, F, F, 4, None, F, 1, 1, 1, None,
                                     0, 4, 128, 16, 10) == BAD


def test_beam_select_refusals(lib):
    def call(out=F, parents=F, tokens=F, fin_out=None, logits=F, stride=100, dtype=0, scores=FAR,
             fin=None, eos=-1, n=2, beams=4, keep=8, vocab=100, ws=F, counters=F, flags=0,
             prepare=False):
        args = (out, parents, tokens, fin_out, logits, stride, dtype, scores, fin, eos, n, beams,
                keep, vocab, ws, counters, flags)
        if prepare:
            h = ctypes.c_void_p(1)
            st = lib.pa_prepare_beam_select(ctypes.byref(h), *args)
            assert not h.value
            return st
        return lib.pa_beam_select(*args, None)

    odd = ctypes.c_void_p(0x10001)
    for prepare in (False, True):
        for bad in (dict(out=None), dict(parents=MIS2), dict(tokens=None), dict(logits=None),
                    dict(logits=odd), dict(logits=MIS2, dtype=2), dict(scores=None),
                    dict(ws=MIS8), dict(counters=None), dict(stride=99), dict(dtype=3),
                    dict(dtype=-1), dict(eos=100), dict(eos=-2), dict(fin=F), dict(n=-1),
                    dict(beams=0), dict(keep=0), dict(vocab=0), dict(flags=2),
                    dict(flags=pa.PA_BEAM_IN_PLACE),
                    dict(out=ctypes.c_void_p(0x20000), scores=ctypes.c_void_p(0x20000)),
                    dict(out=ctypes.c_void_p(0x20000), fin=F, fin_out=F, eos=3),
                    dict(scores=F, keep=4, out=ctypes.c_void_p(0x10000 + 4)),
                    dict(scores=ctypes.c_void_p(0x10000 + 28), keep=4),
                    dict(keep=4, fin=F, fin_out=ctypes.c_void_p(0x10000 + 7), eos=3)):
            assert call(prepare=prepare, **bad) == BAD, bad
        for shape in (dict(beams=33), dict(keep=65), dict(n=20000),
                      dict(vocab=(1 << 27) + 1, stride=1 << 28)):
            assert call(prepare=prepare, **shape) == SHAPE, shape
    assert call(n=0, out=None) == OK
    assert lib.pa_prepare_beam_select(None, *(F,) * 5, 100, 0, F, None, -1, 2, 4, 8, 100, F, F,
                                      0) == BAD


def test_beam_select_workspace(lib):
    size = lib.pa_beam_select_workspace_bytes
    for dtype in (0, 1, 2):
        for n, w, k, v in ((1, 1, 1, 1), (1, 4, 8, 32000), (64, 4, 8, 128256), (3, 32, 64, 50257)):
            b = size(n, w, k, v, dtype)
            assert b % (n * w * 8 * (k + 1)) == 0 and b > 0       # whole parts of every row
    assert size(1, 33, 8, 100, 0) == 0 and size(1, 4, 65, 100, 0) == 0
    assert size(1, 4, 8, 100, 3) == 0 and size(1, 4, 8, 0, 0) == 0


def test_reorder_refusals(lib):
    def call(states=(0x10000,), parents=FAR, groups=2, beams=4, row=64, stride=64, n=None,
             prepare=False):
        ptrs = None if states is None else (ctypes.c_void_p * max(1, len(states)))(*states)
        n = len(states or ()) if n is None else n
        args = (ptrs, n, parents, groups, beams, row, stride)
        if prepare:
            h = ctypes.c_void_p(1)
            st = lib.pa_prepare_reorder_states(ctypes.byref(h), *args)
            assert not h.value
            return st
        return lib.pa_reorder_states(*args, None)

    for prepare in (False, True):
        for bad in (dict(states=None, n=1), dict(states=(0x10000, None)), dict(parents=None),
                    dict(parents=MIS2), dict(groups=-1), dict(beams=0), dict(row=-1),
                    dict(stride=63), dict(n=-1), dict(states=(0x10000, 0x10000)),
                    dict(states=(0x30000, 0x10000, 0x30000 + 511)),
                    dict(states=(0x10000, 0x10000 + 128), stride=100),
                    dict(states=(0x10000, 0x10000 + 64), stride=127),
                    dict(states=(0x10000, 0x10000 + 7 * 100 + 63), stride=100),
                    dict(parents=ctypes.c_void_p(0x10000 + 508)),
                    dict(parents=ctypes.c_void_p(0x10000 - 28))):
            assert call(prepare=prepare, **bad) == BAD, bad
        for shape in (dict(beams=33), dict(groups=65536), dict(row=1 << 41, stride=1 << 41)):
            assert call(prepare=prepare, **shape) == SHAPE, shape
    for nothing in (dict(states=()), dict(groups=0), dict(row=0)):
        assert call(parents=None, **nothing) == OK
    assert lib.pa_prepare_reorder_states(None, None, 0, F, 1, 1, 1, 1) == BAD
