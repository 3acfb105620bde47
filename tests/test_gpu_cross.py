"""Cross attention over paged source states on the GPU (pa_cross_attention)
against the float64 oracle: every group and head_dim, sources from none to
several CTAs' worth, queries from one to many tiles, strided queries, rows of no
sequence, NaN past the sources, bad lengths and blocks.

Tolerance per element, from the roundings: the output to bf16, 2^-8 of itself; each
weight to two bf16 parts, 2^-16 of it, and its exponential, 2^-20, so their sum of
the weighted mean of |V|; the scores' accumulation in fp32 (D terms, truncated: D 2^-23 of sum |q K| each) which moves
every weight by twice that; the accumulation over n keys, n 2^-23 of the mean."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import search as OS
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import bf16_to_f64, dev_bf16

pytestmark = pytest.mark.gpu


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


class Case:
    def __init__(self, seed, sources, counts, hq, hkv, d, gap=0, scale=None):
        """gap: rows of no sequence behind the last one.  Hidden places are NaN."""
        rng = np.random.default_rng(seed)
        self.sources, self.counts = np.array(sources, np.int32), np.array(counts, np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        nblk = -(-self.sources // 16)
        nb = int(nblk.sum()) + 3
        perm = rng.permutation(nb)
        self.tables = np.full((len(sources), max(1, int(nblk.max()))), -1, dtype=np.int32)
        self.k, self.v = (normal_bf16(rng, (nb, hkv, 16, d)) for _ in "kv")
        at = 0
        for b, n in enumerate(nblk.tolist()):
            self.tables[b, :n] = perm[at:at + n]
            at += n
            if self.sources[b] % 16:
                for pool in (self.k, self.v):
                    pool[self.tables[b, n - 1], :, self.sources[b] % 16:] = 0x7FC0
        for pool in (self.k, self.v):
            pool[perm[at:]] = 0x7FC0            # blocks of no sequence
        self.q = normal_bf16(rng, (int(self.counts.sum()) + gap, hq, d))
        self.hq, self.hkv, self.d = hq, hkv, d
        self.scale = d ** -0.5 if scale is None else scale

    def on_gpu(self):
        return (dev_bf16(self.q), dev_bf16(self.k), dev_bf16(self.v), _dev(self.tables),
                _dev(self.sources), _dev(self.start))

    def check(self, out, what=""):
        rows = int(self.counts.sum())
        got = bf16_to_f64(out)[:rows]
        assert np.isfinite(got).all(), what
        ref, mean = OS.cross_attention(self.q[:rows], self.k, self.v, self.tables, self.sources,
                                       self.counts, self.scale)
        q = np.abs(bf16_bits_to_f64(self.q)).sum(-1).max()
        kmax = np.nan_to_num(np.abs(bf16_bits_to_f64(self.k))).max()
        moved = 2 * self.d * 2.0 ** -23 * self.scale * q * kmax
        n = np.repeat(self.sources, self.counts)[:, None, None]
        tol = 2.0 ** -8 * np.abs(ref) + mean * (2.0 ** -16 + 2.0 ** -20 + moved + (n + 64) * 2.0 ** -23)
        bad = np.abs(got - ref) > tol * 1.0001 + 1e-30
        assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])
        assert not got[n[:, 0, 0] == 0].any(), "no source: zeros"


def _call(c, gap_value=7.0, **kw):
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, gap_value)
    ws = pa.CrossWorkspace(max(1, int(c.counts.max())), c.hq, c.hkv, c.d)
    pa.pa_cross_attention(out, q, k, v, tables, sources, start, max(1, int(c.counts.max())),
                          c.scale, ws, **kw)
    torch.cuda.synchronize()
    assert not ws.counters.any(), "counters are left at zero"
    assert bool((out[int(c.counts.sum()):] == gap_value).all()), "rows of no sequence are left"
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_groups_and_heads(d, group):
    pa.pa_clear_device_error()
    c = Case(group, [37, 1, 200], [4, 1, 3], 2 * group, 2, d, gap=2)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_source_lengths(d, n):
    pa.pa_clear_device_error()
    c = Case(10 + n, [n, 40], [5, 2], 4, 2, d)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (128, 8)])
@pytest.mark.parametrize("m", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300])
def test_query_counts(d, group, m):
    pa.pa_clear_device_error()
    c = Case(50 + m, [100, 300, 5], [m, 3, m], 2 * group, 2, d, gap=1)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (128, 4, 1), (128, 16, 2)])
def test_long_sources_shared_by_ctas(d, hq, hkv):
    pa.pa_clear_device_error()
    c = Case(80 + hq, [9000, 33, 0, 5000], [4, 2, 1, 3], hq, hkv, d)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 50, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_any_number_of_ctas(ctas, d):
    """Few CTAs walk many units each, many share units: the same result to rounding."""
    pa.pa_clear_device_error()
    c = Case(90, [700, 0, 64, 1300, 3], [3, 4, 40, 1, 2], 8, 2, d)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, float("nan"))
    ws = pa.CrossWorkspace(40, 8, 2, d, ctas=ctas)
    ws.ws_out.fill_(float("nan"))
    ws.ws_ml.fill_(float("nan"))
    for _ in range(2):
        pa.pa_cross_attention(out, q, k, v, tables, sources, start, 40, c.scale, ws)
    torch.cuda.synchronize()
    c.check(out, f"{ctas} CTAs")
    assert not ws.counters.any() and pa.pa_get_device_error() == 0


@pytest.mark.parametrize("ctas", [1, 2, 5, 40, 304])
@pytest.mark.parametrize("d,m", [(64, 5), (128, 4), (128, 13)])
def test_any_number_of_ctas_for_few_rows(ctas, d, m):
    pa.pa_clear_device_error()
    c = Case(100 + m, [9000, 0, 64, 1300, 3, 2500], [m, 1, m, 1, 0, m], 8, 2, d)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, float("nan"))
    ws = pa.CrossWorkspace(m, 8, 2, d, ctas=ctas)
    ws.ws_out.fill_(float("nan"))
    ws.ws_ml.fill_(float("nan"))
    for _ in range(3):
        pa.pa_cross_attention(out, q, k, v, tables, sources, start, m, c.scale, ws)
    torch.cuda.synchronize()
    c.check(out, f"{ctas} CTAs")
    assert not ws.counters.any() and pa.pa_get_device_error() == 0


def test_many_sequences():
    """More sequences than a CTA has threads, with empty ones among them."""
    pa.pa_clear_device_error()
    rng = np.random.default_rng(7)
    sources = rng.integers(0, 90, 700)
    sources[::5] = 0
    counts = rng.integers(0, 3, 700)
    c = Case(91, sources, counts, 2, 1, 64)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


def test_nothing_but_empty_sources():
    pa.pa_clear_device_error()
    c = Case(92, [0, 0, 0], [2, 0, 130], 4, 1, 128, gap=1)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("scale", [1e-4, 3.0])
def test_flat_and_sharp_scores(scale):
    """Sharp ones climb past the reference maximum, chunk by chunk."""
    pa.pa_clear_device_error()
    c = Case(93, [1500, 200], [3, 20], 4, 2, 128, scale=scale)
    order = np.argsort(bf16_bits_to_f64(c.k[c.tables[0, :93]]).sum((1, 2, 3)))
    c.tables[0, :93] = c.tables[0, order]       # (the last block is kept last)
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


def test_rising_scores():
    """Every chunk's scores pass the last one's by more than the reference allows for."""
    pa.pa_clear_device_error()
    c = Case(94, [640], [2], 2, 1, 64, scale=1.0)
    k = bf16_bits_to_f64(c.k)
    one = np.zeros((640, 64), dtype=np.float32)
    one[:, 0] = np.arange(640) // 64 * 2
    for j in range(640):
        k[c.tables[0, j // 16], 0, j % 16] = one[j]
    c.k = (k.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    c.q[:] = 0
    c.q[..., 0] = 0x4100                        # 8: scores of 16 a chunk
    c.check(_call(c))
    assert pa.pa_get_device_error() == 0


def test_strided_queries():
    pa.pa_clear_device_error()
    c = Case(95, [70, 300], [9, 33], 8, 2, 128, gap=3)
    q, k, v, tables, sources, start = c.on_gpu()
    wide = torch.full((q.shape[0], 11, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = q
    out = torch.zeros_like(q)
    ws = pa.CrossWorkspace(33, 8, 2, 128)
    pa.pa_cross_attention(out, wide[:, 2:10], k, v, tables, sources, start, 33, c.scale, ws)
    c.check(out)
    with pytest.raises(ValueError):
        pa.pa_cross_attention(out, wide[:, 1:9].transpose(0, 1), k, v, tables, sources, start, 33,
                              c.scale, ws)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("m", [5, 50, 300])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80])
def test_a_bad_query_keeps_to_itself(m, bad):
    """A query of NaN or infinities gives NaN and leaves its tile's others as they are."""
    pa.pa_clear_device_error()
    c = Case(98, [700, 130], [m, m], 2, 1, 64)
    clean = _call(c)
    c.q[3], c.q[m + 1, 1] = bad, bad
    got = _call(c)
    rows = torch.ones(2 * m, 2, dtype=torch.bool, device="cuda")
    rows[3], rows[m + 1, 1] = False, False
    assert torch.equal(got[rows].view(torch.int16), clean[rows].view(torch.int16))
    assert bool(got[~rows].isnan().all()) and pa.pa_get_device_error() == 0


def test_queries_past_the_bound_are_left():
    pa.pa_clear_device_error()
    c = Case(96, [70, 90], [40, 4], 4, 1, 128)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, 7.0)
    ws = pa.CrossWorkspace(33, 4, 1, 128)
    pa.pa_cross_attention(out, q, k, v, tables, sources, start, 33, c.scale, ws)
    assert bool((out[33:40] == 7.0).all())
    out[33:40] = _call(c)[33:40]
    c.check(out)


def test_bad_lengths_skip_their_sequence():
    c = Case(97, [70, 90, 33], [4, 5, 6], 4, 2, 64)
    q, k, v, tables, sources, start = c.on_gpu()
    ws = pa.CrossWorkspace(6, 4, 2, 64)
    for bad_s, bad_at in ((-1, None), (tables.shape[1] * 16 + 1, None), (None, 16), (None, 3)):
        s, at = sources.clone(), start.clone()
        if bad_s is not None:
            s[1] = bad_s
        else:
            at[2] = bad_at                       # rows past T, or before their start
        pa.pa_clear_device_error()
        out = torch.full_like(q, 7.0)
        pa.pa_cross_attention(out, q, k, v, tables, s, at, 6, c.scale, ws)
        assert pa.pa_get_device_error() == pa.PA_DEVERR_CONTEXT_LEN
        rest = _call(c)
        if bad_at == 3:                          # sequence 2 now begins at row 3
            rest[:3] = out[:3]
        else:
            assert bool((out[4:9] == 7.0).all())
            rest[:4] = out[:4]
        if bad_s is not None:
            rest[9:] = out[9:]
        c.check(rest)
        pa.pa_clear_device_error()


def test_bad_block_is_reported():
    c = Case(98, [70, 40], [4, 5], 4, 2, 64)
    q, k, v, tables, sources, start = c.on_gpu()
    good = _call(c)
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        pa.pa_clear_device_error()
        t = tables.clone()
        t[0, 2] = bad
        out = torch.zeros_like(q)
        pa.pa_cross_attention(out, q, k, v, t, sources, start, 5, c.scale,
                              pa.CrossWorkspace(5, 4, 2, 64))
        assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
        out[:4] = good[:4]
        c.check(out)
    pa.pa_clear_device_error()


@pytest.mark.parametrize("d", [64, 128])
def test_handle_captured_and_replayed(d):
    """Two handles replayed on two streams at once, their lengths changed between."""
    pa.pa_clear_device_error()
    cases = [Case(99 + i, [900, 17, 300], [4, 4, 4], 8, 2, d) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    made = []
    for c, s in zip(cases, streams):
        q, k, v, tables, sources, start = c.on_gpu()
        out = torch.full_like(q, float("nan"))
        call = pa.CrossAttention(out, q, k, v, tables, sources, start, 4, c.scale)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
            call()
        made.append((c, out, sources, g, call))
    torch.cuda.synchronize()
    for lens in ([900, 17, 300], [1, 0, 299], [64, 16, 128]):
        for (c, out, sources, g, _), s in zip(made, streams):
            c.sources = np.array(lens, np.int32)
            sources.copy_(_dev(lens))
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for (c, out, sources, g, _), s in zip(made, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for c, out, *_ in made:
            fresh = Case.__new__(Case)
            fresh.__dict__ = dict(c.__dict__)
            fresh.k, fresh.v = c.k.copy(), c.v.copy()
            c.check(out, str(lens))
    assert pa.pa_get_device_error() == 0


def test_first_call_on_another_stream():
    """The handle's counters and workspace are ready for whatever stream calls first."""
    pa.pa_clear_device_error()
    c = Case(120, [3000], [4], 4, 1, 64)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, float("nan"))
    other = torch.cuda.Stream()
    work = torch.zeros(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(work, work)
    call = pa.CrossAttention(out, q, k, v, tables, sources, start, 4, c.scale, stream=other)
    call()
    call()
    torch.cuda.synchronize()
    c.check(out)
    assert not call.workspace.counters.any() and pa.pa_get_device_error() == 0


def test_refusals():
    c = Case(121, [70], [4], 4, 2, 64)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.zeros_like(q)
    ws = pa.CrossWorkspace(4, 4, 2, 64)
    small = pa.CrossWorkspace(3, 4, 2, 64)

    def call(out=out, q=q, k=k, v=v, tables=tables, sources=sources, start=start, n=4, ws=ws):
        pa.pa_cross_attention(out, q, k, v, tables, sources, start, n, c.scale, ws)

    for kw in (dict(out=out[:2]), dict(v=v[:1]), dict(sources=sources[:0]), dict(start=start[:1]),
               dict(ws=small), dict(tables=tables[0]), dict(q=q[:, :3], out=out[:, :3]),
               dict(q=q.cpu()), dict(tables=tables.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=q.float()), dict(k=k.float()), dict(sources=sources.long())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(pa.PAError):
        pa.CrossAttention(out, q, k, v, tables, sources, start, 4, 0.0)
    with pytest.raises(pa.PAError):
        call(out=q)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements, read at its end."""
    pa.pa_clear_device_error()
    nb, hkv, d = (1 << 31) // (8 * 16 * 128) + 5, 8, 128
    k = torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case(122, [30], [3], 8, 8, d)
    small_k, small_v = dev_bf16(c.k), dev_bf16(c.v)
    n = small_k.shape[0]
    k[nb - n:], v[nb - n:] = small_k, small_v
    q = dev_bf16(c.q)
    out = torch.zeros_like(q)
    pa.pa_cross_attention(out, q, k, v, _dev(c.tables + nb - n), _dev(c.sources), _dev(c.start), 3,
                          c.scale, pa.CrossWorkspace(3, 8, 8, d))
    c.check(out)
    assert pa.pa_get_device_error() == 0
