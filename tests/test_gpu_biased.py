"""Attention with changed scores on the GPU (pa_decode_step_biased,
pa_prefill_biased) against the float64 oracle: caps, distance biases, windows
and bidirectional prefixes, alone and together, with stale tables and NaN in
hidden places; and the operators run together as a serving step uses them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import biased as OB
from oracle import int4 as O4
from oracle import rope as OR
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _slopes(hq):
    return (2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)).astype(np.float32)


def _case(seed, chunks, hq, hkv, d=128, window=0, hide=True, gain=1.0):
    """chunks: (earlier tokens, new tokens).  hide: blocks before every window
    are stale table entries, and hidden places of the blocks at both ends NaN."""
    rng = np.random.default_rng(seed)
    ctx = np.array([p + n for p, n in chunks], dtype=np.int32)
    n = np.array([n for _, n in chunks], dtype=np.int32)
    nblk = -(-ctx // 16)
    nb = int(nblk.sum()) + 3
    perm = rng.permutation(nb)
    tables = np.full((len(chunks), max(1, int(nblk.max()))), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(nblk.tolist()):
        tables[b, :k] = perm[at:at + k]
        at += k
    kc, vc = normal_bf16(rng, (nb, hkv, 16, d)), normal_bf16(rng, (nb, hkv, 16, d))
    q = normal_bf16(rng, (int(n.sum()), hq, d))
    if gain != 1.0:                     # larger scores, exactly (a power of two)
        q = OR.to_bf16_bits((bf16_bits_to_f64(q) * gain).astype(np.float32))
    if hide:
        for b, c in enumerate(ctx.tolist()):
            if c % 16:
                for pool in (kc, vc):
                    pool[tables[b, c // 16], :, c % 16:] = 0x7FC0
            first = max(0, c - int(n[b]) + 1 - window) if window else 0
            if first // 16 < nblk[b]:
                for pool in (kc, vc):
                    pool[tables[b, first // 16], :, :first % 16] = 0x7FC0
            tables[b, :first // 16] = 10 ** 8
    return ctx, n, tables, kc, vc, q


RULES = [dict(softcap=50.0), dict(softcap=1.5), dict(slopes=True), dict(window=1),
         dict(window=37), dict(window=160), dict(window=100000),
         dict(softcap=20.0, slopes=True, window=100)]


def _split(rule, hq):
    r = dict(rule)
    r["slopes"] = _slopes(hq) if r.get("slopes") else None
    return r


# ----------------------------------------------------------------- decode step

@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 4, 2), (128, 8, 1)])
def test_biased_step(rule, d, hq, hkv):
    r = _split(rule, hq)
    window = r.get("window", 0)
    case = _case(hq + d, [(c - 1, 1) for c in (1, 15, 16, 17, 100, 161, 700, 1111)], hq, hkv, d,
                 window)
    ctx, n, tables, kc, vc, q = case
    ref = OB.batch(q, kc, vc, tables, ctx, n, d ** -0.5, **r)
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    t, c = _dev(tables, np.int32), _dev(ctx, np.int32)
    kw = dict(softcap=r.get("softcap", 0.0), alibi_slopes=_dev(r["slopes"], np.float32),
              window=window)
    out = torch.full_like(dq, float("nan"))
    B = len(ctx)
    pa.pa_clear_device_error()
    pa.pa_decode_step(out, dq, dk, dv, t, c, d ** -0.5, partition_size=0, **kw)
    assert_close(bf16_to_f64(out), ref, f"whole {rule}")
    cover = min(1111, window + 15) if window else 1111
    for part in (16, 48, 512):
        counters = pa.step_counters(B, hkv)
        ws = pa.splitk_workspace(B, hq, d, cover, part)
        for w in ws:
            w.fill_(float("nan"))
        out.fill_(float("nan"))
        pa.pa_decode_step(out, dq, dk, dv, t, c, d ** -0.5, partition_size=part, workspace=ws,
                          counters=counters, **kw)
        assert_close(bf16_to_f64(out), ref, f"split {part} {rule}")
        assert not counters.any()
    for part in (None, 256):          # chosen, and given
        out.fill_(float("nan"))
        step = pa.DecodeStep(None, None, dk, dv, None, dq, t, c, out, d ** -0.5,
                             partition_size=part, host_context_lens=ctx, **kw)
        step()
        step()
        assert_close(bf16_to_f64(out), ref, f"handle {part} {rule}")
        assert not step.counters.any()
    assert pa.pa_get_device_error() == 0


def test_biased_step_large_scores():
    # scores far past the cap: the tanh's flat ends, and its steep middle
    for cap, gain in ((5.0, 64.0), (1000.0, 64.0), (0.01, 1.0)):
        ctx, n, tables, kc, vc, q = _case(3, [(299, 1), (50, 1)], 8, 2, gain=gain)
        ref = OB.batch(q, kc, vc, tables, ctx, n, 0.1, softcap=cap)
        out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_step(out, dev_bf16(q), dev_bf16(kc), dev_bf16(vc), _dev(tables, np.int32),
                          _dev(ctx, np.int32), 0.1, partition_size=0, softcap=cap)
        assert_close(bf16_to_f64(out), ref, f"cap {cap} gain {gain}")


@pytest.mark.parametrize("window", [0, 1, 40])
@pytest.mark.parametrize("part", [0, 32])
def test_biased_step_writes(window, part):
    ctx, n, tables, kc, vc, q = _case(4, [(c - 1, 1) for c in (1, 16, 17, 300)], 8, 2, 128,
                                      window)
    rng = np.random.default_rng(5)
    key, val = normal_bf16(rng, (4, 2, 128)), normal_bf16(rng, (4, 2, 128))
    slots = np.array([tables[b, (c - 1) // 16] * 16 + (c - 1) % 16 for b, c in enumerate(ctx)])
    dk, dv = dev_bf16(kc), dev_bf16(vc)
    for b, s in enumerate(slots):
        kc[s // 16, :, s % 16], vc[s // 16, :, s % 16] = key[b], val[b]
    ref = OB.batch(q, kc, vc, tables, ctx, n, 0.1, window=window, softcap=30.0)
    out = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    kw = {}
    if part:
        kw = dict(workspace=pa.splitk_workspace(4, 8, 128, 300, part),
                  counters=pa.step_counters(4, 2))
    pa.pa_clear_device_error()
    pa.pa_decode_step(out, dev_bf16(q), dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), 0.1,
                      dev_bf16(key), dev_bf16(val), _dev(slots, np.int64), part, softcap=30.0,
                      window=window, **kw)
    assert pa.pa_get_device_error() == 0
    assert_close(bf16_to_f64(out), ref, "step with write")
    assert torch.equal(dk.view(torch.int16), dev_bf16(kc).view(torch.int16))
    assert torch.equal(dv.view(torch.int16), dev_bf16(vc).view(torch.int16))


def test_biased_step_empty_and_bad_lengths():
    ctx, n, tables, kc, vc, q = _case(6, [(99, 1), (20, 1)], 8, 2, hide=False)
    out = torch.full((2, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.pa_clear_device_error()
    for part in (0, 32):
        kw = {} if not part else dict(workspace=pa.splitk_workspace(2, 8, 128, 112, part),
                                      counters=pa.step_counters(2, 2))
        pa.pa_decode_step(out, dev_bf16(q), dev_bf16(kc), dev_bf16(vc), _dev(tables, np.int32),
                          _dev([100, 0], np.int32), 0.1, partition_size=part, window=10, **kw)
        assert pa.pa_get_device_error() == 0
        assert not out[1].any() and torch.isfinite(out).all()
        pa.pa_decode_step(out, dev_bf16(q), dev_bf16(kc), dev_bf16(vc), _dev(tables, np.int32),
                          _dev([1 << 30, -7], np.int32), 0.1, partition_size=part, window=10,
                          **kw)
        assert pa.pa_get_device_error() & pa.PA_DEVERR_CONTEXT_LEN
        pa.pa_clear_device_error()


# --------------------------------------------------------------------- prefill

MIXED = [(0, 5), (0, 37), (100, 1), (13, 40), (300, 200), (0, 128), (1000, 33), (7, 129)]


def _prefill(case, scale, prefix=None, **rule):
    ctx, n, tables, kc, vc, q = case
    dq = dev_bf16(q)
    out = torch.full_like(dq, float("nan"))
    starts = np.concatenate([[0], np.cumsum(n)])
    pa.pa_clear_device_error()
    pa.pa_prefill_biased(out, dq, dev_bf16(kc), dev_bf16(vc), _dev(tables, np.int32),
                         _dev(ctx, np.int32), _dev(starts, np.int32), int(n.max()), scale,
                         rule.get("softcap", 0.0), _dev(rule.get("slopes"), np.float32),
                         rule.get("window", 0), _dev(prefix, np.int32))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    return bf16_to_f64(out), OB.batch(q, kc, vc, tables, ctx, n, scale, prefix_lens=prefix, **rule)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 16), (64, 8)])
def test_biased_prefill(rule, hq, hkv):
    r = _split(rule, hq)
    case = _case(hq * 7 + hkv, MIXED, hq, hkv, window=r.get("window", 0))
    got, ref = _prefill(case, 128 ** -0.5, **r)
    assert_close(got, ref, f"{rule}")


@pytest.mark.parametrize("rule", [dict(), dict(slopes=True), dict(window=50),
                                  dict(softcap=10.0, slopes=True, window=150)])
def test_biased_prefill_prefix(rule):
    r = _split(rule, 16)
    case = _case(8, MIXED, 16, 8, window=r.get("window", 0), hide=not r.get("window"))
    prefix = [5, 20, 0, 53, 400, 64, 1033, 1]
    got, ref = _prefill(case, 0.088, prefix, **r)
    assert_close(got, ref, f"prefix {rule}")


@pytest.mark.parametrize("window", [1200, 2 ** 31 - 1])
def test_biased_windows_past_every_context(window):
    # nothing is hidden: also where a prefix reaches far past the first queries
    slopes = _slopes(16)
    case = _case(14, [(0, 1100), (30, 200)], 16, 8)
    got, ref = _prefill(case, 0.088, [1100, 230], slopes=slopes, window=window)
    assert_close(got, ref, f"prefill window {window}")
    ctx, n, tables, kc, vc, q = case
    last = q[[1099, 1299]]
    out = torch.empty(2, 16, 128, dtype=torch.bfloat16, device="cuda")
    step = pa.DecodeStep(None, None, dev_bf16(kc), dev_bf16(vc), None, dev_bf16(last),
                         _dev(tables, np.int32), _dev(ctx, np.int32), out, 0.088,
                         partition_size=64, alibi_slopes=_dev(slopes, np.float32), window=window)
    step()
    full = OB.batch(last, kc, vc, tables, ctx, np.array([1, 1]), 0.088, slopes=slopes)
    assert_close(bf16_to_f64(out), full, f"step window {window}")


def test_biased_prefill_large_scores():
    # (and scores of up to a sixth and half of their cap)
    for cap, gain in ((5.0, 64.0), (1000.0, 64.0), (0.01, 1.0), (2.0, 4.0), (30.0, 1.0),
                      (10.0, 1.0)):
        case = _case(9, [(40, 30), (0, 150)], 8, 2, gain=gain)
        got, ref = _prefill(case, 0.1, softcap=cap)
        assert_close(got, ref, f"cap {cap} gain {gain}")


def test_biased_prefill_without_a_rule_is_prefill():
    ctx, n, tables, kc, vc, q = _case(10, MIXED, 32, 8)
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    starts = _dev(np.concatenate([[0], np.cumsum(n)]), np.int32)
    outs = []
    for fn in (pa.pa_prefill, pa.pa_prefill_biased):
        out = torch.empty_like(dq)
        fn(out, dq, dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), starts, int(n.max()), 0.1)
        outs.append(out)
    # the same products, their chunks added in the other order: the weights keep
    # 16 bits in both (2^-16 of at most |v| < 6), then each result is rounded to
    # bf16 by half a step (2^-8), so the two are at most a step apart
    a, b = (bf16_to_f64(x) for x in outs)
    assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(a) + 6 * 2.0 ** -15)


def test_biased_prefill_leaves_other_rows_and_bad_prefixes():
    ctx, n, tables, kc, vc, q = _case(11, [(10, 20), (0, 30), (5, 6)], 8, 2)
    dq = dev_bf16(q)
    out = torch.full((q.shape[0] + 9, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    pad = torch.zeros_like(out)
    pad[:q.shape[0]] = dq
    pa.pa_clear_device_error()
    pa.pa_prefill_biased(out, pad, dev_bf16(kc), dev_bf16(vc), _dev(tables, np.int32),
                         _dev(ctx, np.int32), _dev([0, 20, 50, 56], np.int32), 64, 0.1,
                         prefix_lens=_dev([4, 31, -1], np.int32))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_PREFIX
    pa.pa_clear_device_error()
    assert (out[20:] == 3.0).all()                # skipped sequences and rows behind the last
    ref = OB.sequence(q[:20], kc, vc, tables[0], 30, 0.1, prefix=4)
    assert_close(bf16_to_f64(out[:20]), ref, "the good sequence")


def test_biased_prefill_handle_under_a_graph():
    ctx, n, tables, kc, vc, q = _case(12, [(100, 60), (0, 90)], 8, 2, hide=False)
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    out = torch.empty_like(dq)
    t, c = _dev(tables, np.int32), _dev(ctx, np.int32)
    starts = _dev([0, 60, 150], np.int32)
    slopes = _dev(_slopes(8), np.float32)
    for kw in (dict(softcap=30.0, alibi_slopes=slopes, window=70), dict()):
        step = pa.PrefillStep(out, dq, dk, dv, t, c, starts, 90, 0.1, **kw)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            step()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=s):
                step()
        want = out.clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        rule = dict(softcap=30.0, slopes=_slopes(8), window=70) if kw else {}
        assert_close(bf16_to_f64(out), OB.batch(q, kc, vc, tables, ctx, n, 0.1, **rule), "graph")


def test_biased_binding_refusals():
    ctx, n, tables, kc, vc, q = _case(13, [(9, 1)], 8, 2)
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    t, c, st = _dev(tables, np.int32), _dev(ctx, np.int32), _dev([0, 1], np.int32)
    out = torch.empty_like(dq)
    with pytest.raises(ValueError):
        pa.pa_decode_step(out, dq, dk, dv, t, c, 0.1, partition_size=0,
                          alibi_slopes=torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        pa.pa_decode_step(out, dq, dk, dv, t, c, 0.1, partition_size=0,
                          alibi_slopes=torch.ones(8, device="cuda", dtype=torch.float64))
    with pytest.raises(pa.PAError):
        pa.pa_decode_step(out, dq, dk, dv, t, c, 0.1, partition_size=0, window=-2)
    with pytest.raises(ValueError):
        pa.pa_prefill_biased(out, dq, dk, dv, t, c, st, 1, 0.1, prefix_lens=_dev([1, 2], np.int32))
    with pytest.raises(ValueError):
        pa.pa_prefill_biased(out, dq, dk, dv, t, c, st, 1, 0.1,
                             alibi_slopes=torch.ones(8))
    with pytest.raises(pa.PAError):
        pa.pa_prefill_biased(out, dq, dk, dv, t, c, st, 1, 0.1, softcap=float("nan"))


# ------------------------------------------------------- the operators together

def test_prompt_then_decode_steps():
    """A serving step's sequence: rotate and append a prompt, prefill it with
    capped scores, then rotate, append and decode token by token; the same
    tokens kept in a 4-bit cache decode beside it."""
    rng = np.random.default_rng(14)
    hq, hkv, d, n0, steps, cap, window = 8, 2, 128, 45, 4, 30.0, 40
    table = pa.rope_table(256, d, 10000.0)
    alloc = pa.BlockAllocator(8, 16)
    alloc.add_seq(0)
    alloc.reserve(0, n0)
    kc, vc = (torch.zeros(8, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    k4, v4 = pa.int4_pool(8, hkv, d), pa.int4_pool(8, hkv, d)
    hist_k, hist_v = [], []

    def append(qkv, pos, slots):
        x = dev_bf16(qkv)
        T = x.shape[0]
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        out = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        args = (_dev(slots, np.int64), _dev(pos, np.int32), table)
        pa.pa_rope_reshape_and_cache(out, q, k, v, kc, vc, *args)
        pa.pa_rope_reshape_and_cache(None, None, k, v, k4, v4, *args)
        cos, sin = (t.cpu().numpy()[pos] for t in table.split(d // 2, 1))
        rot = OR.rotate_fp32(qkv[:, :hq + hkv], cos, sin, d, False)
        hist_k.append(rot[:, hq:])
        hist_v.append(qkv[:, hq + hkv:])
        return out, rot[:, :hq]

    tab = alloc.block_table(0)
    pos = np.arange(n0)
    q, qbits = append(normal_bf16(rng, (n0, hq + 2 * hkv, d)), pos, tab[pos // 16] * 16 + pos % 16)

    def history():
        n = sum(len(x) for x in hist_k)
        pad = -n % 16
        pools = [np.concatenate(x + [np.zeros((pad, hkv, d), np.uint16)]).reshape(
            -1, 16, hkv, d).transpose(0, 2, 1, 3) for x in (hist_k, hist_v)]
        return pools, np.arange(pools[0].shape[0])

    out = torch.empty_like(q)
    pa.pa_prefill_biased(out, q, kc, vc, _dev(tab[None], np.int32), _dev([n0], np.int32),
                         _dev([0, n0], np.int32), n0, 0.088, softcap=cap, window=window)
    (K, V), ids = history()
    assert_close(bf16_to_f64(out), OB.sequence(qbits, K, V, ids, n0, 0.088, softcap=cap,
                                               window=window), "prompt")
    for i in range(steps):
        slot, _, _ = alloc.append_slot(0)
        tab = alloc.block_table(0)
        p = n0 + i
        q, qbits = append(normal_bf16(rng, (1, hq + 2 * hkv, d)), np.array([p]), np.array([slot]))
        t, c = _dev(tab[None], np.int32), _dev([p + 1], np.int32)
        out = torch.empty_like(q)
        pa.pa_decode_step(out, q, kc, vc, t, c, 0.088, partition_size=32,
                          workspace=pa.splitk_workspace(1, hq, d, p + 1, 32),
                          counters=pa.step_counters(1, hkv), softcap=cap, window=window)
        (K, V), ids = history()
        assert_close(bf16_to_f64(out), OB.sequence(qbits, K, V, ids, p + 1, 0.088, softcap=cap,
                                                   window=window), f"step {i}")
        pa.pa_decode_int4(out, q, k4, v4, t, c, 0.088)
        ref = O4.decode(bf16_bits_to_f64(qbits), O4.values(*O4.quantize(K)),
                        O4.values(*O4.quantize(V)), ids[None], [p + 1], 0.088)
        # as the 4-bit decode's own gate: bf16 and f16 rounding
        assert np.all(np.abs(bf16_to_f64(out) - ref) <=
                      2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * 10 + 2.0 ** -13 * 5)
    assert pa.pa_get_device_error() == 0


def test_two_layers_at_once_on_two_streams():
    """Two chains of append, 4-bit step and capped step, each with buffers of its
    own and captured into a graph, run at once on two streams: the results of
    each are those of running it alone."""
    hq, hkv, d, B, n = 8, 2, 128, 12, 700
    table = pa.rope_table(1024, d, 10000.0)
    ctx = [n - 31 * b for b in range(B)]
    chains = []
    for seed in (21, 22):
        rng = np.random.default_rng(seed)
        nb = 44 * B
        tables = _dev(rng.permutation(nb).reshape(B, 44), np.int32)
        c = _dev(ctx, np.int32)
        pos = c - 1
        slots = (tables.gather(1, (pos // 16).long()[:, None])[:, 0] * 16 + pos % 16).long()
        kc, vc = (dev_bf16(normal_bf16(rng, (nb, hkv, 16, d))) for _ in "kv")
        pools = []
        for src in (kc, vc):
            pools.append(src.clone())
        k4, v4 = pa.int4_pool(nb, hkv, d), pa.int4_pool(nb, hkv, d)
        every = torch.arange(nb * 16, device="cuda")
        rows = [p.permute(0, 2, 1, 3).reshape(nb * 16, hkv, d).contiguous() for p in pools]
        pa.pa_reshape_and_cache_int4(*rows, k4, v4, every)
        qkv = dev_bf16(normal_bf16(rng, (B, hq + 2 * hkv, d)))
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        q_out = torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
        outs = [torch.empty_like(q_out) for _ in range(2)]
        calls = [pa.RopeAppend(q_out, q, k, v, kc, vc, slots, pos, table),
                 pa.RopeAppend(q_out, q, k, v, k4, v4, slots, pos, table),
                 pa.DecodeStep(None, None, k4, v4, None, q_out, tables, c, outs[0], 0.088,
                               partition_size=64),
                 pa.DecodeStep(None, None, kc, vc, None, q_out, tables, c, outs[1], 0.088,
                               partition_size=128, softcap=20.0, window=300)]
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        for call in calls:
            call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            for call in calls:
                call()
        chains.append((calls, stream, graph, outs, want))
    for replay in (False, True):
        for _, _, _, outs, _ in chains:
            for o in outs:
                o.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(20):
            for calls, stream, graph, _, _ in chains:
                with torch.cuda.stream(stream):
                    if replay:
                        graph.replay()
                    else:
                        for call in calls:
                            call()
        torch.cuda.synchronize()
        for _, _, _, outs, want in chains:
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {replay}"
    assert pa.pa_get_device_error() == 0
