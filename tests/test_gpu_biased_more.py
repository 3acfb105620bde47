"""Attention with changed scores where the first tests do not reach: hidden places
that must not change a bit of the output, rules that change nothing against the
plain kernels, windows in more partitions than one launch merges, and slopes that
the launch just before writes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import biased as OB
from paged_kv_cache_283_gb300 import pa

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16
from test_gpu_biased import MIXED, _case, _dev, _slopes

pytestmark = pytest.mark.gpu


def _fill(case, pools, scale, prefix=None, fn=pa.pa_prefill_biased, **rule):
    ctx, n, tables, _, _, q = case
    dq = dev_bf16(q)
    out = torch.full_like(dq, float("nan"))
    pa.pa_clear_device_error()
    fn(out, dq, *pools, _dev(tables, np.int32), _dev(ctx, np.int32),
       _dev(np.concatenate([[0], np.cumsum(n)]), np.int32), int(n.max()), scale,
       **({} if prefix is None else {"prefix_lens": _dev(prefix, np.int32)}), **rule)
    assert pa.pa_get_device_error() == 0
    return out


def _hidden(case, window):
    """(block, offset) of every place that no query of its sequence sees."""
    ctx, n, tables = case[:3]
    blk, off = [], []
    for b, c in enumerate(ctx.tolist()):
        first = max(0, c - int(n[b]) + 1 - window) if window else 0
        for j in [*range(first // 16 * 16, first), *range(c, -(-c // 16) * 16)]:
            blk.append(int(tables[b, j // 16]))
            off.append(j % 16)
    return blk, off


@pytest.mark.parametrize("cap", [50.0, 1e6])
@pytest.mark.parametrize("window,bias", [(0, False), (45, False), (45, True)])
def test_biased_prefill_takes_nothing_from_hidden_places(cap, window, bias):
    # values past every bound of the scores, in K and V, where no query looks
    case = _case(41, MIXED, 16, 4, window=window, hide=False)
    ctx, n, tables, kc, vc, q = case
    slopes = _slopes(16) if bias else None
    kw = dict(softcap=cap, window=window, alibi_slopes=_dev(slopes, np.float32))
    blk, off = _hidden(case, window)
    outs = []
    for fill in (0.0, 1e30, float("inf"), float("nan")):
        pools = [dev_bf16(kc), dev_bf16(vc)]
        for p in pools:
            p[blk, :, off] = fill
        outs.append(_fill(case, pools, 0.088, **kw))
    assert_close(bf16_to_f64(outs[0]), OB.batch(q, kc, vc, tables, ctx, n, 0.088, softcap=cap,
                                                window=window, slopes=slopes), "zeros hidden")
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_biased_prefill_without_a_rule_is_the_plain_kernel():
    case = _case(42, MIXED, 32, 8, hide=False)
    pools = [dev_bf16(case[3]), dev_bf16(case[4])]
    plain = _fill(case, pools, 0.1, fn=pa.pa_prefill)
    assert torch.equal(_fill(case, pools, 0.1), plain)
    assert torch.equal(_fill(case, pools, 0.1, window=1 << 20), plain)


@pytest.mark.parametrize("rule", [dict(prefix=True), dict(slopes=True), dict(softcap=1e4),
                                  dict(softcap=1e4, slopes=True, prefix=True)])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 16), (64, 8)])
def test_rules_that_change_nothing_give_the_plain_result(rule, hq, hkv):
    """Prefixes of no token, slopes of zero, a cap 1000 times the scores: the changed
    kernels beside the plain one.  Both keep 16 bits of a weight (2^-16 of values
    below 6); the cap's tanh moves a score s by s (s / cap)^2 / 3 < 10^-5 and by a
    relative 2^-22; then each result is rounded to bf16 by half a step (2^-8), so
    the two are at most a step apart."""
    case = _case(43, MIXED, hq, hkv, hide=False)
    pools = [dev_bf16(case[3]), dev_bf16(case[4])]
    kw = {"softcap": rule.get("softcap", 0.0)}
    if rule.get("slopes"):
        kw["alibi_slopes"] = torch.zeros(hq, device="cuda")
    got = bf16_to_f64(_fill(case, pools, 0.1, [0] * len(MIXED) if rule.get("prefix") else None,
                            **kw))
    want = bf16_to_f64(_fill(case, pools, 0.1, fn=pa.pa_prefill))
    assert np.all(np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 6 * (2.0 ** -15 + 1e-5))


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 8, 1)])
def test_biased_step_window_of_many_partitions(d, hq, hkv):
    # (more than sixteen partitions merge in a launch of their own)
    window = 700
    case = _case(44 + d, [(c - 1, 1) for c in (3000, 701, 700, 33, 1717)], hq, hkv, d, window)
    ctx, n, tables, kc, vc, q = case
    slopes = _slopes(hq)
    ref = OB.batch(q, kc, vc, tables, ctx, n, 0.09, softcap=20.0, slopes=slopes, window=window)
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    out = torch.empty_like(dq)
    for part in (16, 32):
        ws = pa.splitk_workspace(5, hq, d, window + 15, part)
        assert ws[1].shape[2] > 16
        for w in ws:
            w.fill_(float("nan"))
        counters = pa.step_counters(5, hkv)
        out.fill_(float("nan"))
        pa.pa_clear_device_error()
        pa.pa_decode_step(out, dq, dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), 0.09,
                          partition_size=part, workspace=ws, counters=counters, softcap=20.0,
                          alibi_slopes=_dev(slopes, np.float32), window=window)
        assert pa.pa_get_device_error() == 0
        assert_close(bf16_to_f64(out), ref, f"partitions of {part}")
        assert not counters.any()


@pytest.mark.parametrize("prefix", [False, True])
def test_slopes_of_either_sign(prefix):
    # far keys heavier than near ones: the reference maximum climbs chunk by chunk
    rng = np.random.default_rng(45)
    slopes = (0.05 * rng.standard_normal(16)).astype(np.float32)
    case = _case(46, MIXED, 16, 4)
    ctx, n, tables, kc, vc, q = case
    pre = [5, 20, 0, 53, 400, 64, 1033, 1] if prefix else None
    for cap in (0.0, 4.0):
        out = _fill(case, [dev_bf16(kc), dev_bf16(vc)], 0.088, pre, softcap=cap,
                    alibi_slopes=_dev(slopes, np.float32))
        assert_close(bf16_to_f64(out), OB.batch(q, kc, vc, tables, ctx, n, 0.088, softcap=cap,
                                                slopes=slopes, prefix_lens=pre), f"cap {cap}")
    ends = np.cumsum(n) - 1
    last = q[ends]
    step = pa.DecodeStep(None, None, dev_bf16(kc), dev_bf16(vc), None, dev_bf16(last),
                         _dev(tables, np.int32), _dev(ctx, np.int32),
                         torch.empty(len(n), 16, 128, dtype=torch.bfloat16, device="cuda"), 0.088,
                         partition_size=64, alibi_slopes=_dev(slopes, np.float32))
    step()
    assert_close(bf16_to_f64(step._keep[8]),
                 OB.batch(last, kc, vc, tables, ctx, np.ones_like(n), 0.088, slopes=slopes),
                 "step")


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("part", [0, 64])
def test_prepared_steps_of_the_plain_caches(kind, part):
    # pa_prepare_decode_step without a rule launches what the direct call launches
    torch.manual_seed(kind)
    B, hq, hkv, d, nb = 3, 8, 2, 128, 30
    ctx = torch.tensor([200, 1, 77], dtype=torch.int32, device="cuda")
    tables = torch.randperm(nb, device="cuda")[:39].to(torch.int32)
    tables = torch.cat([tables, tables[:9]]).view(3, 13)
    tables[1, 0], tables[2, :5] = 29, torch.arange(20, 25, device="cuda")
    tables[0] = torch.arange(13, device="cuda")
    dtype = (torch.bfloat16, torch.int8, torch.uint8)[kind]
    pools = [torch.randint(0, 100, (nb, hkv, 16, d), device="cuda").to(dtype) for _ in "kv"]
    scales = [torch.rand(nb, hkv, 16, device="cuda") * 1e-2 for _ in "kv"] if kind else []
    q, key, value = (torch.randn(B, h, d, device="cuda").to(torch.bfloat16)
                     for h in (hq, hkv, hkv))
    last = ctx - 1
    slots = tables.gather(1, (last // 16).long()[:, None])[:, 0].long() * 16 + last % 16
    ws = pa.splitk_workspace(B, hq, d, 208, part) if part else None
    counters = pa.step_counters(B, hkv) if part else None
    outs = []
    for prepared in (False, True):
        mine = [p.clone() for p in pools + scales]
        out = torch.empty_like(q)
        kw = dict(k_scales=mine[2], v_scales=mine[3]) if kind else {}
        call = (out, q, mine[0], mine[1], tables, ctx, 0.088, key, value, slots, part, ws,
                counters, kw.get("k_scales"), kw.get("v_scales"))
        fn, a = pa._step_args(*call)
        if prepared:
            at = 7 if not kind else 9           # the pools, and the scales of these kinds
            a = a[:7] + (a[7:9] if kind else (None, None)) + a[at:]
            a = a[:19] + (0.0, None, 0) + a[19:]
            h = pa._Prepared("pa_prepare_decode_step", kind, *a)
            h.run(torch.cuda.current_stream().cuda_stream)
        else:
            pa._check(fn(*a, torch.cuda.current_stream().cuda_stream), "step")
        torch.cuda.synchronize()
        outs.append([out, *mine])
    assert pa.pa_get_device_error() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("window", [1, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("as_lens", [list, lambda x: np.asarray(x, dtype=np.int32),
                                     lambda x: np.asarray(x, dtype=np.int64)])
def test_handles_plan_for_any_window(window, as_lens):
    case = _case(47, [(c - 1, 1) for c in (500, 17, 900)], 8, 2, 128, window)
    ctx, n, tables, kc, vc, q = case
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    step = pa.DecodeStep(None, None, dev_bf16(kc), dev_bf16(vc), None, dev_bf16(q),
                         _dev(tables, np.int32), _dev(ctx, np.int32), out, 0.088,
                         partition_size=None, host_context_lens=as_lens(ctx), window=window)
    step()
    assert_close(bf16_to_f64(out), OB.batch(q, kc, vc, tables, ctx, n, 0.088, window=window),
                 f"window {window}")


def test_handles_refuse_a_negative_window():
    ctx, n, tables, kc, vc, q = _case(48, [(9, 1)], 8, 2)
    for window in (-1, -100):
        for ps in (None, 64):
            with pytest.raises(ValueError, match="window"):
                pa.DecodeStep(None, None, dev_bf16(kc), dev_bf16(vc), None, dev_bf16(q),
                              _dev(tables, np.int32), _dev(ctx, np.int32), torch.empty_like(
                                  dev_bf16(q)), 0.1, partition_size=ps, host_context_lens=[10],
                              window=window)
