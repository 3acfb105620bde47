"""DecodeStep and the streams around it: a handle is made without stopping the host,
whatever the GPU is doing, and its first call, on any stream or captured, finds its
counters and workspace ready; and what a step with early reads takes from the launch
just before it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as OA
from oracle import biased as OB
from paged_kv_cache_283_gb300 import inputs as I
from paged_kv_cache_283_gb300 import pa

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16, product_tables
from test_gpu_biased import _case, _dev

pytestmark = pytest.mark.gpu


def _busy(work, out):
    """About 40 ms of work on the current stream, which begins by writing `out`."""
    for o in out:
        o.fill_(-1)
    for _ in range(60):
        torch.mm(work, work, out=work[:])


@pytest.mark.parametrize("how", ["call", "captured", "captured where it was made"])
@pytest.mark.parametrize("rule", [{}, dict(window=200)])
def test_handle_is_made_without_waiting(how, rule):
    w = I.random_case(51, 3, [300, 17, 900], 8, 2, 128)
    tables, _ = product_tables(w)
    window = rule.get("window", 0)
    dk, dv, dq = dev_bf16(w.k_cache), dev_bf16(w.v_cache), dev_bf16(w.q)
    t, c = _dev(tables, np.int32), _dev(w.context_lens, np.int32)
    ref = OB.batch(w.q, w.k_cache, w.v_cache, tables, w.context_lens, np.ones(3, int), w.scale,
                   window=window) if window else \
        OA.decode(w.q, w.k_cache, w.v_cache, tables, w.context_lens, w.scale, 16)
    work = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    other = torch.cuda.Stream()
    out = torch.empty_like(dq)
    made = pa.DecodeStep(None, None, dk, dv, None, dq, t, c, out, w.scale, partition_size=64,
                         stream=other, **rule)
    made()
    torch.cuda.synchronize()
    del made                        # (its memory is there for the next handle)
    for _ in range(3):
        dirty = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (6, 6, 6)]
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        own = other if how == "captured where it was made" else torch.cuda.current_stream()
        with torch.cuda.stream(own):
            _busy(work, dirty)
            del dirty               # (the handle's counters may take their place)
            step = pa.DecodeStep(None, None, dk, dv, None, dq, t, c, out, w.scale,
                                 partition_size=64, stream=other, **rule)
            assert not own.query(), "the constructor waited for the GPU"
        if how == "call":
            step()
            step()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(other):
                graph.capture_begin()
                step()
                graph.capture_end()
            graph.replay()          # on the current stream
            graph.replay()
            torch.cuda.current_stream().synchronize()
        other.synchronize()
        assert_close(bf16_to_f64(out), ref, how)
        assert not step.counters.any()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("part", [0, 128])
def test_early_reads_take_slopes_after_the_launch_before(part):
    """A changed step with early reads whose distance slopes are what the launch just
    before it writes: early reads may take tables, lengths and pools before that
    launch is complete, and nothing else."""
    hq, hkv, d = 8, 2, 128
    w = I.random_case(52, 1, [60000], hq, hkv, d)
    tables, _ = product_tables(w)
    ws = pa.splitk_workspace(1, hq, d, 60000, 65536)        # one long partition
    first = (dev_bf16(w.q), dev_bf16(w.k_cache), dev_bf16(w.v_cache), _dev(tables, np.int32),
             _dev(w.context_lens, np.int32), w.scale, 65536)
    slopes = ws[1].view(hq)                                 # its rows' largest scores
    case = _case(53, [(c - 1, 1) for c in (300, 17, 700)], hq, hkv, d)
    ctx, n, t, kc, vc, q = case
    dq, dk, dv = dev_bf16(q), dev_bf16(kc), dev_bf16(vc)
    dt, dc = _dev(t, np.int32), _dev(ctx, np.int32)
    kw = {}
    if part:
        kw = dict(workspace=pa.splitk_workspace(3, hq, d, 700, part),
                  counters=pa.step_counters(3, hkv))
    out = torch.empty_like(dq)
    pa.pa_clear_device_error()
    for _ in range(3):
        out.fill_(float("nan"))
        ws[1].fill_(float("nan"))
        torch.cuda.synchronize()
        pa.pa_decode_splitk(*ws, *first)
        pa.pa_decode_step(out, dq, dk, dv, dt, dc, 0.088, partition_size=part, early_read=True,
                          alibi_slopes=slopes, **kw)
        torch.cuda.synchronize()
        ref = OB.batch(q, kc, vc, t, ctx, n, 0.088, slopes=slopes.cpu().numpy())
        assert_close(bf16_to_f64(out), ref, f"partition {part}")
    assert pa.pa_get_device_error() == 0
