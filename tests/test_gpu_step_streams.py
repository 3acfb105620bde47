"""What a step with early reads takes from the launch just before it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import biased as OB
from paged_kv_cache_283_gb300 import inputs as I
from paged_kv_cache_283_gb300 import pa

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16, product_tables
from test_gpu_biased import _case, _dev

pytestmark = pytest.mark.gpu


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
