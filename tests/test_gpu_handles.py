"""Handles that are gone before their calls have run."""
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

from test_gpu_beam import Search
from test_gpu_cross import Case

pytestmark = pytest.mark.gpu


def _dirty(shapes):
    """New tensors of the same sizes, written on the current stream at once."""
    return [torch.full(s, 123, dtype=d, device="cuda") for s, d in shapes]


def _kept_busy(stream):
    """Some milliseconds of work in front of what follows on `stream`."""
    x = torch.zeros(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(6):
            x = x @ x
    return x


def test_cross_attention_on_another_stream():
    pa.pa_clear_device_error()
    c = Case(31, [9000, 33, 0, 5000], [4, 2, 1, 3], 8, 2, 128)
    q, k, v, tables, sources, start = c.on_gpu()
    out = torch.full_like(q, float("nan"))
    side = torch.cuda.Stream()
    for how in range(2):
        out.fill_(float("nan"))
        busy = _kept_busy(side)
        call = pa.CrossAttention(out, q, k, v, tables, sources, start, 4, c.scale,
                                 stream=side if how else None)
        w = call.workspace
        shapes = [(t.shape, t.dtype) for t in (w.ws_out, w.ws_ml, w.counters)]
        if how:
            call()
        else:
            call(stream=side)
        del call, w
        held = _dirty(shapes)
        torch.cuda.synchronize()
        c.check(out)
        assert all(bool((t == 123).all()) for t in held)
        del busy, held
    assert pa.pa_get_device_error() == 0


def test_selection_on_another_stream():
    pa.pa_clear_device_error()
    s = Search(32, 6, 4, 8, 50257, "bf16")
    s.eos = -1
    out = (torch.zeros((6, 8), device="cuda"),
           *(torch.zeros((6, 8), dtype=torch.int32, device="cuda") for _ in "pt"))
    side = torch.cuda.Stream()
    busy = _kept_busy(side)
    call = pa.BeamSelect(*out, s.logits, s.scores, 4)
    shapes = [(t.shape, t.dtype) for t in call.workspace]
    with torch.cuda.stream(side):
        call()
    del call
    held = _dirty(shapes)
    torch.cuda.synchronize()
    s.check([x.cpu().numpy() for x in out] + [None])
    assert all(bool((t == 123).all()) for t in held) and busy is not None
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("fused", [True, False])
def test_decode_step_on_another_stream(fused):
    pa.pa_clear_device_error()
    g = torch.Generator(device="cuda").manual_seed(33)
    b, hq, hkv, d, mb = 6, 8, 2, 128, 40
    kc, vc = (torch.randn((b * mb, hkv, 16, d), generator=g, device="cuda").bfloat16()
              for _ in "kv")
    tables = torch.randperm(b * mb, generator=g, device="cuda").to(torch.int32).view(b, mb)
    lens = torch.tensor([600, 1, 64, 333, 16, 510], dtype=torch.int32, device="cuda")
    q = torch.randn((b, hq, d), generator=g, device="cuda").bfloat16()
    key, value = (torch.randn((b, hkv, d), generator=g, device="cuda").bfloat16() for _ in "kv")
    at = (lens - 1).long()
    slots = tables[torch.arange(b, device="cuda"), at // 16].long() * 16 + at % 16
    outs = []
    for drop in (False, True):
        out = torch.full_like(q, float("nan"))
        k, v = kc.clone(), vc.clone()
        side = torch.cuda.Stream()
        busy = _kept_busy(side)
        step = pa.DecodeStep(key, value, k, v, slots, q, tables, lens, out, d ** -0.5,
                             partition_size=64, fused=fused)
        if not drop:
            torch.cuda.synchronize()
        step(stream=side)
        shapes = [(t.shape, t.dtype) for t in step.workspace]
        if fused:
            shapes.append((step.counters.shape, step.counters.dtype))
        if drop:
            del step
        held = _dirty(shapes)
        torch.cuda.synchronize()
        assert all(bool((t == 123).all()) for t in held) and busy is not None
        outs.append(out)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
    assert pa.pa_get_device_error() == 0
