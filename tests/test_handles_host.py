"""What the handles of the search operators keep, on the CPU: a stand-in for the prepared
call takes the addresses and launches nothing."""
import gc
import weakref
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa


@pytest.fixture
def prepared(monkeypatch):
    """The calls that handles made."""
    calls = []

    class Call:
        def __init__(self, name, *args):
            calls.append((name, args))

        def run(self, stream):
            return pa.PA_OK

    monkeypatch.setattr(pa, "_Prepared", Call)
    return calls


def _states():
    return [torch.zeros(8, 5) for _ in range(3)]


@pytest.mark.parametrize("how", ["iterator", "cleared list", "list", "one"])
def test_reordering_keeps_its_states(monkeypatch, prepared, how):
    """The call holds their addresses: they live as long as the handle, whatever becomes of
    what the caller handed over."""
    monkeypatch.setattr(pa, "_reorder_args", lambda states, parents, beams: tuple(
        t.data_ptr() for t in ([states] if isinstance(states, torch.Tensor) else list(states))))
    tensors = _states()[:1] if how == "one" else _states()
    refs = [weakref.ref(t) for t in tensors]
    given = {"iterator": iter, "one": lambda t: t[0]}.get(how, list)(tensors)
    call = pa.ReorderStates(given, torch.zeros(8, dtype=torch.int32), 4)
    if how == "cleared list":
        given.clear()
    del tensors, given
    gc.collect()
    assert all(r() is not None for r in refs)
    assert prepared[0][1] == tuple(r().data_ptr() for r in refs)
    del call
    gc.collect()
    assert all(r() is None for r in refs)


def test_own_buffers_are_held_for_the_streams_that_used_them(monkeypatch, prepared):
    """A workspace that a handle made goes back to its allocator with the handle: every
    stream that it ran on is told of first, once."""
    told = []

    class Made:
        device = "cuda:0"

        def record_stream(self, stream):
            told.append(stream)

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device: (at, device))
    one, other = (SimpleNamespace(cuda_stream=at) for at in (77, 78))
    call = pa._FixedCall()
    call._fix("a call", "pa_prepare_beam_select", (), one, [], [Made()])
    assert told == []
    call()
    call()
    call(stream=one)
    assert told == [(77, "cuda:0")]
    call(stream=other)
    call(stream=other)
    call(stream=SimpleNamespace(cuda_stream=0))
    assert told == [(77, "cuda:0"), (78, "cuda:0"), (0, "cuda:0")]
    # the caller's workspace is the caller's
    call = pa._FixedCall()
    call._fix("a call", "pa_prepare_beam_select", (), one, [object()])
    call()
    assert len(told) == 3


@pytest.mark.parametrize("fused", [True, False])
def test_a_decode_step_holds_its_own_buffers_too(monkeypatch, fused):
    told = []

    class Made:
        device, shape = "cuda:0", (2, 4, 1, 64)

        def record_stream(self, stream):
            told.append((self, stream))

    made = [Made() for _ in range(4)]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device: at)
    monkeypatch.setattr(pa, "splitk_workspace", lambda *a: tuple(made[:3]))
    monkeypatch.setattr(pa, "step_counters", lambda *a: made[3])
    monkeypatch.setattr(pa, "_step_args", lambda *a: (lambda *b: pa.PA_OK, ()))
    monkeypatch.setattr(pa, "_dev", lambda *a: None)
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 16, 64).bfloat16()
    new = torch.zeros(2, 2, 64).bfloat16()
    ints = torch.zeros(2, 1, dtype=torch.int32)

    def step(**kw):
        return pa.DecodeStep(new, new, kv, kv, ints[:, 0].long(), q, ints, ints[:, 0], q, 0.1,
                             stream=SimpleNamespace(cuda_stream=77), fused=fused, **kw)

    # (a step of separate launches calls these)
    monkeypatch.setattr(pa, "_lib", SimpleNamespace(**{
        f: lambda *a: pa.PA_OK for f in ("pa_reshape_and_cache", "pa_decode_splitk", "pa_decode",
                                         "pa_splitk_reduce")}))
    call = step()
    call()
    call()
    call(stream=SimpleNamespace(cuda_stream=78))
    of = made if fused else made[:3]
    assert told == [(t, at) for at in (77, 78) for t in of]
    # the caller's are the caller's
    step(workspace=tuple(made[:3]), counters=made[3])()
    assert len(told) == 2 * len(of)
