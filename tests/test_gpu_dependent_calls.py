"""Calls back to back, each reading what the one before it wrote: parents from a
selection, tables from a reordering, rows of a cache through those tables.  Each kernel
may start while the one before it runs; the results are those of calls that wait."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

pytestmark = pytest.mark.gpu


class Steps:
    """`steps` steps of 8 searches of 4 beams; their outputs are kept, step by step."""

    def __init__(self, d, steps):
        g = torch.Generator(device="cuda").manual_seed(d)
        n, beams, hq, hkv, mb = 8, 4, 4, 2, 6
        rows, nb = n * beams, n * beams * mb

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.scores0 = -rand(n, beams).abs()
        self.scores = self.scores0.clone()
        self.tables0 = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(rows, mb)
        self.tables = self.tables0.clone()
        self.lens0 = torch.randint(1, 16 * mb, (rows, 1), generator=g, device="cuda",
                                   dtype=torch.int32)
        self.lens = self.lens0.clone()
        self.k, self.v = (rand(nb, hkv, 16, d).bfloat16() for _ in "kv")
        self.pool = [torch.zeros_like(self.k) for _ in "kv"]
        self.q = rand(rows, hq, d).bfloat16()
        starts = torch.arange(rows + 1, device="cuda", dtype=torch.int32)
        spans = starts * mb * 16
        self.parents, self.tokens = (torch.zeros((n, beams), dtype=torch.int32, device="cuda")
                                     for _ in "pt")
        self.out, self.rows, self.calls = [], [], []
        slots = torch.randperm(nb * 16, generator=g, device="cuda")
        ws = pa.CrossWorkspace(1, hq, hkv, d)
        for _ in range(steps):
            logits = 3 * rand(rows, 2003)
            out = torch.zeros_like(self.q)
            ko, vo = (torch.zeros((nb * 16, hkv, d), dtype=torch.bfloat16, device="cuda")
                      for _ in "kv")
            self.out.append(out)
            self.rows.append((ko, vo))
            self.calls += [
                pa.BeamSelect(self.scores, self.parents, self.tokens, logits, self.scores, beams,
                              in_place=True),
                pa.ReorderStates([self.tables], self.parents, beams),
                pa.ReorderStates([self.lens], self.parents, beams),
                pa.CrossAttention(out, self.q, self.k, self.v, self.tables, self.lens.view(-1),
                                  starts, 1, d ** -0.5, ws),
                pa.ReadCache(ko, vo, self.k, self.v, self.tables, spans, mb * 16),
                pa.ReadCache(*self.pool, self.k, self.v, self.tables, spans, mb * 16,
                             slot_mapping=slots),
            ]

    def reset(self):
        self.scores.copy_(self.scores0)
        self.tables.copy_(self.tables0)
        self.lens.copy_(self.lens0)
        for t in [*self.out, *(x for r in self.rows for x in r), *self.pool]:
            t.zero_()
        torch.cuda.synchronize()

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in [self.scores, self.tables, self.lens, self.tokens, *self.out,
                                    *(x for r in self.rows for x in r), *self.pool]]


@pytest.mark.parametrize("d", [64, 128])
def test_calls_read_what_the_last_one_wrote(d):
    pa.pa_clear_device_error()
    s = Steps(d, 12)
    s.reset()
    for call in s.calls:
        call()
        torch.cuda.synchronize()
    want = s.results()
    assert not torch.equal(want[1], s.tables0) and not torch.equal(want[2], s.lens0)
    # rows of the last tables, by indexing
    at = s.tables.long().reshape(-1)
    for got, pool in zip(s.rows[-1], (s.k, s.v)):
        assert torch.equal(got, pool[at].transpose(1, 2).reshape(got.shape))
    for _ in range(5):
        s.reset()
        for call in s.calls:
            call()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        for call in s.calls:
            call()
    for _ in range(20):
        s.reset()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    assert pa.pa_get_device_error() == 0
