"""The float64 references of the search operators against plain loops and closed
forms, and the allocator's reordering against its model, on the CPU."""
import math

import numpy as np
import pytest

from oracle import search as OS
from oracle.allocator import BlockAllocatorModel, InvalidArg, PrefixCachingAllocatorModel
from paged_kv_cache_283_gb300 import pa


def _paged(rng, lens, hkv, d):
    nblk = [-(-n // 16) for n in lens]
    perm = rng.permutation(sum(nblk) + 2)
    tables = np.full((len(lens), max(1, *nblk)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(nblk):
        tables[b, :k] = perm[at:at + k]
        at += k
    return tables, *(rng.standard_normal((perm.shape[0], hkv, 16, d)) for _ in "kv")


def test_cross_attention_by_loops():
    rng = np.random.default_rng(1)
    lens, counts = [5, 0, 33], [2, 3, 1]
    tables, k, v = _paged(rng, lens, 2, 4)
    q = rng.standard_normal((6, 4, 4))
    out, mean = OS.cross_attention(q, k, v, tables, lens, counts, 0.5)
    row = 0
    for b, (n, m) in enumerate(zip(lens, counts)):
        for t in range(row, row + m):
            for h in range(4):
                ks = [k[tables[b, j // 16], h // 2, j % 16] for j in range(n)]
                vs = [v[tables[b, j // 16], h // 2, j % 16] for j in range(n)]
                w = [math.exp(0.5 * sum(a * c for a, c in zip(q[t, h], x))) for x in ks]
                for e in range(4):
                    want = sum(a * x[e] for a, x in zip(w, vs)) / sum(w) if n else 0.0
                    size = sum(a * abs(x[e]) for a, x in zip(w, vs)) / sum(w) if n else 0.0
                    assert abs(out[t, h, e] - want) < 1e-12
                    assert abs(mean[t, h, e] - size) < 1e-12
        row += m


def test_cross_attention_closed_forms():
    rng = np.random.default_rng(2)
    tables, k, v = _paged(rng, [1, 40], 1, 4)
    k[tables[1, :3]] = 0.25                              # equal keys: the mean of V
    out, _ = OS.cross_attention(rng.standard_normal((2, 1, 4)), k, v, tables, [1, 40], [1, 1], 1.0)
    assert np.allclose(out[0, 0], v[tables[0, 0], 0, 0], atol=1e-14)
    rows = OS.read_rows(v, tables, [0, 0], [1, 40])[1:, 0]
    assert np.allclose(out[1, 0], rows.mean(0), atol=1e-13)


def test_selection_by_loops():
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((6, 7)) * 3
    logits[4, 2:5] = -np.inf
    scores = rng.standard_normal(6)
    got = OS.beam_select(logits, scores, 3, 5, finished=[0, 1, 0, 0, 0, 0], eos=6)
    for b in range(2):
        every = []
        for w in range(3):
            r = 3 * b + w
            if r == 1:
                every.append((scores[r], r, 6))
                continue
            z = sum(math.exp(x) for x in logits[r])
            every += [(scores[r] + math.log(math.exp(x) / z), r, v)
                      for v, x in enumerate(logits[r]) if x > -np.inf]
        every.sort(key=lambda e: -e[0])
        for i, (x, r, v) in enumerate(every[:5]):
            assert abs(got[0][b, i] - x) < 1e-12 and got[1][b, i] == r and got[2][b, i] == v
            assert got[3][b, i] == (v == 6 or r == 1)


def test_selection_probabilities_sum_to_one():
    rng = np.random.default_rng(4)
    t = OS.totals(rng.standard_normal((3, 50)) * 10, [0.0, -1.0, -np.inf])
    assert np.allclose(np.exp(t).sum(1), [1.0, math.exp(-1.0), 0.0])


def test_selection_ties_and_missing():
    logits = np.zeros((2, 4))
    s, p, t, _ = OS.beam_select(logits, [0.0, 0.0], 2, 6)
    assert p[0].tolist() == [0] * 4 + [1] * 2 and t[0].tolist() == [0, 1, 2, 3, 0, 1]
    logits[0, 1:] = -np.inf
    logits[1] = [np.nan, np.inf, -np.inf, 1.0]
    s, p, t, _ = OS.beam_select(logits, [-1.0, -0.5], 2, 3)
    assert p[0].tolist() == [1, 0, -1] and t[0].tolist() == [3, 0, -1]
    assert s[0].tolist() == [-0.5, -1.0, -np.inf]


@pytest.mark.parametrize("parents,place", [
    ([0, 1, 2], [0, 1, 2]), ([2, 2, 2], [2, 0, 1]), ([1, 0, 1], [1, 0, 2]),
    ([2, 0, 0], [2, 0, 1]), ([1, None, None], [1, 0, 2]), ([None] * 3, [0, 1, 2])])
def test_places(parents, place):
    assert OS.keep_places(parents, 3) == place


def test_places_make_moves_idempotent():
    rng = np.random.default_rng(5)
    for _ in range(50):
        beams = int(rng.integers(1, 9))
        who = rng.integers(0, beams, beams).tolist()
        place = OS.keep_places(who, beams)
        parents = np.empty(beams, dtype=int)
        parents[place] = who
        assert sorted(place) == list(range(beams))
        assert (parents[parents] == parents).all()


def test_reorder_rows():
    x = np.arange(12).reshape(6, 2)
    got = OS.reorder(x, [2, 0, 1, 3, 3, -1], 3)
    assert got.tolist() == x[[2, 0, 1, 3, 3, 5]].tolist()
    assert OS.reorder(x, [5, 1, 2, 0, 4, 5], 3).tolist() == x.tolist()   # other groups' rows


def _same(model, real, seqs):
    assert list(real.free_list()) == model.free_list()
    assert [real.refcount(b) for b in range(model.num_blocks)] == model.ref
    for s in seqs:
        assert list(real.block_table(s)) == model.block_table(s)
        assert real.seq_len(s) == model.seq_len(s)


@pytest.mark.parametrize("seed", range(4))
def test_allocator_reorder_matches_model(seed):
    rng = np.random.default_rng(100 + seed)
    nb, beams = 64, 4
    model, real = BlockAllocatorModel(nb, 16), pa.BlockAllocator(nb, 16)
    seqs = list(range(beams))
    for a in (model, real):
        a.add_seq(0)
        a.reserve(0, 37)
        for s in seqs[1:]:
            a.fork(0, s)
    for _ in range(60):
        want = model.append_slots(seqs)
        got = real.append_slots(seqs)
        assert [w[0] for w in want] == got[0].tolist()
        assert [(w[1], w[2]) for w in want] == list(zip(got[1].tolist(), got[2].tolist()))
        parents = rng.integers(-1, beams, beams).tolist()
        model.reorder(seqs, parents)
        real.reorder(seqs, parents)
        _same(model, real, seqs)
    for s in seqs:
        model.free_seq(s)
        real.free_seq(s)
    assert real.num_free() == nb
    _same(model, real, [])


def test_allocator_reorder_keeps_cached_blocks():
    model, real = PrefixCachingAllocatorModel(16, 16), pa.BlockAllocator(16, 16)
    real.enable_prefix_cache()
    for a in (model, real):
        a.add_seq_prompt(0, list(range(40)))
        a.add_seq_prompt(1, list(range(100, 133)))
        a.reorder([0, 1], [1, 1])            # sequence 0's named blocks become evictable
    _same(model, real, [0, 1])
    assert real.evictable_list().tolist() == model.evictable_list() != []


def test_allocator_reorder_refusals():
    a = pa.BlockAllocator(8, 16)
    for s in range(3):
        a.add_seq(s)
        a.reserve(s, 17)
    before = [a.block_table(s).tolist() for s in range(3)]
    for seqs, parents in (([0, 0], [0, 1]), ([0, 9], [0, 0]), ([0, 1], [2, 0])):
        with pytest.raises(pa.PAError):
            a.reorder(seqs, parents)
    with pytest.raises(ValueError):
        a.reorder([0, 1], [0])
    with pytest.raises(InvalidArg):
        BlockAllocatorModel(2, 16).reorder([0], [0])
    assert [a.block_table(s).tolist() for s in range(3)] == before
    assert pa.lib().pa_alloc_reorder(None, None, None, 0) == pa.PA_ERR_INVALID_ARG
    a.reorder([], [])
