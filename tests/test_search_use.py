"""What the README shows of a search, as far as it runs without a GPU."""
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _searches(n, beams):
    alloc = pa.BlockAllocator(64, 16)
    ids = [10 + r for r in range(n * beams)]
    for r in ids:
        alloc.add_seq(r)
        alloc.reserve(r, 5 + r)
    return alloc, ids


def _same(a, b, ids):
    x, y = a.block_tables(ids, 4), b.block_tables(ids, 4)
    return np.array_equal(x[0], y[0]) and np.array_equal(x[1], y[1]) and np.array_equal(
        a.free_list(), b.free_list())


@pytest.mark.parametrize("n,beams", [(1, 3), (2, 4), (5, 1)])
def test_readme_reorders_by_a_selections_parents(n, beams):
    """parents as the selection leaves them: [searches, beams], numbers of rows."""
    with open(README) as f:
        lines = re.findall(r"^(alloc\.reorder\(.*?\))\s*#", f.read(), flags=re.M)
    assert lines
    rows = np.arange(n * beams)
    parents = np.where(rows % 3 == 2, -1, rows // beams * beams + (rows * 7 + 1) % beams)
    want, ids = _searches(n, beams)
    want.reorder(ids, parents.tolist())
    for line in lines:
        for beam_ids in (ids, np.array(ids).reshape(n, beams)):
            alloc, _ = _searches(n, beams)
            exec(line, {"alloc": alloc, "beam_ids": beam_ids,
                        "parents": torch.tensor(parents, dtype=torch.int32).view(n, beams)})
            assert _same(alloc, want, ids)


def test_one_parent_per_sequence():
    alloc, ids = _searches(2, 2)
    before, _ = _searches(2, 2)
    for parents in ([0, 1, 2], [[0, 1], [2, 3], [0, 1]], [0], []):
        with pytest.raises(ValueError):
            alloc.reorder(ids, parents)
    for parents in ([0, 1, 2, 4], [[0, 1], [2, 9]]):
        with pytest.raises(pa.PAError):
            alloc.reorder(ids, parents)
    assert _same(alloc, before, ids)
    alloc.reorder([], [])
    assert _same(alloc, before, ids)
