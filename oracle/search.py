"""Beam search and encoder-decoder operators in float64 (oracle, test-only): cross
attention to a paged source, the selection over beams and vocabulary, the
reordering of states, and the values a cache stands for read back.
"""
import math

import numpy as np

from .attention import as_f64


def cross_attention(q, k_cache, v_cache, block_tables, source_lens, query_lens, scale,
                    block_size=16):
    """q [T, Hq, D], the sequences' queries back to back; every query sees all of
    its source.  Returns (out, mean): out [T, Hq, D] and, in its place, the
    weighted mean of |V|, by which the rounding of the weights counts."""
    q = as_f64(q)
    out, mean = np.zeros(q.shape), np.zeros(q.shape)
    group = q.shape[1] // k_cache.shape[1]
    row = 0
    for b, (n, m) in enumerate(zip(np.asarray(source_lens).tolist(),
                                   np.asarray(query_lens).tolist())):
        if n:
            j = np.arange(n)
            phys = np.asarray(block_tables[b], dtype=np.int64)[j // block_size]
            K, V = (as_f64(c[phys, :, j % block_size, :]) for c in (k_cache, v_cache))
            for h in range(q.shape[1]):
                x = scale * (q[row:row + m, h] @ K[:, h // group].T)
                w = np.exp(x - x.max(axis=1, keepdims=True))
                w /= w.sum(axis=1, keepdims=True)
                out[row:row + m, h] = w @ V[:, h // group]
                mean[row:row + m, h] = w @ np.abs(V[:, h // group])
        row += m
    return out, mean


def totals(logits, scores, finished=None, eos=-1):
    """[rows, vocab] float64: each continuation's total, -inf where there is none."""
    logits = np.asarray(logits, dtype=np.float64)
    out = np.full(logits.shape, -np.inf)
    for r, row in enumerate(logits):
        s = float(scores[r])
        if not math.isfinite(s):
            continue
        if finished is not None and finished[r]:
            out[r, eos] = s
            continue
        x = np.where(row < np.inf, row, -np.inf)     # NaN and +inf are hidden
        if not np.any(x > -np.inf):
            continue
        top = x.max()
        out[r] = s + (x - (top + math.log(math.fsum(np.exp(x - top).tolist()))))
    return out


def keep_places(parents, beams):
    """The place of each of a search's continuations (parents: local beams, best
    first, None: none): the first of a beam takes its parent's place, the others
    the places left, in order."""
    place, free = [None] * len(parents), list(range(beams))
    for r, w in enumerate(parents):
        if w is not None and w in free:
            place[r] = w
            free.remove(w)
    return [free.pop(0) if p is None else p for p in place]


def beam_select(logits, scores, beams, keep, finished=None, eos=-1, in_place=False):
    """(scores float64, parents, tokens, finished) [searches, keep] of the best
    continuations; equal totals (in float64): the lower beam, of one beam the larger
    logit, then the lower token first."""
    logits = np.asarray(logits, dtype=np.float64)
    t = totals(logits, scores, finished, eos)
    rows, vocab = t.shape
    n = rows // beams
    out = np.full((n, keep), -np.inf)
    parents, tokens = (np.full((n, keep), -1, dtype=np.int64) for _ in "pt")
    done = np.zeros((n, keep), dtype=bool)
    for b in range(n):
        flat = t[b * beams:(b + 1) * beams].reshape(-1)
        index = np.arange(beams * vocab)
        x = np.nan_to_num(logits[b * beams:(b + 1) * beams].reshape(-1), nan=-np.inf)
        best = [i for i in np.lexsort((index, -x, index // vocab, -flat))[:keep].tolist()
                if flat[i] > -np.inf]
        who = [i // vocab for i in best] + [None] * (keep - len(best))
        place = keep_places(who, beams) if in_place else list(range(keep))
        for r, i in enumerate(best):
            out[b, place[r]] = flat[i]
            parents[b, place[r]] = b * beams + i // vocab
            tokens[b, place[r]] = i % vocab
            done[b, place[r]] = (i % vocab == eos) or bool(
                finished is not None and finished[b * beams + i // vocab])
    return out, parents, tokens, done


def reorder(state, parents, beams):
    """Rows of `state` after the move; a parent outside the row's group leaves it."""
    out = np.array(state, copy=True)
    for i, p in enumerate(np.asarray(parents).tolist()):
        if p >= 0 and p // beams == i // beams:
            out[i] = state[p]
    return out


def read_rows(values, block_tables, first, counts, block_size=16):
    """Rows of positions first[b] .. first[b] + counts[b] - 1 of pools of values
    [NB, Hkv, bs, D], the sequences' one after another."""
    rows = []
    for b, (f, n) in enumerate(zip(first, counts)):
        pos = np.arange(f, f + n)
        phys = np.asarray(block_tables[b], dtype=np.int64)[pos // block_size]
        rows.append(values[phys, :, pos % block_size, :])
    return np.concatenate(rows) if rows else np.zeros((0,) + values.shape[1::2])
