"""Paged attention with changed scores and masks, in float64 (oracle, test-only).

The query at position p sees the keys j with (j <= p or j < prefix) and, with a
window, j > p - window; its scores are

    s_j = cap tanh(x_j / cap) - slope |p - j|,   x_j = scale q . k_j

(cap 0: x_j itself; no slopes: no second term).  One new token per sequence is a
decode step.
"""
import numpy as np

from .attention import as_f64


def sequence(q_seq, k_cache, v_cache, table_row, ctx, scale, block_size=16, softcap=0.0,
             slopes=None, window=0, prefix=0):
    """Outputs [n, Hq, D] of the n newest tokens of one sequence.  Only the rows
    some query sees are read."""
    q_seq = as_f64(q_seq)
    n, hq, d = q_seq.shape
    out = np.zeros((n, hq, d))
    if n == 0 or ctx == 0:
        return out
    group = hq // k_cache.shape[1]
    first = max(0, ctx - n + 1 - window) if window else 0
    last = max(ctx, prefix)
    j = np.arange(first, last)
    phys = np.asarray(table_row, dtype=np.int64)[j // block_size]
    K, V = (as_f64(c[phys, :, j % block_size, :]) for c in (k_cache, v_cache))
    p = (ctx - n + np.arange(n))[:, None]
    seen = (j <= p) | (j < prefix)
    if window:
        seen &= j > p - window
    for h in range(hq):
        x = scale * (q_seq[:, h] @ K[:, h // group].T)
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[h]) * np.abs(p - j)
        x = np.where(seen, x, -np.inf)
        w = np.exp(x - x.max(axis=1, keepdims=True))
        out[:, h] = (w @ V[:, h // group]) / w.sum(axis=1, keepdims=True)
    return out


def batch(q, k_cache, v_cache, block_tables, context_lens, query_lens, scale, prefix_lens=None,
          **rule):
    """Sequences' new tokens back to back: q [T, Hq, D] -> [T, Hq, D] float64."""
    outs, row = [], 0
    for b, (ctx, n) in enumerate(zip(np.asarray(context_lens).tolist(),
                                     np.asarray(query_lens).tolist())):
        outs.append(sequence(q[row:row + n], k_cache, v_cache, block_tables[b], ctx, scale,
                             prefix=0 if prefix_lens is None else int(prefix_lens[b]), **rule))
        row += n
    return np.concatenate(outs, axis=0)
