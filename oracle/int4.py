"""4-bit KV cache: quantisation and the values it stands for (oracle, test-only).

Each (token, KV head) row is quantised in groups of 64 dims:

    lo    = min of the group            (a bf16 value)
    scale = bf16((max - lo) * fl(1 / 15))   (float32 arithmetic, nearest even)
    code  = clamp(round_half_even((x - lo) / scale), 0, 15), 0 where scale is 0
    x    ~= lo + scale * code

Every step is one IEEE float32 operation, so the codes are reproduced exactly.
"""
import numpy as np

from .attention import softmax_attention
from .bf16 import bf16_bits_to_f64
from .rope import to_bf16_bits

GROUP = 64


def quantize(x_bits):
    """bf16 bits [..., D] -> codes uint8 [..., D], lo and scale bf16 bits [..., D / 64]."""
    x = bf16_bits_to_f64(np.asarray(x_bits)).astype(np.float32)
    g = x.reshape(x.shape[:-1] + (-1, GROUP))
    lo, hi = g.min(-1), g.max(-1)
    with np.errstate(over="ignore"):
        rng = np.minimum(hi - lo, np.finfo(np.float32).max)
    sc_bits = to_bf16_bits(rng * np.float32(1.0 / 15.0))
    sc = bf16_bits_to_f64(sc_bits).astype(np.float32)
    safe = np.where(sc > 0, sc, np.float32(1.0))[..., None]
    with np.errstate(over="ignore"):
        codes = np.clip(np.rint((g - lo[..., None]) / safe), 0, 15)
    codes = np.where(sc[..., None] > 0, codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), to_bf16_bits(lo), sc_bits


def values(codes, lo, scale):
    """The float64 values lo + scale * code."""
    lo, sc = (np.repeat(bf16_bits_to_f64(a), GROUP, axis=-1) for a in (lo, scale))
    return lo + sc * codes.astype(np.float64)


def decode(q, k_values, v_values, block_tables, context_lens, scale):
    """Paged decode over pools of values [NB, Hkv, 16, D] (float64): q [B, Hq, D]
    float64; an empty sequence gives zeros."""
    B, hq, _ = q.shape
    group = hq // k_values.shape[1]
    out = np.zeros(q.shape)
    for b in range(B):
        n = int(context_lens[b])
        if n == 0:
            continue
        pos = np.arange(n)
        phys = np.asarray(block_tables[b], dtype=np.int64)[pos // 16]
        K, V = k_values[phys, :, pos % 16, :], v_values[phys, :, pos % 16, :]
        for h in range(hq):
            out[b, h] = softmax_attention(q[b, h], K[:, h // group], V[:, h // group], scale)
    return out
