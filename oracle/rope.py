"""Rotary position embedding (oracle, test-only).

For a token at position p and a head vector x, each pair (a, b) of its first R
dims -- (x[i], x[i + R / 2]), or (x[2 i], x[2 i + 1]) when interleaved -- turns
by the angle p f_i:  (a cos - b sin, b cos + a sin).  Dims from R on stay.

``rotate`` works in float64 from the angles' cosines and sines; ``rotate_fp32``
takes a float32 cosine / sine table and rounds every product and sum to float32
once, then the result to bf16: the library's definition, reproduced bit for bit.
"""
import numpy as np


def pair_index(rotary_dim, interleaved):
    """(first, second): the dims of pair i, i < R / 2."""
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def table(max_position, rotary_dim, base):
    """float64 cosines and sines [max_position, R / 2] each."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    angle = np.arange(max_position, dtype=np.float64)[:, None] * base ** (-2.0 * i / rotary_dim)
    return np.cos(angle), np.sin(angle)


def rotate(x, cos, sin, rotary_dim, interleaved):
    """x [T, H, D] float64; cos / sin [T, R / 2] float64."""
    x = np.array(x, dtype=np.float64)
    fa, fb = pair_index(rotary_dim, interleaved)
    a, b = x[..., fa].copy(), x[..., fb].copy()
    c, s = cos[:, None], sin[:, None]
    x[..., fa], x[..., fb] = a * c - b * s, b * c + a * s
    return x


def to_bf16_bits(x):
    """float32 -> bf16 bits, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rotate_fp32(x_bits, cos, sin, rotary_dim, interleaved):
    """bf16 bits [T, H, D] rotated with float32 cos / sin [T, R / 2]: bf16 bits."""
    x = (np.asarray(x_bits).astype(np.uint32) << 16).view(np.float32).copy()
    fa, fb = pair_index(rotary_dim, interleaved)
    a, b = x[..., fa].copy(), x[..., fb].copy()
    c, s = cos[:, None].astype(np.float32), sin[:, None].astype(np.float32)
    x[..., fa] = a * c - b * s
    x[..., fb] = b * c + a * s
    return to_bf16_bits(x)
