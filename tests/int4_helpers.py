"""The 4-bit pool's storage restated from the library's header, for the tests:
tiles of 9 * D bytes, codes then parameters."""
import numpy as np

from oracle import int4 as O4


def k_nibbles(d):
    """[d]: the nibble of a K row that holds dim j."""
    j = np.arange(d)
    e = j % 64
    return (d // 4) * (e // 16) + e % 16 + 16 * (j // 64)


def v_bytes(d):
    """([16, d] byte of the V tile, [d] shift) of token t's code of dim j."""
    t = np.arange(16)[:, None]
    j = np.arange(d)[None, :]
    c, i = j // 16, j % 8
    lane = 4 * i + (t % 8) // 2
    run = ((c // 4) ^ (i % 2)) if d == 128 else 0 * (c + i)
    at = lane * (d // 4) + 16 * run + 4 * (c % 4) + t // 8 + 2 * (t % 2)
    return at, np.where(np.arange(d) % 16 < 8, 0, 4)


def pack(codes, lo, scale, is_v):
    """codes uint8 [NB, Hkv, 16, D], parameters uint16 [NB, Hkv, 16, D / 64] -> pool bytes."""
    nb, hkv, _, d = codes.shape
    out = np.zeros((nb, hkv, 9 * d), dtype=np.uint8)
    if is_v:
        at, shift = v_bytes(d)
        for t in range(16):
            for j in range(d):
                out[:, :, at[t, j]] |= codes[:, :, t, j] << np.uint8(shift[j])
    else:
        nib = k_nibbles(d)
        for t in range(16):
            for j in range(d):
                out[:, :, t * d // 2 + nib[j] // 2] |= codes[:, :, t, j] << np.uint8(4 * (nib[j] % 2))
    par = np.stack([lo, scale], -1).astype("<u2")
    out[:, :, 8 * d:] = np.ascontiguousarray(par).view(np.uint8).reshape(nb, hkv, d)
    return out


def unpack(pool, d, is_v):
    """Inverse of pack: (codes, lo, scale)."""
    nb, hkv, _ = pool.shape
    codes = np.empty((nb, hkv, 16, d), dtype=np.uint8)
    if is_v:
        at, shift = v_bytes(d)
        codes[:] = (pool[:, :, at] >> shift.astype(np.uint8)) & 15
    else:
        nib = k_nibbles(d)
        rows = pool[:, :, :8 * d].reshape(nb, hkv, 16, d // 2)
        codes[:] = (rows[..., nib // 2] >> (4 * (nib % 2)).astype(np.uint8)) & 15
    par = np.ascontiguousarray(pool[:, :, 8 * d:]).view("<u2").reshape(nb, hkv, 16, d // 64, 2)
    return codes, par[..., 0], par[..., 1]


def pool_values(pool, d, is_v):
    """The float64 values [NB, Hkv, 16, D] a pool's bytes stand for."""
    return O4.values(*unpack(pool, d, is_v))


def write(key, value, kpool, vpool, slots):
    """The cache write on host pools (returned as new arrays)."""
    kpool, vpool = kpool.copy(), vpool.copy()
    d = key.shape[-1]
    for pool, x, is_v in ((kpool, key, False), (vpool, value, True)):
        codes, lo, sc = unpack(pool, d, is_v)
        qc, ql, qs = O4.quantize(x)
        for t, s in enumerate(np.asarray(slots).tolist()):
            if s >= 0:
                codes[s // 16, :, s % 16], lo[s // 16, :, s % 16] = qc[t], ql[t]
                sc[s // 16, :, s % 16] = qs[t]
        pool[:] = pack(codes, lo, sc, is_v)
    return kpool, vpool
