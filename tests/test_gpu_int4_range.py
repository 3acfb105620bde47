"""The 4-bit decode where its weights' range and its long contexts can go wrong:
tokens whose V scale is far above the others' and whose weight is not, a heavy
token before many light ones, V scales at both ends of their type, and contexts in
which every block in turn holds all of one query's weight."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from int4_helpers import pack, pool_values, unpack
from oracle import int4 as O4
from oracle.bf16 import bf16_bits_to_f64
from oracle.rope import to_bf16_bits
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import bf16_to_f64, dev_bf16

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _bits(x):
    """A float32 value as bf16 bits."""
    return int(to_bf16_bits(np.array([x], dtype=np.float32))[0])


def _normal(rng, nb, hkv, d):
    """(codes, offsets, scales) of quantised normal values."""
    return list(O4.quantize(normal_bf16(rng, (nb, hkv, 16, d))))


def _ways(q, pools, tables, ctx, scale, parts):
    """The outputs of the whole pass, and of the split step for each partition size."""
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    t, c, dq = _dev(tables, np.int32), _dev(ctx, np.int32), dev_bf16(q)
    B, hq, d = q.shape
    pa.pa_clear_device_error()
    out = torch.full_like(dq, float("nan"))
    pa.pa_decode_int4(out, dq, dk, dv, t, c, scale)
    yield "whole", bf16_to_f64(out)
    for part in parts:
        ws = pa.splitk_workspace(B, hq, d, int(np.max(ctx)), part)
        for w in ws:
            w.fill_(float("nan"))
        counters = pa.step_counters(B, dk.shape[1])
        out.fill_(float("nan"))
        pa.pa_decode_step(out, dq, dk, dv, t, c, scale, partition_size=part, workspace=ws,
                          counters=counters)
        yield f"partitions of {part}", bf16_to_f64(out)
        assert not counters.any()
    assert pa.pa_get_device_error() == 0


def _rows(q, pools, tables, ctx, scale):
    """The float64 outputs and each one's tolerance [B, Hq, D].

    An output is sum p (lo + sc code) / sum p.  Half a step of bf16 (2^-8 of the
    result); half a step of f16 (2^-11) in each weight p sc, so at most that of sum
    p sc code; the scores to 2^-13 (sums of up to 128 products in fp32 and the
    exponential's 2^-22), so at most that of sum p (|lo| + sc code)."""
    d = q.shape[2]
    K = pool_values(pools[0], d, False)
    codes, lo, sc = unpack(pools[1], d, True)
    lo, sc = (np.repeat(bf16_bits_to_f64(a), 64, axis=-1) for a in (lo, sc))
    part = sc * codes
    args = (tables, ctx, scale)
    q = bf16_bits_to_f64(q)
    ref = O4.decode(q, K, lo + part, *args)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * O4.decode(q, K, part, *args) + \
        2.0 ** -13 * O4.decode(q, K, np.abs(lo) + part, *args)
    return ref, tol


def _check(q, pools, tables, ctx, scale, parts, what):
    ref, tol = _rows(q, pools, tables, ctx, scale)
    for how, got in _ways(q, pools, tables, ctx, scale, parts):
        assert np.isfinite(got).all(), f"{what}, {how}: not finite"
        bad = np.abs(got - ref) > tol
        assert not bad.any(), \
            f"{what}, {how}: off by up to {(np.abs(got - ref) / tol).max():.1f} tolerances"


@pytest.mark.parametrize("ratio", [14, 17, 20, 60])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (128, 8, 1), (64, 4, 2)])
def test_int4_light_token_with_a_large_scale(ratio, d, hq, hkv):
    # one token in thirty has a weight of about e^-60 of the others' and a V scale
    # 2^ratio times theirs
    rng = np.random.default_rng(ratio + d + hq)
    n = 700
    K, V = _normal(rng, 44, hkv, d), _normal(rng, 44, hkv, d)
    light = np.arange(9, n, 30)
    at = (light // 16, slice(None), light % 16)
    K[0][at], K[1][at], K[2][at] = 0, _bits(-60 / (0.08 * 0.8 * d)), 0
    V[2][at] = _bits(0.3 * 2.0 ** ratio)
    pools = [pack(*K, False), pack(*V, True)]
    q = normal_bf16(rng, (1, hq, d)) & 0x7FFF       # sum q about 0.8 d
    _check(q, pools, np.arange(44)[None], [n], 0.08, (16, 64, 512), f"2^{ratio}")


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (128, 8, 1), (64, 4, 2)])
def test_int4_heavy_token_beside_large_scales(d, hq, hkv):
    # scores of 0 but for one of about 13 in sixteen blocks' first tokens; every
    # fiftieth token has 64 times the others' V scale
    rng = np.random.default_rng(d + hq)
    n, nb = 8190, 512
    K, V = _normal(rng, nb, hkv, d), _normal(rng, nb, hkv, d)
    K[0][:], K[1][:], K[2][:] = 0, 0, 0
    heavy = np.arange(16) * 16
    K[1][heavy // 16, :, heavy % 16] = _bits(13 / (0.08 * 0.8 * d))
    big = np.arange(37, n, 50)
    V[2][big // 16, :, big % 16] = _bits(0.3 * 64)
    pools = [pack(*K, False), pack(*V, True)]
    q = normal_bf16(rng, (1, hq, d)) & 0x7FFF
    _check(q, pools, np.arange(nb)[None], [n], 0.08, (512, 4096), "heavy token")


@pytest.mark.parametrize("power", [115, 110, 60, -60, -110, -124])
def test_int4_scales_at_the_ends_of_their_type(power):
    rng = np.random.default_rng(200 + power)
    K, V = _normal(rng, 4, 2, 128), _normal(rng, 4, 2, 128)
    V[1][:] = _bits(2.0 ** power)
    V[2][:] = rng.choice([_bits(2.0 ** power * f) for f in (1.0, 1.25, 1.75)], V[2].shape)
    pools = [pack(*K, False), pack(*V, True)]
    q = normal_bf16(rng, (1, 8, 128))
    _check(q, pools, np.arange(4)[None], [61], 0.08, (16, 64), f"2^{power}")


def test_int4_scales_that_rise_and_fall():
    # scales over 80 powers of two in both directions, scores rising along the context
    rng = np.random.default_rng(31)
    n, nb = 1600, 100
    K, V = _normal(rng, nb, 2, 128), _normal(rng, nb, 2, 128)
    j = np.arange(nb * 16)
    for dims, power in ((0, 40 * np.sin(j / 200.0)), (1, 40 - j / 20.0)):
        V[2][j // 16, :, j % 16, dims] = to_bf16_bits((2.0 ** power).astype(np.float32))[:, None]
        V[1][j // 16, :, j % 16, dims] = 0
    K[1][j // 16, :, j % 16] = to_bf16_bits((j / 1600.0 * 4).astype(np.float32))[:, None, None]
    pools = [pack(*K, False), pack(*V, True)]
    q = normal_bf16(rng, (1, 8, 128)) & 0x7FFF
    _check(q, pools, np.arange(nb)[None], [n], 0.05, (64, 512), "rise and fall")


@pytest.mark.parametrize("d,hq,hkv,n", [(128, 8, 2, 20000), (128, 8, 1, 9000), (128, 4, 2, 8191),
                                        (64, 8, 2, 12345)])
def test_int4_every_block_holds_some_query(d, hq, hkv, n):
    """Sequences that share one table, and for every block a (sequence, head) whose
    whole weight lies on it: a block that is skipped, taken twice, or taken in
    another's place shows in that output."""
    rng = np.random.default_rng(n)
    nb = -(-n // 16)
    group = hq // hkv
    sign = rng.choice([0, 15], (nb, hkv, 1, d)).astype(np.uint8)
    one = np.full((nb, hkv, 16, d // 64), 0x3F80, dtype=np.uint16)
    K = pack(np.repeat(sign, 16, 2), np.full_like(one, _bits(-7.5)), one, False)
    V = _normal(rng, nb, hkv, d)
    perm = rng.permutation(nb)                     # logical block i lies at perm[i]
    B = -(-nb // group)                            # every block for every KV head
    aim = (np.arange(B)[:, None] * group + np.arange(hq) % group) % nb
    r = (sign.astype(np.int64) - 7.5)[perm[aim], (np.arange(hq) // group)[None], 0]
    q = to_bf16_bits((r / 7.5).astype(np.float32))
    # the aimed block's scores are 7.5 d scale, any other's at least 30 below (two
    # random rows of signs agree in less than d / 2 + 6 sqrt(d) / 2 places)
    scale = 30 / (7.5 * (d - 6 * d ** 0.5))
    v = O4.values(*V)[perm]
    part = (np.repeat(bf16_bits_to_f64(V[2]), 64, -1) * V[0])[perm]
    live = np.minimum(16, n - 16 * np.arange(nb))[:, None, None]
    keep = (np.arange(16)[None, :] < live[:, :, 0])[:, None, :, None]
    mean, size = ((x * keep).sum(2) / live for x in (v, part))
    pick = (aim, (np.arange(hq) // group)[None])
    ref = mean[pick]
    # bf16 and f16 rounding as in _rows; 20,000 other tokens weigh at most e^-30 each
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * size[pick] + 2.0 ** -12
    tables = np.repeat(perm[None], B, 0)
    for how, got in _ways(q, [K, pack(*V, True)], tables, [n] * B, scale, (1024, 4096, 8192)):
        bad = (np.abs(got - ref) > tol).any(-1)
        assert not bad.any(), f"{how}: blocks {sorted(set(aim[bad].tolist()))[:9]} wrong"


@pytest.mark.parametrize("ctx,hq,hkv,d", [([9000, 4096, 4097, 63, 1], 8, 2, 128),
                                          ([5000, 8191, 7], 4, 2, 128), ([9000, 4160], 4, 2, 64)])
def test_int4_long_contexts_by_norm(ctx, hq, hkv, d):
    """Normal values: each (sequence, head)'s error against the size of its output.
    bf16 takes 2^-8 of it at most.  A product p sc has a rounding of its own, 2^-11 of
    it at most (a root mean square of 0.58 of that); with scores of one unit's spread
    sum p^2 is e / n of (sum p)^2, and sc code is 3 in root mean square, so that an
    output is off by 0.58 * 3 * 2^-11 = 8.5e-4 of its own spread, sqrt(e / n), in root
    mean square: four times that at most (twice what the largest of a thousand groups
    of 64 values that share their roundings should be).  The MMA's sums are truncated,
    some 2^-25 a step of sums of 2.4: 128 steps make 1e-5, of outputs of 0.018.  In all
    2^-8 + 3.4e-3 + 5e-4 = 7.8e-3."""
    rng = np.random.default_rng(len(ctx) + d)
    nblk = [-(-n // 16) for n in ctx]
    perm = rng.permutation(sum(nblk))
    tables = np.full((len(ctx), max(nblk)), -1, dtype=np.int32)
    for b, at in enumerate(np.cumsum([0] + nblk[:-1])):
        tables[b, :nblk[b]] = perm[at:at + nblk[b]]
    pools = [pack(*_normal(rng, len(perm), hkv, d), v) for v in (False, True)]
    q = normal_bf16(rng, (len(ctx), hq, d))
    ref = O4.decode(bf16_bits_to_f64(q), pool_values(pools[0], d, False),
                    pool_values(pools[1], d, True), tables, ctx, 0.088)
    for how, got in _ways(q, pools, tables, ctx, 0.088, (1024, 4096)):
        off = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert (off <= 7.8e-3).all(), f"{how}: off by {off.max():.2e} of the output"


@pytest.mark.parametrize("d,hq,hkv,n", [(128, 4, 1, 100000), (64, 2, 1, 100000),
                                        (128, 8, 1, 40000)])
def test_int4_whole_long_contexts_by_norm(d, hq, hkv, n):
    """One warp's sums over thousands of tokens: 7.8e-3 of each output's norm, as above
    (the MMA's truncation in runs of 32 steps of 64 tokens at most, so 1e-5 again, of
    outputs of 0.005: 2e-3 instead of 5e-4), together 9.3e-3."""
    rng = np.random.default_rng(n + d)
    nb = -(-n // 16)
    pools = [pack(*_normal(rng, nb, hkv, d), v) for v in (False, True)]
    q = normal_bf16(rng, (1, hq, d))
    tables = rng.permutation(nb)[None]
    scale = d ** -0.5
    ref = O4.decode(bf16_bits_to_f64(q), pool_values(pools[0], d, False),
                    pool_values(pools[1], d, True), tables, [n], scale)
    for how, got in _ways(q, pools, tables, [n], scale, (8192, 16384, 131072)):
        off = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert (off <= 9.3e-3).all(), f"{how}: off by {off.max():.2e} of the output"
