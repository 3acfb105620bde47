"""The oracles of the rotary embedding, the 4-bit cache and attention with
changed scores, pinned by closed forms, brute force and the plain oracles; the
refusals of the entry points, which no call passes to a GPU."""
import ctypes
import math

import numpy as np
import pytest

from int4_helpers import k_nibbles, pack, pool_values, unpack, v_bytes, write
from oracle import attention as OA
from oracle import biased as OB
from oracle import int4 as O4
from oracle import prefill as OP
from oracle import rope as OR
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(pa.LIB_PATH):
        from paged_kv_cache_283_gb300 import build
        build.build()
    return pa.lib()


# ------------------------------------------------------------------- rotation

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_turn(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64))
    cos, sin = OR.table(300, 32, 10000.0)
    p = np.array([0, 1, 7, 100, 299])
    y = OR.rotate(x, cos[p], sin[p], 32, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    fa, fb = OR.pair_index(32, interleaved)
    assert np.allclose(y[..., fa] ** 2 + y[..., fb] ** 2, x[..., fa] ** 2 + x[..., fb] ** 2)
    # position 1, pair 0: the angle is one radian
    a, b = x[1, 0, fa[0]], x[1, 0, fb[0]]
    assert math.isclose(y[1, 0, fa[0]], a * math.cos(1) - b * math.sin(1))
    # scores depend on the distance alone
    q, k = rng.standard_normal((2, 1, 1, 64))
    dots = [float(np.sum(OR.rotate(q, cos[[i]], sin[[i]], 32, interleaved) *
                         OR.rotate(k, cos[[j]], sin[[j]], 32, interleaved)))
            for i, j in ((10, 3), (110, 103))]
    assert math.isclose(dots[0], dots[1])


def test_rotation_in_fp32_is_near_the_exact_one():
    # three float32 roundings of |a c| + |b s| each half a step (2^-24), and
    # the table's 2^-24 twice; the bf16 rounding half a step (2^-8)
    rng = np.random.default_rng(2)
    x = normal_bf16(rng, (9, 2, 128))
    cos, sin = OR.table(100, 128, 10000.0)
    p = rng.integers(0, 100, 9)
    got = bf16_bits_to_f64(OR.rotate_fp32(x, cos[p].astype(np.float32),
                                          sin[p].astype(np.float32), 128, False))
    f = bf16_bits_to_f64(x)
    ref = OR.rotate(f, cos[p], sin[p], 128, False)
    size = np.abs(f).max()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * size * 4 * 2.0 ** -24)


def test_bf16_rounding():
    x = np.array([1.0, 1.00390625, 1.01171875, -2.5, 0.0], dtype=np.float32)
    # 1 + 2^-8 ties to even (1.0), 1 + 3 * 2^-8 ties to even (1 + 2^-6)
    assert bf16_bits_to_f64(OR.to_bf16_bits(x)).tolist() == [1.0, 1.0, 1.015625, -2.5, 0.0]


# ---------------------------------------------------------------- 4-bit cache

def test_int4_hand_worked_group():
    x = np.zeros(64, dtype=np.float32)
    x[:4] = [-3.0, 12.0, 0.5, 1.5]          # lo -3, scale 1; 3.5 and 4.5 tie to 4
    codes, lo, sc = O4.quantize(OR.to_bf16_bits(x))
    assert bf16_bits_to_f64(lo) == [-3.0] and bf16_bits_to_f64(sc) == [1.0]
    assert codes[:5].tolist() == [0, 15, 4, 4, 3]
    same = O4.quantize(OR.to_bf16_bits(np.full(64, 2.5, np.float32)))
    assert not same[0].any() and bf16_bits_to_f64(same[2]) == [0.0]
    assert np.all(O4.values(*same) == 2.5)


def test_int4_error_is_half_a_step():
    # the code's rounding (scale / 2) and, at the top, the scale's (15 * 2^-9 of it)
    x = normal_bf16(np.random.default_rng(3), (50, 2, 128))
    codes, lo, sc = O4.quantize(x)
    err = np.abs(O4.values(codes, lo, sc) - bf16_bits_to_f64(x))
    step = np.repeat(bf16_bits_to_f64(sc), 64, -1)
    assert np.all(err <= step * (0.5 + 15 * 2.0 ** -8 + 1e-6))
    assert codes.max() == 15 and codes.min() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_int4_layout_is_a_bijection(d):
    at, shift = v_bytes(d)
    places = 2 * at + shift[None] // 4
    assert np.array_equal(np.sort(places.reshape(-1)), np.arange(16 * d))
    assert np.array_equal(np.sort(k_nibbles(d)), np.arange(d))
    for t in range(16):            # two tokens share no byte
        for u in range(t):
            assert not set(at[t]) & set(at[u])
    rng = np.random.default_rng(d)
    codes = rng.integers(0, 16, (3, 2, 16, d)).astype(np.uint8)
    lo, sc = rng.integers(0, 1 << 15, (2, 3, 2, 16, d // 64)).astype(np.uint16)
    for is_v in (False, True):
        back = unpack(pack(codes, lo, sc, is_v), d, is_v)
        assert all(np.array_equal(a, b) for a, b in zip(back, (codes, lo, sc)))


def test_int4_layout_hand_worked():
    assert k_nibbles(128)[[0, 1, 15, 16, 64, 79, 80, 127]].tolist() == \
        [0, 1, 15, 32, 16, 31, 48, 127]
    at, shift = v_bytes(128)
    assert [at[t, 0] for t in (0, 8, 1, 9)] == [0, 1, 2, 3] and shift[0] == 0
    assert at[0, 8] == 0 and shift[8] == 4          # dim 8: the same byte's high half
    assert at[2, 0] == 32 and at[0, 16] == 4 and at[0, 64] == 16
    assert at[0, 1] == 4 * 32 + 16 and at[0, 65] == 4 * 32


def test_int4_write_and_decode_of_exact_values():
    rng = np.random.default_rng(4)
    nb, hkv, d = 4, 2, 64
    kp, vp = rng.integers(0, 256, (2, nb, hkv, 9 * d)).astype(np.uint8)
    # integers 0..15 with both ends present are exact: lo 0, scale 1
    x = rng.integers(0, 16, (20, hkv, d))
    x[..., 0], x[..., 1] = 0, 15
    key = OR.to_bf16_bits(x.astype(np.float32))
    val = OR.to_bf16_bits(x[::-1].astype(np.float32))
    table = np.array([[3, 1]])
    slots = [3 * 16 + i for i in range(16)] + [16 + i for i in range(4)]
    k2, v2 = write(key, val, kp, vp, slots)
    K, V = pool_values(k2, d, False), pool_values(v2, d, True)
    assert np.array_equal(K[3, :, 5], x[5]) and np.array_equal(V[1, :, 2], x[::-1][18])
    assert np.array_equal(k2[[0, 2]], kp[[0, 2]])
    q = rng.standard_normal((1, 4, d))
    got = O4.decode(q, K, V, table, [20], 0.1)
    ref = OA.decode(q, K, V, table, np.array([20]), 0.1, 16)
    assert np.allclose(got, ref, atol=1e-12)


# --------------------------------------------------------- changed scores

def _case(seed, chunks, hq=4, hkv=2, d=8):
    rng = np.random.default_rng(seed)
    ctx = np.array([p + n for p, n in chunks])
    nblk = -(-ctx // 16)
    nb = int(nblk.sum()) + 2
    perm = rng.permutation(nb)
    tables = np.full((len(chunks), int(nblk.max())), -1)
    at = 0
    for b, k in enumerate(nblk):
        tables[b, :k] = perm[at:at + k]
        at += k
    kc, vc = rng.standard_normal((2, nb, hkv, 16, d))
    q = rng.standard_normal((sum(n for _, n in chunks), hq, d))
    return q, kc, vc, tables, ctx, np.array([n for _, n in chunks])


def test_biased_without_a_rule_is_prefill():
    q, kc, vc, tables, ctx, n = _case(5, [(0, 5), (30, 1), (7, 20)])
    assert np.allclose(OB.batch(q, kc, vc, tables, ctx, n, 0.3),
                       OP.prefill(q, kc, vc, tables, ctx, n, 0.3, 16), atol=1e-12)


def test_biased_by_brute_force():
    q, kc, vc, tables, ctx, n = _case(6, [(11, 9), (0, 18)])
    slopes, cap, window, prefix = [0.5, 0.25, 0.1, 0.0], 0.7, 6, [15, 3]
    got = OB.batch(q, kc, vc, tables, ctx, n, 0.9, prefix_lens=prefix, softcap=cap,
                   slopes=slopes, window=window)
    row = 0
    for b in range(2):
        for i in range(n[b]):
            p = ctx[b] - n[b] + i
            for h in range(4):
                num, den = np.zeros(8), 0.0
                for j in range(ctx[b]):
                    if not ((j <= p or j < prefix[b]) and p - j < window):
                        continue
                    k = kc[tables[b, j // 16], h // 2, j % 16]
                    x = 0.9 * sum(q[row, h, e] * k[e] for e in range(8))
                    w = math.exp(cap * math.tanh(x / cap) - slopes[h] * abs(p - j))
                    num, den = num + w * vc[tables[b, j // 16], h // 2, j % 16], den + w
                assert np.allclose(got[row, h], num / den, atol=1e-12)
            row += 1


def test_biased_closed_forms():
    q, kc, vc, tables, ctx, n = _case(7, [(40, 1)])
    last = vc[tables[0, 2], :, 8].repeat(2, axis=0)
    # a window of one token, or a steep slope, leaves the newest value alone
    assert np.allclose(OB.batch(q, kc, vc, tables, ctx, n, 1.0, window=1)[0], last)
    assert np.allclose(OB.batch(q, kc, vc, tables, ctx, n, 1.0, slopes=[1e4] * 4)[0], last)
    # a window as long as the context hides nothing; an infinite-like cap changes nothing
    full = OB.batch(q, kc, vc, tables, ctx, n, 1.0)
    assert np.allclose(OB.batch(q, kc, vc, tables, ctx, n, 1.0, window=41), full)
    assert np.allclose(OB.batch(q, kc, vc, tables, ctx, n, 1.0, softcap=1e6), full)


# ------------------------------------------------------------------- refusals
# Every call fails a host check: the fake addresses never reach a kernel.

F = ctypes.c_void_p(0x10000)


def test_rope_host_checks(lib):
    def call(kind="", q_out=ctypes.c_void_p(0x90000000), q=F, qs=4096, key=F, ks=1024, value=F,
             vs=1024, slots=F, pos=F, cs=F, maxp=100, rot=128, inter=0, T=3, hq=32, hkv=8, d=128,
             bs=16, nb=10, kc=F, scales=F):
        fn = getattr(lib, "pa_rope_reshape_and_cache" + kind)
        sc = (scales, scales) if kind in ("_int8", "_fp8") else ()
        return fn(q_out, q, qs, key, ks, value, vs, kc, F, *sc, slots, pos, cs, maxp, rot, inter,
                  T, hq, hkv, d, bs, nb, None)

    bad, shape = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED_SHAPE
    for kind in ("", "_int8", "_fp8", "_int4"):
        assert call(kind, d=96) == shape
        assert call(kind, rot=24) == shape           # not a multiple of 16
        assert call(kind, rot=0) == bad and call(kind, rot=144) == bad
        assert call(kind, maxp=0) == bad and call(kind, inter=2) == bad
        assert call(kind, qs=4000) == bad and call(kind, qs=4100) == bad
        assert call(kind, ks=1020) == bad and call(kind, vs=1025) == bad
        assert call(kind, key=None) == bad and call(kind, pos=None) == bad
        assert call(kind, cs=ctypes.c_void_p(0x10004)) == bad
        assert call(kind, slots=ctypes.c_void_p(0x10004)) == bad
        assert call(kind, q_out=None) == bad and call(kind, q=ctypes.c_void_p(0x10008)) == bad
        assert call(kind, q_out=F, qs=8192) == bad   # in place, but not the same rows
        assert call(kind, q_out=ctypes.c_void_p(0x10100)) == bad     # overlaps q
        assert call(kind, q=ctypes.c_void_p(0x80000000), q_out=F) == bad  # overlaps key
        assert call(kind, T=-1) == bad and call(kind, hkv=0) == bad and call(kind, nb=0) == bad
        assert call(kind, T=0) == pa.PA_OK
    assert call("_int4", bs=32) == shape and call("_int8", bs=32) == shape
    assert call("_fp8", scales=None) == bad


def test_int4_host_checks(lib):
    bad, shape = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED_SHAPE
    assert lib.pa_reshape_and_cache_int4(F, F, F, F, F, 3, 8, 96, 16, 10, None) == shape
    assert lib.pa_reshape_and_cache_int4(F, F, F, F, F, 3, 8, 128, 32, 10, None) == shape
    assert lib.pa_reshape_and_cache_int4(F, None, F, F, F, 3, 8, 128, 16, 10, None) == bad
    assert lib.pa_reshape_and_cache_int4(None, None, None, None, None, 0, 8, 128, 16, 10,
                                         None) == pa.PA_OK
    dec = (4, F, 2, 32, 8, 128, 16, 10, 0.1)
    assert lib.pa_decode_int4(None, F, F, F, F, *dec, None) == bad
    assert lib.pa_decode_int4(F, F, F, ctypes.c_void_p(0x10008), F, *dec, None) == bad
    assert lib.pa_decode_int4(F, F, F, F, F, 4, F, 2, 32, 8, 96, 16, 10, 0.1, None) == shape
    assert lib.pa_decode_int4(F, F, F, F, F, 4, F, 2, 8, 8, 128, 16, 10, 0.1, None) == shape
    assert lib.pa_decode_splitk_int4(F, F, F, 4, F, F, F, F, *dec, 100, None) == bad
    assert lib.pa_decode_splitk_int4(None, F, F, 4, F, F, F, F, *dec, 512, None) == bad

    def step(out=F, key=F, part=512, ws=F, counters=F, maxp=4, order=None, flags=0, seqs=2):
        return lib.pa_decode_step_int4(out, F, key, F, F, F, F, F, 4, F, seqs, 32, 8, 128, 16, 10,
                                       0.1, part, ws, ws, ws, counters, maxp, order, flags, None)

    assert step(out=None) == bad and step(key=None) == bad and step(part=100) == bad
    assert step(ws=None) == bad and step(counters=None) == bad and step(flags=2) == bad
    assert step(order=F, part=0) == bad
    assert step(order=F, seqs=300, maxp=300) == shape
    assert step(seqs=0) == pa.PA_OK
    assert step(part=-1) == bad


def test_biased_host_checks(lib):
    bad, shape = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED_SHAPE

    def step(cap=0.0, slopes=None, window=0, out=F, d=128, part=512):
        return lib.pa_decode_step_biased(out, F, None, None, None, F, F, F, 4, F, 2, 32, 8, d, 16,
                                         10, 0.1, cap, slopes, window, part, F, F, F, F, 4, None,
                                         0, None)

    def fill(cap=0.0, slopes=None, window=0, prefix=None, out=F, d=128, scale=0.1):
        return lib.pa_prefill_biased(out, F, F, F, F, 4, F, F, 8, 2, 16, 32, 8, d, 16, 10, scale,
                                     cap, slopes, window, prefix, None)

    for call in (step, fill):
        for cap in (-1.0, float("nan"), float("inf"), 3e38, 1e-40):
            assert call(cap=cap) == bad
        assert call(window=-1) == bad
        assert call(slopes=ctypes.c_void_p(0x10002)) == bad
        assert call(out=None) == bad
        assert call(d=96) == shape
    assert step(part=100) == bad
    assert fill(d=64) == shape and fill(scale=0.0) == bad
    assert fill(prefix=ctypes.c_void_p(0x10002)) == bad


def test_partition_size_of_a_4bit_cache():
    for ctx in ([1], [37, 1000], [131072] * 8, list(range(1, 2048, 7))):
        for ordered in (False, True):
            p = pa.splitk_partition_size(ctx, 32, 8, 128, "int4", num_sms=152, ordered=ordered)
            assert p >= 256 and p % 16 == 0


def test_binding_refuses_without_a_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        pa.pa_reshape_and_cache_int4(x, x, torch.zeros(3, 4, 1152, dtype=torch.uint8),
                                     torch.zeros(3, 4, 1152, dtype=torch.uint8),
                                     torch.zeros(2, dtype=torch.int64))


def test_prepared_calls_check_as_the_calls_do(lib):
    h = ctypes.c_void_p(123)
    bad, shape = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED_SHAPE

    def step(kind=4, part=512, cap=0.0, window=0, out=F):
        return lib.pa_prepare_decode_step(
            ctypes.byref(h), kind, out, F, None, None, None, F, F, None, None, F, 4, F, 2, 32, 8,
            128, 16, 10, 0.1, cap, None, window, part, F, F, F, F, 4, None, 0)

    assert step(kind=3) == bad and step(kind=-1) == bad and step(out=None) == bad
    assert h.value is None                          # an error leaves no object
    assert step(part=100) == bad and step(cap=30.0) == bad      # rules: bf16 only
    assert step(kind=1) == bad                      # INT8 needs scales
    assert step(kind=0, window=-1) == bad
    assert lib.pa_prepare_rope_reshape_and_cache(
        ctypes.byref(h), 0, None, None, 0, F, 1024, F, 1024, F, F, None, None, F, F, F, 100, 24,
        0, 3, 0, 8, 128, 16, 10) == shape
    assert lib.pa_prepare_prefill(ctypes.byref(h), F, F, F, F, F, 4, F, F, 8, 2, 16, 32, 8, 64,
                                  16, 10, 0.1, 0.0, None, 0, None) == shape
    assert lib.pa_prepare_prefill(None, F, F, F, F, F, 4, F, F, 8, 2, 16, 32, 8, 128, 16, 10,
                                  0.1, 0.0, None, 0, None) == bad
    assert lib.pa_run(None, None) == bad
    lib.pa_prepared_destroy(None)
