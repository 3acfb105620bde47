"""Rotary embedding + cache write on the GPU: q and the bf16 pools bit-exact
against the float32 definition and near the float64 rotation; the 4-bit pools
the bytes that the plain cache write gives for the rotated k, the INT8 and FP8
pools those of their rule; padding, bad
positions and slots, strided inputs, in-place q, graph replay."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import rope as OR
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits, v_pool_logical, v_pool_stored

pytestmark = pytest.mark.gpu

BASE, MAXPOS = 10000.0, 4096


def _pools(kind, nb, hkv, d, rng):
    if kind == "bf16":
        return [dev_bf16(normal_bf16(rng, (nb, hkv, 16, d))) for _ in "kv"]
    if kind == "int4":
        return [torch.from_numpy(rng.integers(0, 256, (nb, hkv, 9 * d)).astype(np.uint8)).cuda()
                for _ in "kv"]
    t = np.int8 if kind == "int8" else np.uint8
    return [torch.from_numpy(rng.integers(0, 100, (nb, hkv, 16, d)).astype(t)).cuda()
            for _ in "kv"] + [torch.from_numpy(rng.random((nb, hkv, 16)).astype(np.float32)).cuda()
                              for _ in "kv"]


def _write_1byte(key, value, kp, vp, ks, vs, slots):
    """INT8 / FP8 rows in float32: scale = amax * fl(1 / 127 or 1 / 448), codes by
    division, round half to even (E4M3: torch's conversion of the quotient)."""
    fp8 = kp.dtype == torch.uint8
    r = np.float32(1.0 / (448.0 if fp8 else 127.0))
    logical = [kp.cpu().numpy(), v_pool_logical(vp.cpu().numpy(), fp8)]
    for pool, sc, x in zip(logical, (ks, vs), (key, value)):
        f = x.float().cpu().numpy()
        scale = np.abs(f).max(-1) * r
        y = torch.from_numpy(f / np.where(scale > 0, scale, np.float32(1))[..., None])
        codes = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else \
            y.round().clamp(-127, 127).to(torch.int8)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                pool[s // 16, :, s % 16] = codes[t].numpy()
                sc[s // 16, :, s % 16] = torch.from_numpy(scale[t]).cuda()
    kp.copy_(torch.from_numpy(logical[0]))
    vp.copy_(torch.from_numpy(v_pool_stored(logical[1], fp8)))


PLAIN = {"bf16": pa.pa_reshape_and_cache, "int8": _write_1byte, "fp8": _write_1byte,
         "int4": pa.pa_reshape_and_cache_int4}


def _inputs(seed, T, hq, hkv, d, strided):
    rng = np.random.default_rng(seed)
    qkv = normal_bf16(rng, (T, hq + 2 * hkv, d))
    dev = dev_bf16(qkv)
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return rng, qkv, q, k, v


def _run(seed, kind, T, hq, hkv, d, rot, interleaved, strided, pad=(), gone=()):
    """pad: tokens with slot -1; gone: tokens with position -1."""
    rng, qkv, q, k, v = _inputs(seed, T, hq, hkv, d, strided)
    nb = T // 8 + 3
    pools = _pools(kind, nb, hkv, d, rng)
    before = [p.clone() for p in pools]
    slots = rng.choice(nb * 16, size=T, replace=False).astype(np.int64)
    pos = rng.integers(0, MAXPOS, T).astype(np.int32)
    pos[0] = MAXPOS - 1
    slots[list(pad)] = -1
    pos[list(gone)] = -1
    table = pa.rope_table(MAXPOS, rot, BASE)
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pa.pa_clear_device_error()
    pa.pa_rope_reshape_and_cache(q_out, q, k, v, pools[0], pools[1],
                                 torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(),
                                 table, interleaved, *pools[2:])
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    cos, sin = (x.cpu().numpy()[np.maximum(pos, 0)] for x in table.split(rot // 2, 1))
    want = OR.rotate_fp32(qkv[:, :hq + hkv], cos, sin, rot, interleaved)
    here = np.ones(T, bool)
    here[list(gone)] = False
    got = host_bits(q_out)
    assert np.array_equal(got[here], want[here, :hq])
    assert np.all(got[~here] == 0x40E0)             # 7.0: left as it was
    # near the float64 rotation: the bf16 rounding (half a step, 2^-8), and per
    # product and sum half a float32 step of values below |a| + |b|
    c64, s64 = OR.table(MAXPOS, rot, BASE)
    p0 = np.maximum(pos, 0)
    x = (qkv[:, :hq].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    ref = OR.rotate(x, c64[p0], s64[p0], rot, interleaved)
    size = np.abs(x).max()
    assert np.all(np.abs(bf16_to_f64(q_out) - ref)[here] <=
                  (2.0 ** -8 * np.abs(ref) + 2 * size * 4 * 2.0 ** -24)[here])
    # the pools: what the plain write of the rotated k and of v stores
    kept = here & (slots >= 0)
    s2 = np.where(kept, slots, -1)
    PLAIN[kind](dev_bf16(want[:, hq:]), v.contiguous(), *before,
                torch.from_numpy(s2).cuda())
    torch.cuda.synchronize()
    for a, b in zip(pools, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append(kind, d, rot, interleaved):
    _run(d + rot, kind, 37, 8, 2, d, rot, interleaved, strided=rot != d, pad=(3, 20),
         gone=(5, 36))


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("T,hq,hkv", [(1, 4, 2), (1, 1, 1), (64, 32, 8), (777, 6, 3)])
def test_rope_append_sizes(kind, T, hq, hkv):
    _run(T + hq, kind, T, hq, hkv, 128, 128, False, strided=True)


def test_rope_whole_prompt_blocks():
    # consecutive slots: tokens of one block written by one launch
    for kind in ("int8", "int4"):
        rng, qkv, q, k, v = _inputs(9, 64, 4, 2, 128, True)
        pools = _pools(kind, 6, 2, 128, rng)
        before = [p.clone() for p in pools]
        slots = torch.arange(16, 80, device="cuda")
        pos = torch.arange(64, dtype=torch.int32, device="cuda")
        table = pa.rope_table(64, 128, BASE)
        pa.pa_rope_reshape_and_cache(None, None, k, v, pools[0], pools[1], slots, pos, table,
                                     False, *pools[2:])
        cos, sin = (x.cpu().numpy() for x in table.split(64, 1))
        rot = OR.rotate_fp32(qkv[:, 4:6], cos, sin, 128, False)
        PLAIN[kind](dev_bf16(rot), v.contiguous(), *before, slots)
        torch.cuda.synchronize()
        for a, b in zip(pools, before):
            assert torch.equal(a, b)


def test_rope_bad_positions_and_slots():
    rng, qkv, q, k, v = _inputs(10, 6, 4, 2, 64, False)
    pools = _pools("bf16", 3, 2, 64, rng)
    before = [p.clone() for p in pools]
    slots = torch.tensor([0, 1, 2, 3, 48, 5], device="cuda")        # 48: past the pool
    pos = torch.tensor([0, 100, 2, 1 << 30, 4, -1], dtype=torch.int32, device="cuda")
    q_out = torch.zeros_like(q)
    pa.pa_clear_device_error()
    pa.pa_rope_reshape_and_cache(q_out, q, k, v, *pools, slots, pos,
                                 pa.rope_table(100, 64, BASE))
    assert pa.pa_get_device_error() == pa.PA_DEVERR_POSITION | pa.PA_DEVERR_SLOT
    pa.pa_clear_device_error()
    assert not q_out[[1, 3, 5]].any() and q_out[4].any()
    same = [torch.equal(pools[0][0, :, i], before[0][0, :, i]) for i in range(16)]
    assert same == [i not in (0, 2) for i in range(16)]
    assert torch.equal(pools[0][1:], before[0][1:])


def test_rope_in_place_and_handle_under_a_graph():
    rng, qkv, q, k, v = _inputs(11, 33, 8, 2, 128, False)
    pools = _pools("bf16", 6, 2, 128, rng)
    slots = torch.randperm(96, device="cuda")[:33]
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    table = pa.rope_table(128, 128, BASE)
    keep = q.clone()
    out = torch.empty_like(q)
    pa.pa_rope_reshape_and_cache(out, q, k, v, *pools, slots, pos, table)
    first = [p.clone() for p in pools]
    step = pa.RopeAppend(q, q, k, v, *pools, slots, pos, table)     # in place
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        assert torch.equal(q, out)
        with torch.cuda.graph(g, stream=s):
            step()
    for shift in (0, 5):
        q.copy_(keep)
        pos.copy_(torch.arange(33) + shift)
        for p in pools:
            p.zero_()
        g.replay()
        torch.cuda.synchronize()
        if shift == 0:
            assert torch.equal(q, out)
            blk, off = slots // 16, slots % 16
            assert torch.equal(pools[0][blk, :, off], first[0][blk, :, off])
    pa.pa_rope_reshape_and_cache(out, keep, k, v, *pools, slots, pos, table)
    torch.cuda.synchronize()
    assert torch.equal(q, out)


def test_rope_far_offsets():
    # a pool of more than 2^31 elements (2^32 bytes): the last block's offset does
    # not fit 32 bits
    nb, hkv, d = 140000, 8, 128
    pools = [torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    assert pools[0].numel() > 1 << 31
    rng, qkv, q, k, v = _inputs(12, 2, 8, hkv, d, False)
    slots = torch.tensor([nb * 16 - 1, 5], device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    pa.pa_rope_reshape_and_cache(torch.empty_like(q), q, k, v, *pools, slots, pos,
                                 pa.rope_table(8, 128, BASE))
    assert torch.equal(pools[0][nb - 1, :, 15], k[0]) and torch.equal(pools[1][0, :, 5], v[1])
    assert int(torch.count_nonzero(pools[0])) == int(torch.count_nonzero(k))


def test_rope_refusals():
    rng, qkv, q, k, v = _inputs(13, 4, 4, 2, 128, False)
    pools = _pools("bf16", 3, 2, 128, rng)
    slots = torch.arange(4, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = pa.rope_table(8, 128, BASE)
    ok = dict(q_out=torch.empty_like(q), q=q, key=k, value=v, k_cache=pools[0], v_cache=pools[1],
              slot_mapping=slots, positions=pos, cos_sin=table)
    for bad, err in [(dict(q=q.float()), TypeError), (dict(positions=pos.long()), TypeError),
                     (dict(key=k.transpose(1, 2)), ValueError), (dict(q_out=None), ValueError),
                     (dict(value=v[:, :1]), ValueError), (dict(slot_mapping=slots[:3]), ValueError),
                     (dict(cos_sin=table.cpu()), ValueError), (dict(key=k.cpu()), ValueError),
                     (dict(k_cache=pools[0][:, :1]), ValueError),
                     (dict(k_scales=torch.zeros(3, 2, 16, device="cuda")), ValueError),
                     (dict(cos_sin=table[:, :24].contiguous()), pa.PAError)]:
        with pytest.raises(err):
            pa.pa_rope_reshape_and_cache(**{**ok, **bad})
