"""4-bit KV cache on the GPU: the cache write bit-exact against the oracle, and
the decode (whole, split-K + merge, fused step) against the oracle's attention
over the values the pool stands for."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from int4_helpers import pack, pool_values, write
from oracle import int4 as O4
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import bf16_to_f64, dev_bf16

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _case(seed, ctx, hq, hkv, d, spread=1.0, shift=0.0):
    """Tables, quantised pools (bytes) and q of contexts `ctx`."""
    rng = np.random.default_rng(seed)
    ctx = np.asarray(ctx, dtype=np.int32)
    nblk = -(-ctx // 16)
    nb = int(nblk.sum()) + 3
    perm = rng.permutation(nb)
    tables = np.full((len(ctx), max(1, int(nblk.max()))), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(nblk.tolist()):
        tables[b, :k] = perm[at:at + k]
        at += k
    pools = []
    for is_v in (False, True):
        x = normal_bf16(rng, (nb, hkv, 16, d))
        if spread != 1.0 or shift:
            f = torch.from_numpy(bf16_bits_to_f64(x)) * spread + shift
            x = f.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
        pools.append(pack(*O4.quantize(x), is_v))
    return rng, ctx, tables, pools, normal_bf16(rng, (len(ctx), hq, d))


def _ref(case, scale, ctx=None):
    _, c, tables, pools, q = case
    d = q.shape[2]
    K, V = pool_values(pools[0], d, False), pool_values(pools[1], d, True)
    return O4.decode(bf16_bits_to_f64(q), K, V, tables, c if ctx is None else ctx, scale), V


def _gate(out, ref, V, what):
    """The output's bf16 rounding (half a step: 2^-8 of it); the weights' f16
    rounding (2^-11 of each term, whose part beside the offset is at most the
    spread of V); scores to about 2^-13: sums of 128 products in fp32 and the
    exponential's 2^-22, against values of up to |V|."""
    got = bf16_to_f64(out)
    V = V[np.isfinite(V)]
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * (V.max() - V.min()) + 2.0 ** -13 * np.abs(V).max()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: off by up to {np.abs(got - ref).max():.3e}"


def _all_ways(case, scale, parts=(512,), what=""):
    rng, ctx, tables, pools, q = case
    ref, V = _ref(case, scale)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    t, c, dq = _dev(tables, np.int32), _dev(ctx, np.int32), dev_bf16(q)
    pa.pa_clear_device_error()
    out = torch.full_like(dq, float("nan"))
    pa.pa_decode_int4(out, dq, dk, dv, t, c, scale)
    _gate(out, ref, V, what + " whole")
    B, hq, d = q.shape
    for part in parts:
        ws = pa.splitk_workspace(B, hq, d, int(ctx.max()), part)
        for w in ws:
            w.fill_(float("nan"))
        pa.pa_decode_splitk_int4(*ws, dq, dk, dv, t, c, scale, part)
        out.fill_(float("nan"))
        pa.pa_splitk_reduce(out, *ws, c, part)
        _gate(out, ref, V, f"{what} split {part}")
        counters = pa.step_counters(B, dk.shape[1])
        for early in (False, True):
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            pa.pa_decode_step(out, dq, dk, dv, t, c, scale, partition_size=part, workspace=ws,
                              counters=counters, early_read=early)
            _gate(out, ref, V, f"{what} step {part}")
        assert not counters.any()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d", [128, 64])
def test_int4_cache_write_bit_exact(d):
    rng = np.random.default_rng(d)
    nb, hkv, T = 9, 4, 45
    key, val = normal_bf16(rng, (T, hkv, d)), normal_bf16(rng, (T, hkv, d))
    key[3] = 0x4040                               # a constant row: scale 0
    val[4, :, :64] = np.where(np.arange(64) == 7, 0x7F7F, 0xFF7F)   # the whole range of bf16
    pools = [rng.integers(0, 256, (nb, hkv, 9 * d)).astype(np.uint8) for _ in "kv"]
    slots = rng.choice(nb * 16, size=T, replace=False).astype(np.int64)
    slots[[5, 11]] = -1
    want = write(key, val, *pools, slots)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    pa.pa_clear_device_error()
    pa.pa_reshape_and_cache_int4(dev_bf16(key), dev_bf16(val), dk, dv, _dev(slots, np.int64))
    assert pa.pa_get_device_error() == 0
    assert np.array_equal(dk.cpu().numpy(), want[0])
    assert np.array_equal(dv.cpu().numpy(), want[1])


@pytest.mark.parametrize("hq,hkv", [(4, 2), (32, 8), (8, 1)])
@pytest.mark.parametrize("d", [128, 64])
def test_int4_decode(hq, hkv, d):
    case = _case(hq + d, [1, 0, 15, 16, 17, 31, 32, 33, 500, 1023], hq, hkv, d)
    _all_ways(case, d ** -0.5, (16, 48, 256, 512), f"hq={hq} hkv={hkv} d={d}")


@pytest.mark.parametrize("ctx,hq,hkv,d", [
    ([9000, 4096, 4097, 63, 0, 1], 8, 2, 128), ([5000, 8191, 7], 4, 2, 128),
    ([20000, 64, 65], 8, 1, 128), ([33] * 300, 4, 1, 64), ([9000, 4160, 0], 4, 2, 64)])
def test_int4_decode_long_partitions(ctx, hq, hkv, d):
    # (partitions of 4096 tokens on take 64 at a time)
    _all_ways(_case(len(ctx), ctx, hq, hkv, d), 0.088, (1024, 4096, 8192), f"{len(ctx)} sequences")


def test_int4_decode_more_than_sixteen_partitions():
    _all_ways(_case(3, [1700, 40, 0], 8, 2, 128), 0.088, (64, 96), "many partitions")


@pytest.mark.parametrize("spread,shift", [(100.0, 0.0), (1e-3, 0.0), (1.0, 50.0), (1e-20, 0.0)])
def test_int4_decode_of_other_ranges(spread, shift):
    case = _case(4, [70, 300], 8, 2, 128, spread, shift)
    _all_ways(case, 0.088 / spread if spread > 1 else 0.088, (64,), f"{spread} {shift}")


def test_int4_scales_that_grow_along_the_context():
    # later tokens' V scales far above the first ones': the weights' bound moves
    rng, ctx, tables, pools, q = _case(5, [200], 8, 2, 128)
    par = pools[1][:, :, 8 * 128:].copy().view(np.uint16).reshape(pools[1].shape[0], 2, 16, 2, 2)
    for j in range(200):
        blk = tables[0, j // 16]
        par[blk, :, j % 16, :, 1] = np.uint16((127 - 20 + j // 10) << 7)
    pools[1][:, :, 8 * 128:] = par.view(np.uint8).reshape(pools[1].shape[0], 2, 128)
    _all_ways((rng, ctx, tables, pools, q), 0.088, (64, 512), "growing scales")


def test_int4_garbage_past_the_context():
    # codes of any kind, offsets and scales NaN and infinite, in the hidden slots
    case = _case(6, [3, 21, 40, 17], 8, 2, 128)
    rng, ctx, tables, pools, q = case
    ref, V = _ref(case, 0.1)
    for p in pools:
        par = p[:, :, 1024:].view(np.uint16).reshape(p.shape[0], 2, 16, 2, 2)
        for b, n in enumerate(ctx):
            if n % 16:
                par[tables[b, n // 16], :, n % 16:] = rng.choice(
                    [0x7FC0, 0x7F80, 0xFF80], par[tables[b, n // 16], :, n % 16:].shape)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    out = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_int4(out, dev_bf16(q), dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), 0.1)
    _gate(out, ref, V, "garbage past the context")


def test_int4_bad_block_ids_and_lengths():
    rng, ctx, tables, pools, q = _case(7, [100, 60], 8, 2, 128)
    tables[0, 2] = 10 ** 6
    tables[1, 1] = -5
    good = tables.copy()
    good[0, 2] = good[1, 1] = 0                    # a bad id reads block 0
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    out, want = (torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    pa.pa_clear_device_error()
    pa.pa_decode_int4(want, dev_bf16(q), dk, dv, _dev(good, np.int32), _dev(ctx, np.int32), 0.1)
    assert pa.pa_get_device_error() == 0
    pa.pa_decode_int4(out, dev_bf16(q), dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), 0.1)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_BLOCK_ID
    assert torch.equal(out, want)
    pa.pa_clear_device_error()
    pa.pa_decode_int4(out, dev_bf16(q), dk, dv, _dev(good, np.int32),
                      _dev([5000, -1], np.int32), 0.1)
    assert pa.pa_get_device_error() & pa.PA_DEVERR_CONTEXT_LEN
    pa.pa_clear_device_error()


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("part", [0, 16, 48, 256, 4096])
def test_int4_step_writes_and_attends(d, part):
    rng, ctx, tables, pools, q = _case(8 + d, [1, 16, 17, 33, 400], 8, 2, d)
    B = len(ctx)
    key, val = normal_bf16(rng, (B, 2, d)), normal_bf16(rng, (B, 2, d))
    slots = np.array([tables[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(ctx)])
    want = write(key, val, *pools, slots)
    ref, V = _ref((rng, ctx, tables, want, q), 0.1)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    out = torch.empty(B, 8, d, dtype=torch.bfloat16, device="cuda")
    pa.pa_clear_device_error()
    kw = {}
    if part:
        kw = dict(workspace=pa.splitk_workspace(B, 8, d, 400, part),
                  counters=pa.step_counters(B, 2))
    pa.pa_decode_step(out, dev_bf16(q), dk, dv, _dev(tables, np.int32), _dev(ctx, np.int32), 0.1,
                      dev_bf16(key), dev_bf16(val), _dev(slots, np.int64), part, **kw)
    assert pa.pa_get_device_error() == 0
    assert np.array_equal(dk.cpu().numpy(), want[0])
    assert np.array_equal(dv.cpu().numpy(), want[1])
    _gate(out, ref, V, f"step d={d} part={part}")


def test_int4_decode_step_handle_plans_and_replays():
    ctx = [5, 300, 1000, 64, 2000, 129]
    rng, ctx, tables, pools, q = _case(9, ctx, 32, 8, 128)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    dq, c = dev_bf16(q), _dev(ctx, np.int32)
    out = torch.empty_like(dq)
    step = pa.DecodeStep(None, None, dk, dv, None, dq, _dev(tables, np.int32), c, out, 0.088,
                         partition_size=None, host_context_lens=ctx)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
    for less in (0, 3):                         # lengths change between replays
        now = np.maximum(ctx - less, 0)
        c.copy_(torch.from_numpy(now.astype(np.int32)))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, V = _ref((rng, ctx, tables, pools, q), 0.088, now)
        _gate(out, ref, V, f"replay {less}")


def test_int4_handle_made_on_one_stream_and_run_on_another():
    # its counters are zeros before the first call, whatever the stream that makes
    # it is doing
    rng, ctx, tables, pools, q = _case(16, [5000, 6000, 17000], 32, 8, 64)
    dk, dv = (torch.from_numpy(p).cuda() for p in pools)
    dq, t, c = dev_bf16(q), _dev(tables, np.int32), _dev(ctx, np.int32)
    ref, V = _ref((rng, ctx, tables, pools, q), 0.125)
    out = torch.empty(3, 32, 64, dtype=torch.bfloat16, device="cuda")
    other = torch.cuda.Stream()
    for ps in (None, 2048):
        out.fill_(float("nan"))
        dirty = torch.full((24,), -1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        del dirty                               # (the handle's counters may take its place)
        work = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            work = work @ work * 1e-2
        step = pa.DecodeStep(None, None, dk, dv, None, dq, t, c, out, 0.125, partition_size=ps,
                             host_context_lens=ctx, stream=other)
        step()
        other.synchronize()
        _gate(out, ref, V, f"partition {ps}")
        torch.cuda.synchronize()


def test_int4_blocks_copy_as_bf16():
    # pa_copy_blocks on a 4-bit pool seen as [NB, 1, 1, bytes / 2] bf16
    rng = np.random.default_rng(10)
    pools = [torch.from_numpy(rng.integers(0, 256, (6, 3, 9 * 64)).astype(np.uint8)).cuda()
             for _ in "kv"]
    want = [p.clone() for p in pools]
    for w in want:
        w[4], w[2] = w[1], w[0]
    views = [[p.view(torch.bfloat16).view(6, 1, 1, -1)] for p in pools]
    pa.pa_copy_blocks(*views, torch.tensor([[1, 4], [0, 2]], device="cuda"))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_int4_far_offsets():
    # the last block of a pool of more than 2^32 bytes
    nb, hkv, d = 470000, 8, 128
    pools = [pa.int4_pool(nb, hkv, d) for _ in "kv"]
    assert pools[0].numel() > 1 << 32
    rng = np.random.default_rng(11)
    key, val = normal_bf16(rng, (16, hkv, d)), normal_bf16(rng, (16, hkv, d))
    slots = torch.arange((nb - 1) * 16, nb * 16, device="cuda")
    pa.pa_reshape_and_cache_int4(dev_bf16(key), dev_bf16(val), *pools, slots)
    q = normal_bf16(rng, (1, 32, d))
    out = torch.empty(1, 32, d, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_int4(out, dev_bf16(q), *pools, _dev([[nb - 1]], np.int32), _dev([16], np.int32),
                      0.1)
    K, V = (O4.values(*O4.quantize(x)).transpose(1, 0, 2)[None] for x in (key, val))
    ref = O4.decode(bf16_bits_to_f64(q), K, V, np.array([[0]]), [16], 0.1)
    _gate(out, ref, V, "far offsets")


def test_int4_binding_refusals():
    pool = pa.int4_pool(3, 2, 128)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    t, c = _dev([[0], [1]], np.int32), _dev([3, 4], np.int32)
    ok = dict(out=torch.empty_like(q), q=q, k_cache=pool, v_cache=pool.clone(), block_tables=t,
              context_lens=c, scale=0.1)
    for bad in (dict(v_cache=pa.int4_pool(3, 2, 64)), dict(k_cache=pool[:, :, :100].contiguous()),
                dict(k_cache=pool[:, :1]), dict(context_lens=c[:1]), dict(out=q[:1]),
                dict(block_tables=t.cpu())):
        with pytest.raises(ValueError):
            pa.pa_decode_int4(**{**ok, **bad})
    with pytest.raises(ValueError):
        pa.pa_decode_step(**ok, softcap=30.0)       # rules need a bf16 cache
    with pytest.raises(ValueError):                 # no workspace
        pa.pa_decode_step(**ok, partition_size=256)
    with pytest.raises(ValueError):
        pa.pa_decode_step(**ok, k_scales=torch.zeros(3, 2, 16, device="cuda"))
    with pytest.raises(ValueError):
        pa.DecodeStep(None, None, pool, pool.clone(), None, q, t, c, torch.empty_like(q), 0.1,
                      fused=False)
