"""Positions of a cache read back (pa_read_cache) on the GPU, bit for bit against
the values that the caches' bytes stand for: every cache type, ranges that begin
and end inside blocks, strided rows, slots of another pool; the cache writes' own
inverse; and a quantised prompt's next chunk prefilled over its prefix read back."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8 as O8
from oracle import prefill as OP
from oracle import rope as OR
from oracle import search as OS
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import bf16_to_f64, dev_bf16, host_bits, v_pool_stored
from int4_helpers import pack, pool_values

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "int8", "fp8", "int4"]


def _dev(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


class Cache:
    """Pools of random contents, on the GPU, and the bf16 bits they stand for."""

    def __init__(self, seed, kind, nb, hkv, d):
        rng = np.random.default_rng(seed)
        self.kind, self.nb, self.hkv, self.d = kind, nb, hkv, d
        self.scales = (None, None)
        shape = (nb, hkv, 16, d)
        if kind == "bf16":
            bits = [normal_bf16(rng, shape) for _ in "kv"]
            self.pools = [dev_bf16(b) for b in bits]
        elif kind == "int4":
            self.pools, bits = [], []
            for is_v in (False, True):
                par = [OR.to_bf16_bits(x.astype(np.float32)) for x in (
                    rng.standard_normal((nb, hkv, 16, d // 64)) - 2,
                    rng.random((nb, hkv, 16, d // 64)))]
                pool = pack(rng.integers(0, 16, shape).astype(np.uint8), *par, is_v)
                self.pools.append(torch.from_numpy(pool).cuda())
                # scale * code is exact in fp32, the sum rounded once, then to bf16
                bits.append(OR.to_bf16_bits(pool_values(pool, d, is_v).astype(np.float32)))
        else:
            fp8 = kind == "fp8"
            self.pools, self.scales, bits = [], [], []
            for is_v in (False, True):
                codes = rng.integers(0, 256, shape).astype(np.uint8)
                if fp8:
                    codes[(codes & 127) == 127] = 8
                    x = O8.e4m3_decode(codes).astype(np.float32)
                else:
                    codes = np.where(codes == 128, 127, codes).astype(np.uint8).view(np.int8)
                    x = codes.astype(np.float32)
                sc = (rng.random((nb, hkv, 16)) * 0.1).astype(np.float32)
                bits.append(OR.to_bf16_bits(x * sc[..., None]))
                stored = v_pool_stored(codes, fp8) if is_v else codes
                self.pools.append(torch.from_numpy(np.ascontiguousarray(stored)).cuda())
                self.scales.append(torch.from_numpy(sc).cuda())
        self.bits = bits


def _ranges(seed, cache, first, counts):
    rng = np.random.default_rng(seed)
    nblk = [-(-(f + n) // 16) for f, n in zip(first, counts)]
    tables = np.full((len(first), max(1, *nblk) + 1), -1, dtype=np.int32)
    perm = rng.permutation(cache.nb)
    at = 0
    for b, k in enumerate(nblk):
        tables[b, :k] = perm[at:at + k]
        at += k
    start = np.concatenate([[0], np.cumsum(counts)])
    return tables, start


def _want(cache, tables, first, counts):
    return [OS.read_rows(b, tables, first, counts) for b in cache.bits]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_ranges(kind, d, hkv):
    pa.pa_clear_device_error()
    first = [0, 5, 16, 31, 0, 40, 15, 0]
    counts = [1, 11, 16, 2, 0, 100, 1, 33]
    cache = Cache(1, kind, 40, hkv, d)
    tables, start = _ranges(2, cache, first, counts)
    T = int(start[-1])
    ko, vo = (torch.full((T + 2, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pa.pa_read_cache(ko, vo, *cache.pools, _dev(tables, np.int32), _dev(start, np.int32), 100,
                     first_positions=_dev(first, np.int32), k_scales=cache.scales[0],
                     v_scales=cache.scales[1])
    for o, want in zip((ko, vo), _want(cache, tables, first, counts)):
        assert np.array_equal(host_bits(o[:T]), want)
        assert bool((o[T:] == 7.0).all())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_without_first(kind):
    pa.pa_clear_device_error()
    cache = Cache(3, kind, 30, 2, 64)
    counts = [65, 3, 130]
    tables, start = _ranges(4, cache, [0] * 3, counts)
    wide = torch.full((198, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    call = pa.ReadCache(wide[:, 1:3], wide[:, 4:6], *cache.pools, _dev(tables, np.int32),
                        _dev(start, np.int32), 130, k_scales=cache.scales[0],
                        v_scales=cache.scales[1])
    call()
    for at, want in zip((1, 4), _want(cache, tables, [0] * 3, counts)):
        assert np.array_equal(host_bits(wide[:, at:at + 2]), want)
    assert bool((wide[:, [0, 3]] == 7.0).all())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_into_slots(kind, d):
    pa.pa_clear_device_error()
    cache = Cache(5, kind, 40, 3, d)
    first, counts = [7, 0, 30], [50, 17, 3]
    tables, start = _ranges(6, cache, first, counts)
    slots = np.random.default_rng(7).permutation(12 * 16)[:70].astype(np.int64)
    slots[[3, 60]] = -1
    ko, vo = (torch.full((12, 3, 16, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pa.pa_read_cache(ko, vo, *cache.pools, _dev(tables, np.int32), _dev(start, np.int32), 50,
                     first_positions=_dev(first, np.int32), k_scales=cache.scales[0],
                     v_scales=cache.scales[1], slot_mapping=_dev(slots, np.int64))
    seven = OR.to_bf16_bits(np.array([7.0], dtype=np.float32))[0]
    for o, rows in zip((ko, vo), _want(cache, tables, first, counts)):
        want = np.full((12, 3, 16, d), seven, dtype=np.uint16)
        for r, s in enumerate(slots.tolist()):
            if s >= 0:
                want[s // 16, :, s % 16] = rows[r]
        assert np.array_equal(host_bits(o), want)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_bf16_writes_read_back(d):
    pa.pa_clear_device_error()
    rng = np.random.default_rng(8)
    key, value = (dev_bf16(normal_bf16(rng, (90, 2, d))) for _ in "kv")
    kc, vc = (torch.zeros((8, 2, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = np.array([[5, 1, 7, 0, 2, 6]], dtype=np.int32)
    pos = np.arange(90)
    pa.pa_reshape_and_cache(key, value, kc, vc, _dev(table[0, pos // 16] * 16 + pos % 16, np.int64))
    ko, vo = torch.zeros_like(key), torch.zeros_like(value)
    pa.pa_read_cache(ko, vo, kc, vc, _dev(table, np.int32), _dev([0, 90], np.int32), 90)
    assert torch.equal(ko, key) and torch.equal(vo, value)
    assert pa.pa_get_device_error() == 0


def test_bad_values_are_reported():
    cache = Cache(9, "int8", 20, 2, 64)
    first, counts = [3, 0], [40, 20]
    tables, start = _ranges(10, cache, first, counts)
    want = _want(cache, tables, first, counts)

    def call(first=first, start=start, tables=tables, rows=40, slots=None):
        pa.pa_clear_device_error()
        shape = (60, 2, 64) if slots is None else (4, 2, 16, 64)
        ko, vo = (torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        pa.pa_read_cache(ko, vo, *cache.pools, _dev(tables, np.int32), _dev(start, np.int32),
                         rows, first_positions=_dev(first, np.int32), k_scales=cache.scales[0],
                         v_scales=cache.scales[1], slot_mapping=_dev(slots, np.int64))
        err = pa.pa_get_device_error()
        pa.pa_clear_device_error()
        return err, ko, vo

    capacity = tables.shape[1] * 16
    for kw in (dict(first=[-1, 0]), dict(first=[capacity - 39, 0]), dict(first=[2 ** 31 - 1, 0]),
               dict(start=[0, 61, 60])):
        err, ko, vo = call(**kw)
        assert err == pa.PA_DEVERR_CONTEXT_LEN, kw
        assert bool((ko[:40] == 7.0).all())
        if "first" in kw:
            assert np.array_equal(host_bits(ko[40:]), want[0][40:])
    err, ko, vo = call(rows=30)                          # rows past the bound are left
    assert err == pa.PA_DEVERR_CONTEXT_LEN
    assert np.array_equal(host_bits(vo[:30]), want[1][:30]) and bool((vo[30:40] == 7.0).all())
    bad = tables.copy()
    bad[1, 0] = cache.nb
    err, ko, vo = call(tables=bad)
    assert err == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(host_bits(ko[:40]), want[0][:40])
    slots = np.arange(60, dtype=np.int64)
    slots[5], slots[59] = 64, -1
    err, ko, vo = call(slots=slots)
    assert err == pa.PA_DEVERR_SLOT
    got = host_bits(ko).transpose(0, 2, 1, 3).reshape(64, 2, 64)
    assert np.array_equal(got[:5], want[0][:5]) and np.array_equal(got[6:59], want[0][6:59])


def test_refusals():
    cache = Cache(11, "fp8", 20, 2, 64)
    tables, start = _ranges(12, cache, [0], [40])
    t, s = _dev(tables, np.int32), _dev(start, np.int32)
    ko, vo = (torch.zeros((40, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kw = dict(k_scales=cache.scales[0], v_scales=cache.scales[1])
    for args, more in (((ko, vo[:3]), kw), ((ko, vo), {}), ((ko[:, :1], vo[:, :1]), kw),
                       ((ko, vo), dict(kw, first_positions=t)),
                       ((ko, vo), dict(kw, slot_mapping=_dev(np.arange(40), np.int64))),
                       ((ko.cpu(), vo), kw)):
        with pytest.raises(ValueError):
            pa.pa_read_cache(*args, *cache.pools, t, s, 40, **more)
    with pytest.raises(TypeError):
        pa.pa_read_cache(ko.float(), vo.float(), *cache.pools, t, s, 40, **kw)
    plain = Cache(13, "bf16", 20, 2, 64)
    with pytest.raises(ValueError):
        pa.pa_read_cache(ko, vo, *plain.pools, t, s, 40, **kw)
    with pytest.raises(pa.PAError):                      # into the pools that are read
        pa.pa_read_cache(*plain.pools, *plain.pools, t, s, 40,
                         slot_mapping=_dev(np.arange(40), np.int64))


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4"])
def test_quantised_prompt_prefilled_in_chunks(kind):
    """A prompt's first chunk lies in a quantised cache: it is read back into a bf16
    cache's blocks, the second chunk's K and V are written behind it, and the second
    chunk attends to all of it."""
    pa.pa_clear_device_error()
    hq, hkv, d = 8, 2, 128
    cache = Cache(14, kind, 40, hkv, d)
    prior, new = [37, 160, 5], [20, 33, 64]
    tables, start = _ranges(15, cache, [0] * 3, prior)
    ctx = [p + n for p, n in zip(prior, new)]
    alloc = pa.BlockAllocator(64, 16)
    for b, c in enumerate(ctx):
        alloc.add_seq(b)
        alloc.reserve(b, c)
    bt, lens = alloc.block_tables([0, 1, 2], 16)
    where = [bt[b, np.arange(c) // 16] * 16 + np.arange(c) % 16 for b, c in enumerate(ctx)]
    old = np.concatenate([w[:p] for w, p in zip(where, prior)])
    kc, vc = (torch.full((64, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in "kv")
    pa.pa_read_cache(kc, vc, *cache.pools, _dev(tables, np.int32), _dev(start, np.int32), 160,
                     k_scales=cache.scales[0], v_scales=cache.scales[1],
                     slot_mapping=_dev(old, np.int64))
    rng = np.random.default_rng(16)
    key, value = normal_bf16(rng, (sum(new), hkv, d)), normal_bf16(rng, (sum(new), hkv, d))
    q = normal_bf16(rng, (sum(new), hq, d))
    fresh = np.concatenate([w[p:] for w, p in zip(where, prior)])
    pa.pa_reshape_and_cache(dev_bf16(key), dev_bf16(value), kc, vc, _dev(fresh, np.int64))
    out = torch.zeros_like(dev_bf16(q))
    at = np.concatenate([[0], np.cumsum(new)])
    pa.pa_prefill(out, dev_bf16(q), kc, vc, _dev(bt, np.int32), _dev(lens, np.int32),
                  _dev(at, np.int32), 64, d ** -0.5)
    pools = []
    for bits, rows in zip(cache.bits, (key, value)):
        pool = np.zeros((64, hkv, 16, d))
        read = bf16_bits_to_f64(OS.read_rows(bits, tables, [0] * 3, prior))
        pool[old // 16, :, old % 16] = read
        pool[fresh // 16, :, fresh % 16] = bf16_bits_to_f64(rows)
        pools.append(pool)
    ref = OP.prefill(bf16_bits_to_f64(q), *pools, bt, lens, new, d ** -0.5, 16)
    # The caches' values reach 12.7 and the outputs 8 to 16, where half a bf16 step is
    # 2^-5, more than the absolute gate of outputs near 1 allows.  So by the roundings: the
    # output's, 2^-8 of itself; the weights' to two bf16 parts, 2^-16, and what the scores'
    # accumulation moves them by, 2 D 2^-23 scale |q| |K|; over 224 keys, 224 2^-23.
    size = [np.linalg.norm(x, axis=-1).max() for x in (bf16_bits_to_f64(q), pools[0])]
    moved = 2.0 ** -16 + 2 * d * 2.0 ** -23 * d ** -0.5 * size[0] * size[1] + 288 * 2.0 ** -23
    err = np.abs(bf16_to_f64(out) - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + moved * np.abs(pools[1]).max())
    assert pa.pa_get_device_error() == 0
