"""Rotary append of prompts: the launch in which a thread takes several rows of a
token, for every cache type, against the same definitions as a decode step's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from int4_helpers import write
from oracle import rope as OR
from paged_kv_cache_283_gb300 import pa

from gpu_helpers import dev_bf16, host_bits
from test_gpu_rope_append import PLAIN, _inputs, _pools, _run

pytestmark = pytest.mark.gpu

# (a thread takes several rows from 77,825 (token, row, lane) triples on; D / 16
# lanes a row, and rows of 7, 8, 9 and 10: with every remainder by 3)


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("T,hq,hkv,d,rot,interleaved", [
    (1400, 5, 1, 128, 128, False), (1300, 4, 2, 128, 64, True), (2200, 5, 2, 64, 64, True),
    (2000, 4, 3, 64, 48, False)])
def test_rope_append_of_a_prompt(kind, T, hq, hkv, d, rot, interleaved):
    _run(T + d, kind, T, hq, hkv, d, rot, interleaved, strided=rot != d, pad=(3, 20, T - 1),
         gone=(5, 36))


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("hkv,d", [(4, 128), (7, 64)])
def test_rope_prompt_without_q(kind, hkv, d):
    # whole blocks in a row, and a block that the prompt fills in part
    T = 2500
    rng, qkv, _, k, v = _inputs(d, T, 0, hkv, d, True)
    pools = _pools(kind, 200, hkv, d, rng)
    before = [p.clone() for p in pools]
    slots = torch.arange(21, 21 + T, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    table = pa.rope_table(T, d, 10000.0)
    pa.pa_clear_device_error()
    pa.pa_rope_reshape_and_cache(None, None, k, v, pools[0], pools[1], slots, pos, table, False,
                                 *pools[2:])
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    cos, sin = (x.cpu().numpy() for x in table.split(d // 2, 1))
    rot = OR.rotate_fp32(qkv[:, :hkv], cos, sin, d, False)
    PLAIN[kind](dev_bf16(rot), v.contiguous(), *before, slots)
    torch.cuda.synchronize()
    for a, b in zip(pools, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("hkv,d", [(4, 128), (7, 64)])
def test_int4_write_of_a_prompt_bit_exact(hkv, d):
    # against the oracle's codes (the plain 4-bit write is the append's kernel); some
    # rows constant, or over the whole range of bf16
    T = 2500
    rng, qkv, _, k, v = _inputs(50 + d, T, 0, hkv, d, False)
    key, val = host_bits(k), host_bits(v)
    key[3] = 0x4040
    val[4, :, :64] = np.where(np.arange(64) == 7, 0x7F7F, 0xFF7F)
    key[5:90] = (key[5:90] & 0x807F) | 0x0080     # normal numbers of the least exponent
    pools = _pools("int4", 170, hkv, d, rng)
    slots = rng.choice(170 * 16, size=T, replace=False).astype(np.int64)
    slots[[5, 11]] = -1
    want = write(key, val, *(p.cpu().numpy() for p in pools), slots)
    pa.pa_reshape_and_cache_int4(dev_bf16(key), dev_bf16(val), *pools,
                                 torch.from_numpy(slots).cuda())
    for got, ref in zip(pools, want):
        assert np.array_equal(got.cpu().numpy(), ref)
