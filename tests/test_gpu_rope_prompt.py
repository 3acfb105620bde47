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


def _border_rows(rng, T, hkv, d, kind):
    """Rows whose quotients lie on the borders between two codes, or next to them: bf16
    values that are halves of the code's steps times a power of two."""
    if kind == "int4":      # a range of 15 steps from its least value
        x = rng.integers(0, 31, (T, hkv, d)) / 2.0
        x[..., 0::64], x[..., 1::64] = 0, 15
        x -= rng.choice([0.0, 7.5, 15.0], (T, hkv, 1))
    elif kind == "int8":    # max 127, 63.5 or 72, 104, ...: some with inexact quotients
        top = rng.choice([127, 63.5, 72, 104, 71.5, 119.5], (T, hkv, 1))
        x = np.minimum(rng.integers(-254, 255, (T, hkv, d)) / 2.0, top)
        x = np.maximum(x, -top)
        x[..., :1], x[..., 1:2] = top, top / 2
    else:                   # E4M3's 3 bits of mantissa, and halves of its last
        top = rng.choice([448, 224, 240, 416, 390], (T, hkv, 1))
        x = rng.integers(16, 32, (T, hkv, d)) * 2.0 ** rng.integers(-16, 4, (T, hkv, d))
        x = np.minimum(x, top) * rng.choice([-1, 1], (T, hkv, d))
        x[..., :1] = top
    return OR.to_bf16_bits((x * 2.0 ** rng.integers(-9, 10, (T, hkv, 1))).astype(np.float32))


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("T,hkv,d", [(60, 2, 128), (60, 2, 64), (2500, 4, 128), (2500, 7, 64)])
def test_codes_of_rows_at_the_borders(kind, T, hkv, d):
    # (position 0 turns nothing)
    rng = np.random.default_rng(T + d)
    key, val = (_border_rows(rng, T, hkv, d, kind) for _ in "kv")
    pools = _pools(kind, T // 16 + 5, hkv, d, rng)
    before = [p.clone() for p in pools]
    slots = rng.permutation((T // 16 + 5) * 16)[:T].astype(np.int64)
    pa.pa_rope_reshape_and_cache(None, None, dev_bf16(key), dev_bf16(val), pools[0], pools[1],
                                 torch.from_numpy(slots).cuda(),
                                 torch.zeros(T, dtype=torch.int32, device="cuda"),
                                 pa.rope_table(4, d), False, *pools[2:])
    torch.cuda.synchronize()
    if kind == "int4":
        want = write(key, val, *(p.cpu().numpy() for p in before), slots)
        want = [torch.from_numpy(w).cuda() for w in want]
    else:
        PLAIN[kind](dev_bf16(key), dev_bf16(val), *before, torch.from_numpy(slots).cuda())
        want = before
    for a, b in zip(pools, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("d", [128, 64])
def test_the_fused_step_writes_the_codes_of_the_append(d):
    # 4-bit rows at the borders, and over the whole range of bf16, by either call
    B, hkv = 96, 2
    rng = np.random.default_rng(90 + d)
    key, val = (_border_rows(rng, B, hkv, d, "int4") for _ in "kv")
    val[4, :, :64] = np.where(np.arange(64) == 7, 0x7F7F, 0xFF7F)
    key[5:30] = (key[5:30] & 0x807F) | 0x0080
    key[7] = 0x4040
    k, v = dev_bf16(key), dev_bf16(val)
    pools = _pools("int4", B, hkv, d, rng)
    want = [p.clone() for p in pools]
    slots = torch.arange(B, device="cuda") * 16
    pa.pa_reshape_and_cache_int4(k, v, *want, slots)
    q = torch.zeros(B, 4, d, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_step(torch.empty_like(q), q, *pools, slots[:, None].int() // 16,
                      torch.ones(B, dtype=torch.int32, device="cuda"), 0.1, k, v, slots, 0)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for a, b in zip(pools, want):
        assert torch.equal(a, b)
