"""Every device input of a call may be what the launch just before it on the stream
writes.  The library's kernels may be scheduled before that launch is complete, so
each input is here copied into place by pa_copy_blocks, as the last of many blocks,
right before the call that reads it; until then it holds other valid values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

pytestmark = pytest.mark.gpu

BLOCK = 1 << 20         # bytes of a block: one CTA takes some 50 us to copy it


class Late:
    """Tensors that pa_copy_blocks brings into place, each at the end of a long block."""

    def __init__(self):
        self.pool, self.v = (torch.zeros(8, 1, 1, BLOCK // 2, dtype=torch.bfloat16,
                                         device="cuda") for _ in "kv")
        self.items = []

    def _view(self, block, like):
        n = like.numel() * like.element_size()
        end = (block + 1) * BLOCK
        raw = self.pool.view(-1).view(torch.uint8)[end - -(-n // 16) * 16:]
        return raw[:n].view(like.dtype).view(like.shape)

    def put(self, now, before):
        """A tensor that holds `before`, and `now` once run()'s copies are complete."""
        at = 2 * len(self.items)
        self._view(at, now).copy_(now)
        self.items.append((self._view(at + 1, now), before))
        return self.items[-1][0]

    def run(self):
        for x, before in self.items:
            x.copy_(before)
        pairs = torch.tensor([(2 * i, 2 * i + 1) for i in range(len(self.items))], device="cuda")
        torch.cuda.synchronize()
        pa.pa_copy_blocks([self.pool], [self.v], pairs)


def _normal(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def _check(call, outs, late, inputs):
    """call(inputs) -> None writes outs; the same with late inputs as with ready ones."""
    pa.pa_clear_device_error()
    keep = [o.clone() for o in outs]
    call(**inputs)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for name, (now, before) in late.items():
        stale = [o.clone() for o in want]
        for _ in range(3):
            for o, k in zip(outs, keep):
                o.copy_(k)
            box = Late()
            x = box.put(now, before)
            box.run()
            call(**{**inputs, name: x})
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"{name} was read early"
        for o, k in zip(outs, keep):        # (the other values give another result)
            o.copy_(k)
        call(**{**inputs, name: before})
        torch.cuda.synchronize()
        assert not all(torch.equal(o, w) for o, w in zip(outs, stale)), name
    assert pa.pa_get_device_error() == 0


def _pools(kind, nb, hkv, d):
    rows = [_normal(nb * 16, hkv, d) for _ in "kv"]
    slots = torch.arange(nb * 16, device="cuda")
    if kind == "int4":
        pools = [pa.int4_pool(nb, hkv, d) for _ in "kv"]
        pa.pa_reshape_and_cache_int4(*rows, *pools, slots)
        return pools, {}
    if kind == "bf16":
        pools = [torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        pa.pa_reshape_and_cache(*rows, *pools, slots)
        return pools, {}
    t = torch.int8 if kind == "int8" else torch.uint8
    pools = [torch.zeros(nb, hkv, 16, d, dtype=t, device="cuda") for _ in "kv"]
    scales = [torch.zeros(nb, hkv, 16, device="cuda") for _ in "kv"]
    write = pa.pa_reshape_and_cache_int8 if kind == "int8" else pa.pa_reshape_and_cache_fp8
    write(*rows, *pools, *scales, slots)
    return pools, dict(k_scales=scales[0], v_scales=scales[1])


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("kind,rule", [("bf16", False), ("bf16", True), ("int8", False),
                                       ("fp8", False), ("int4", False)])
def test_a_step_reads_after_the_launch_before(kind, rule, part, early):
    torch.manual_seed(1)
    B, hq, hkv, d, n = 3, 8, 2, 128, 200
    pools, scales = _pools(kind, 40, hkv, d)
    ctx = torch.tensor([n, 33, 100], dtype=torch.int32, device="cuda")
    tables = torch.randperm(39, device="cuda").to(torch.int32).view(3, 13)
    last = (ctx - 1).long()
    slots = tables.gather(1, (last // 16)[:, None])[:, 0].long() * 16 + last % 16
    out = torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
    kw = {}
    if part:
        kw = dict(workspace=pa.splitk_workspace(B, hq, d, 13 * 16, part),
                  counters=pa.step_counters(B, hkv))
    late = dict(q=(_normal(B, hq, d), _normal(B, hq, d)),
                key=(_normal(B, hkv, d), _normal(B, hkv, d)),
                value=(_normal(B, hkv, d), _normal(B, hkv, d)),
                slot_mapping=(slots, torch.full_like(slots, -1)))
    if rule:
        late["alibi_slopes"] = (torch.rand(hq, device="cuda"), torch.rand(hq, device="cuda"))
        kw["softcap"] = 20.0
    if not early:
        late["context_lens"] = (ctx, ctx - 7)
        late["block_tables"] = (tables, tables.flip(0).contiguous())
    inputs = dict(q=late["q"][0], key=late["key"][0], value=late["value"][0],
                  slot_mapping=slots, context_lens=ctx, block_tables=tables)
    if rule:
        inputs["alibi_slopes"] = late["alibi_slopes"][0]

    def call(**x):
        pa.pa_decode_step(out, k_cache=pools[0], v_cache=pools[1], scale=0.088,
                          partition_size=part, early_read=early, **x, **scales, **kw)

    outs = [out, *pools]
    pa.pa_clear_device_error()
    # lengths and tables of other values make the slot another sequence's place: no write
    write = {k: v for k, v in late.items() if k not in ("context_lens", "block_tables")}
    _check(call, outs, write, inputs)
    if not early:
        for k in ("key", "value", "slot_mapping"):
            inputs[k] = None
        _check(call, outs, {k: late[k] for k in ("context_lens", "block_tables")}, inputs)


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8", "int4"])
@pytest.mark.parametrize("tokens", [9, 1500])
def test_an_append_reads_after_the_launch_before(kind, tokens):
    torch.manual_seed(2)
    hq, hkv, d = 4, 2, 128
    pools, scales = _pools(kind, tokens // 16 + 2, hkv, d)
    table, other = pa.rope_table(64, d), pa.rope_table(64, d, base=100.0)
    slots = torch.randperm(pools[0].shape[0] * 16, device="cuda")[:tokens]
    pos = torch.randint(0, 64, (tokens,), dtype=torch.int32, device="cuda")
    late = dict(slot_mapping=(slots, slots.flip(0).contiguous()),
                positions=(pos, pos.flip(0).contiguous()), cos_sin=(table, other))
    if tokens < 100:
        for k, h in (("q", hq), ("key", hkv), ("value", hkv)):
            late[k] = (_normal(tokens, h, d), _normal(tokens, h, d))
    inputs = dict(q=_normal(tokens, hq, d), key=_normal(tokens, hkv, d),
                  value=_normal(tokens, hkv, d))
    inputs.update({k: v[0] for k, v in late.items()})
    q_out = torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    _check(lambda **x: pa.pa_rope_reshape_and_cache(q_out, k_cache=pools[0], v_cache=pools[1],
                                                    **x, **scales),
           [q_out, *pools, *scales.values()], late, inputs)


@pytest.mark.parametrize("rule", [False, True])
def test_a_prefill_reads_after_the_launch_before(rule):
    torch.manual_seed(3)
    hq, hkv, d = 8, 2, 128
    pools, _ = _pools("bf16", 40, hkv, d)
    ctx = torch.tensor([200, 40], dtype=torch.int32, device="cuda")
    tables = torch.randperm(40, device="cuda")[:26].to(torch.int32).view(2, 13)
    starts = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    out = torch.zeros(70, hq, d, dtype=torch.bfloat16, device="cuda")
    late = dict(q=(_normal(70, hq, d), _normal(70, hq, d)), context_lens=(ctx, ctx + 5),
                block_tables=(tables, tables.flip(0).contiguous()),
                query_start_loc=(starts, torch.tensor([0, 35, 70], dtype=torch.int32,
                                                      device="cuda")))
    kw = {}
    if rule:
        late["alibi_slopes"] = (torch.rand(hq, device="cuda"), torch.rand(hq, device="cuda"))
        late["prefix_lens"] = tuple(torch.tensor(x, dtype=torch.int32, device="cuda")
                                    for x in ([190, 39], [0, 3]))
        kw["softcap"] = 20.0
    inputs = {k: v[0] for k, v in late.items()}
    fn = pa.pa_prefill_biased if rule else pa.pa_prefill
    _check(lambda **x: fn(out, k_cache=pools[0], v_cache=pools[1], max_query_len=40, scale=0.088,
                          **x, **kw), [out], late, inputs)


@pytest.mark.parametrize("kind,rule", [("bf16", False), ("bf16", True), ("int8", False),
                                       ("fp8", False), ("int4", False)])
def test_early_reads_find_what_the_launch_before_the_last_wrote(kind, rule):
    """A step with early reads may read lengths, tables and pools while the launch just
    before it runs, which is itself such a step over other buffers; what the launch
    before that one writes is complete by then."""
    torch.manual_seed(4)
    B, hq, hkv, d = 2, 8, 2, 128
    (k0, v0), s0 = _pools(kind, 8, hkv, d)
    (k1, v1), s1 = _pools(kind, 26, hkv, d)
    ctx = torch.tensor([200, 100], dtype=torch.int32, device="cuda")
    tables = torch.randperm(26, device="cuda").to(torch.int32).view(2, 13)
    small = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    short = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    q = _normal(B, hq, d)
    kw = dict(scale=0.088, partition_size=0, early_read=True)
    if rule:
        kw["window"] = 150
    between, out = torch.empty_like(q), torch.empty_like(q)

    def call(context_lens, block_tables):
        pa.pa_decode_step(between, q, k0, v0, small, short, **kw, **s0)
        pa.pa_decode_step(out, q, k1, v1, block_tables, context_lens, **kw, **s1)

    _check(call, [between, out], dict(context_lens=(ctx, ctx - 60),
                                      block_tables=(tables, tables.flip(0).contiguous())),
           dict(context_lens=ctx, block_tables=tables))
