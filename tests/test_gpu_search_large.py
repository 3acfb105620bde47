"""Selection and reordering where offsets pass 32 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

pytestmark = pytest.mark.gpu


def test_selection_of_the_largest_vocabulary():
    """2^27 tokens, 1024 parts a row; the last rows begin past 2^31 elements."""
    pa.pa_clear_device_error()
    vocab, beams, keep = 1 << 27, 18, 20
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.empty((beams, vocab + 3), dtype=torch.bfloat16, device="cuda")
    for row in wide:
        row.normal_(generator=g)
    wide[:, vocab:] = float("nan")
    logits = wide[:, :vocab]
    scores = -torch.rand(beams, generator=g, device="cuda")
    rng = np.random.default_rng(2)
    planted = {}                                 # above every other logit of its row
    for r in range(beams):
        for i, v in enumerate(rng.choice(vocab, 3, replace=False).tolist() + [vocab - 1 - r]):
            logits[r, v] = 8.0 + 0.25 * i
            planted[r, v] = 8.0 + 0.25 * i
    total = {}
    for r in range(beams):
        lse = torch.logsumexp(logits[r].double(), 0).item()
        for (row, v), x in planted.items():
            if row == r:
                total[row, v] = scores[r].double().item() + x - lse
    out = (torch.zeros((1, keep), device="cuda"),
           *(torch.zeros((1, keep), dtype=torch.int32, device="cuda") for _ in "pt"))
    ws = pa.beam_select_workspace(logits, beams, keep)
    for _ in range(2):
        pa.pa_beam_select(*out, logits, scores, beams, ws)
    got = [x.cpu().numpy()[0] for x in out]
    best = sorted(total.values(), reverse=True)[:keep]
    mine = [total[int(r), int(v)] for r, v in zip(got[1], got[2])]
    assert len(set(zip(got[1].tolist(), got[2].tolist()))) == keep
    # (a log-sum is off by less than 2e-5, a score by half a unit of fp32)
    assert np.abs(np.array(mine) - got[0]).max() < 2e-5 + 2.0 ** -24 * 16
    assert np.abs(np.array(mine) - np.array(best)).max() < 4e-5
    assert not ws[1].any() and pa.pa_get_device_error() == 0


@pytest.mark.parametrize("beams,row", [(16, 300_000_016), (9, 500_000_001)])
def test_reordering_of_many_beams(beams, row):
    pa.pa_clear_device_error()
    x = torch.zeros((beams, row), dtype=torch.uint8, device="cuda")
    want = torch.arange(beams * 40, device="cuda").view(beams, 40).to(torch.uint8)
    x[:, :20], x[:, -20:] = want[:, :20], want[:, 20:]
    x[:, row // 2] = want[:, 5]
    parents = np.random.default_rng(beams).permutation(beams)
    parents[2], parents[-1] = -1, 0
    at = np.where(parents < 0, np.arange(beams), parents).tolist()
    pa.pa_reorder_states(x, torch.tensor(parents, dtype=torch.int32, device="cuda"), beams)
    assert torch.equal(x[:, :20], want[at][:, :20]) and torch.equal(x[:, -20:], want[at][:, 20:])
    assert torch.equal(x[:, row // 2], want[at][:, 5])
    assert int(x[:, 20:row // 2].max()) == 0 and int(x[:, row // 2 + 1:-20].max()) == 0
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_reading_back_past_32_bits(kind):
    """Blocks at the end of pools of more than 2^31 elements, to rows more than 2^31 elements
    from the first one and to slots at the end of such a pool."""
    pa.pa_clear_device_error()
    hkv, d, n = 8, 128, 37
    nb = (1 << 31) // (hkv * 16 * d) + 7
    g = torch.Generator(device="cuda").manual_seed(3)
    if kind == "bf16":
        pools = [torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        kw = {}
    else:
        pools = [torch.zeros((nb, hkv, 16, d), dtype=torch.int8, device="cuda") for _ in "kv"]
        scales = [torch.zeros((nb, hkv, 16), device="cuda") for _ in "kv"]
        kw = dict(k_scales=scales[0], v_scales=scales[1])
    key, value = (torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16() for _ in "kv")
    table = torch.tensor([[nb - 1, nb - 3, nb - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = table[0].long()[pos // 16] * 16 + pos % 16
    small = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")   # the same, in 3 blocks
    small_slots = small[0].long()[pos // 16] * 16 + pos % 16
    few = [torch.zeros((3, *p.shape[1:]), dtype=p.dtype, device="cuda") for p in pools]
    if kind == "bf16":
        pa.pa_reshape_and_cache(key, value, *pools, slots)
        few_kw = {}
        pa.pa_reshape_and_cache(key, value, *few, small_slots)
    else:
        pa.pa_reshape_and_cache_int8(key, value, *pools, *scales, slots)
        few_kw = {k: torch.zeros((3, hkv, 16), device="cuda") for k in kw}
        pa.pa_reshape_and_cache_int8(key, value, *few, *few_kw.values(), small_slots)
    want = [torch.zeros((n, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pa.pa_read_cache(*want, *few, small, start, n, **few_kw)
    if kind == "bf16":
        assert torch.equal(want[0], key) and torch.equal(want[1], value)
    assert bool(want[0].any()) and bool(want[1].any())
    stride = (1 << 31) // (n - 2) // 8 * 8
    far = [torch.zeros(stride * (n - 1) + hkv * d, dtype=torch.bfloat16, device="cuda")
           .as_strided((n, hkv, d), (stride, d, 1)) for _ in "kv"]
    pa.pa_read_cache(*far, *pools, table, start, n, **kw)
    assert all(torch.equal(a, b) for a, b in zip(far, want))
    del far
    if kind == "bf16":                           # and into the slots of another such pool
        there = [torch.zeros_like(p) for p in pools]
        pa.pa_read_cache(*there, *pools, table, start, n, slot_mapping=slots)
        assert all(torch.equal(a[-3:], b[-3:]) for a, b in zip(there, pools))
        assert not any(bool(t[:-3].any()) for t in there)
    assert pa.pa_get_device_error() == 0
