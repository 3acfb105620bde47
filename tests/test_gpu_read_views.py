"""Reading a cache back into views of one tensor."""
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 2)])
def test_keys_and_values_may_alternate(d, hkv):
    """Rows [T, 2, Hkv, D], and heads side by side in wider rows; rows that meet are refused."""
    pa.pa_clear_device_error()
    g = torch.Generator(device="cuda").manual_seed(d)
    k, v = (torch.randn((9, hkv, 16, d), generator=g, device="cuda").bfloat16() for _ in "kv")
    tables = torch.tensor([[3, 8, 1], [0, 5, 7]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 37, 40], dtype=torch.int32, device="cuda")
    want = [p[tables.long()].transpose(2, 3).reshape(2, 48, hkv, d) for p in (k, v)]
    want = [torch.cat([w[0, :37], w[1, :3]]) for w in want]
    for shape in ((40, 2, hkv, d), (40, 3, hkv, d)):
        whole = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pa.pa_read_cache(whole[:, 0], whole[:, 1], k, v, tables, start, 37)
        assert torch.equal(whole[:, 0], want[0]) and torch.equal(whole[:, 1], want[1])
        whole[:] = 7.0
        pa.pa_read_cache(whole[:, 1], whole[:, 0], k, v, tables, start, 37)
        assert torch.equal(whole[:, 1], want[0]) and torch.equal(whole[:, 0], want[1])
        assert bool((whole[:, 2:] == 7.0).all())
        before = whole.clone()
        flat = whole.view(40, -1, d)
        with pytest.raises(pa.PAError):                      # a head of K is one of V
            pa.pa_read_cache(flat[:, :hkv], flat[:, hkv - 1:2 * hkv - 1], k, v, tables, start, 37)
        with pytest.raises(pa.PAError):                      # V's row is K's next one
            pa.pa_read_cache(whole[:39, 0], whole[1:, 0], k, v, tables[:1], start[:2], 37)
        assert torch.equal(whole, before)
    assert pa.pa_get_device_error() == 0
