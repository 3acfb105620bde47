"""Selection from parts of the greatest length: sixteen blocks of logits, of which a
thread's maxima fill their room.  With more than 304 rows a row is one part as far as
it may be: 65,536 fp32 logits, 131,072 of 16 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_cache_283_gb300 import pa

from test_gpu_beam import Search, T, check_some

pytestmark = pytest.mark.gpu

MOST = {"fp32": 65536, "bf16": 131072, "fp16": 131072}


@pytest.mark.parametrize("dtype", sorted(T))
@pytest.mark.parametrize("more", [-1, 0, 1, 9])
def test_parts_of_the_greatest_length(dtype, more):
    """The finds of some searches in the sixteenth block and in what follows the part."""
    pa.pa_clear_device_error()
    most = MOST[dtype]
    vocab = most + more
    s = Search(most + more, 77, 4, 6, vocab, dtype)
    block = most // 16
    # the largest ones: the first and last logits of the last block, and the row's end
    at = [15 * block, 15 * block + 1, most - 2, vocab - 1, vocab - 2, 14 * block + 77]
    s.logits[12:16] = -1.0
    for i, e in enumerate(at):
        s.logits[12 + i % 4, e] = 5.0 + i
    s.logits[16:20, :15 * block] = -float("inf")           # nothing but the last block
    s.logits[20:24] = torch.linspace(-9, 9, vocab, device="cuda").to(T[dtype])
    got = s.call()
    check_some(s, got, np.array([0, 3, 4, 5, 30, 76]))
    assert (got[2][4] >= 15 * block).all()                 # (4: nothing else can be found)
    assert pa.pa_get_device_error() == 0
    # a bad logit in the last block, and in the part's last place
    s.logits[28, most - 2] = float("nan")
    s.logits[29, vocab - 1] = float("inf")
    got = s.call()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_LOGITS
    pa.pa_clear_device_error()
    check_some(s, got, np.array([6, 7, 8]))


def test_more_rows_than_ctas_at_once():
    """Two parts a row of a vocabulary above the bound, in several waves."""
    pa.pa_clear_device_error()
    s = Search(5, 80, 8, 8, 128256, "fp32", finished=0.1)
    check_some(s, s.call(in_place=False), np.array([0, 1, 40, 79]))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_hidden_by_the_lowest_number(dtype):
    """Rows masked with the type's lowest finite number, with fewer tokens left than are
    asked for: the masked ones follow, the lowest token first."""
    pa.pa_clear_device_error()
    s = Search(6, 77, 4, 6, 40001, dtype)
    low = torch.finfo(T[dtype]).min
    keep = s.logits[4:8, [3, 39999]].clone()
    s.logits[4:8] = low
    s.logits[4:8, [3, 39999]] = keep
    s.logits[8:12] = low
    s.scores[8:12] = -1.0
    got = s.call()
    check_some(s, got, np.array([0, 1, 2, 50]))
    assert sorted(set(got[2][1].tolist())) == [3, 39999]
    assert got[1][2].tolist() == [8] * 6 and got[2][2].tolist() == list(range(6))
    assert pa.pa_get_device_error() == 0
