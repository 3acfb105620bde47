"""Beam search's selection and the reordering of states on the GPU against the
float64 oracle, and a search run with them over the paged cache."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import search as OS
from paged_kv_cache_283_gb300 import pa

pytestmark = pytest.mark.gpu

# A total's error: the exponentials (2^-22 of each), the sums of at most 64 terms (2^-24
# each) under at most 16 changes of a thread's reference (2^-22 + 2^-24 each) and those of
# the threads, warps and parts move the log-sum by less than 1e-5 of 1; the total is
# rounded to fp32 (2^-24 of itself).
ATOL = 1e-5
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


class Search:
    def __init__(self, seed, n, beams, keep, vocab, dtype="bf16", finished=0.0, masked=0.0,
                 pad=0, spread=2.5, eos=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = n * beams
        wide = torch.randn((rows, vocab + pad), generator=g, device="cuda") * spread
        if masked:
            wide[torch.rand(wide.shape, generator=g, device="cuda") < masked] = -float("inf")
        wide[:, vocab:] = float("nan")
        self.logits = wide.to(T[dtype])[:, :vocab]
        self.scores = -10 * torch.rand(rows, generator=g, device="cuda")
        self.eos = vocab // 2 if eos is None else eos
        self.finished = torch.rand(rows, generator=g, device="cuda") < finished if finished \
            else None
        self.n, self.beams, self.keep, self.vocab = n, beams, keep, vocab

    def call(self, in_place=False, with_done=True, **kw):
        shape = (self.n, self.keep)
        out = (torch.full(shape, 7.0, device="cuda"),
               *(torch.full(shape, 7, dtype=torch.int32, device="cuda") for _ in "pt"))
        done = torch.zeros(shape, dtype=torch.bool, device="cuda") if with_done else None
        ws = pa.beam_select_workspace(self.logits, self.beams, self.keep)
        for _ in range(2):
            pa.pa_beam_select(*out, self.logits, self.scores, self.beams, ws,
                              finished=self.finished, eos_token=self.eos, finished_out=done,
                              in_place=in_place, **kw)
        torch.cuda.synchronize()
        assert not ws[1].any()
        return [x.cpu().numpy() for x in out] + [done.cpu().numpy() if with_done else None]

    def host(self):
        return (self.logits.double().cpu().numpy(), self.scores.double().cpu().numpy(),
                None if self.finished is None else self.finished.cpu().numpy())

    def check(self, got, in_place=False):
        logits, scores, finished = self.host()
        t = OS.totals(logits, scores, finished, self.eos)
        want = OS.beam_select(logits, scores, self.beams, self.keep, finished, self.eos, in_place)
        assert np.array_equal(np.isfinite(got[0]), np.isfinite(want[0]))
        fine = np.isfinite(want[0])
        assert np.all(got[1][~fine] == -1) and np.all(got[2][~fine] == -1)
        # the chosen are the best ones (equal but for totals closer than the errors)
        for b in range(self.n):
            f = np.isfinite(got[0][b])
            mine = t[got[1][b][f], got[2][b][f]]
            assert np.all(np.abs(np.sort(mine) - np.sort(want[0][b][f])) <= 2 * ATOL)
            assert np.all(np.abs(mine - got[0][b][f]) <= ATOL + 2.0 ** -24 * np.abs(mine))
            assert len({(r, v) for r, v in zip(got[1][b][f], got[2][b][f])}) == f.sum()
            gaps = np.diff(np.sort(t[b * self.beams:(b + 1) * self.beams].reshape(-1))[
                -self.keep - 1:])
            if not np.any((gaps > 0) & (gaps < 4 * ATOL)):       # then the order is theirs too
                assert np.array_equal(got[1][b], want[1][b]), b
                assert np.array_equal(got[2][b], want[2][b]), b
                if got[3] is not None:
                    assert np.array_equal(got[3][b], want[3][b]), b


@pytest.mark.parametrize("dtype", sorted(T))
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 100, 255, 2047, 2048, 2049, 5003, 32000, 50257])
def test_vocabularies(dtype, vocab):
    pa.pa_clear_device_error()
    s = Search(vocab, 3, 4, 8, vocab, dtype)
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("beams,keep", [(1, 1), (1, 2), (2, 4), (3, 5), (5, 10), (8, 16), (16, 32),
                                        (32, 64), (32, 1), (7, 33)])
@pytest.mark.parametrize("vocab", [5, 3001])
def test_beams(beams, keep, vocab):
    pa.pa_clear_device_error()
    s = Search(beams * 100 + keep, 5, beams, keep, vocab, "fp32", finished=0.2)
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("n,beams,vocab,dtype", [(200, 4, 9000, "bf16"), (150, 4, 70001, "bf16"),
                                                 (40, 16, 40003, "fp16"), (160, 4, 33001, "fp32"),
                                                 (4000, 16, 1025, "bf16")])
def test_many_rows(n, beams, vocab, dtype):
    """As many rows as make threads take more logits each."""
    pa.pa_clear_device_error()
    s = Search(n + vocab, n, beams, beams, vocab, dtype, finished=0.1)
    check_some(s, s.call(), np.random.default_rng(0).choice(n, 12, replace=False))
    assert pa.pa_get_device_error() == 0


def check_some(s, got, take):
    """Searches `take` of s alone."""
    few = Search.__new__(Search)
    few.__dict__ = dict(s.__dict__)
    rows = (take[:, None] * s.beams + np.arange(s.beams)).reshape(-1)
    few.n = len(take)
    few.logits, few.scores = s.logits[rows], s.scores[rows]
    few.finished = None if s.finished is None else s.finished[rows]
    shift = (take - np.arange(len(take)))[:, None] * s.beams
    part = [g[take] for g in got]
    part[1] = np.where(part[1] >= 0, part[1] - shift, -1)
    few.check(part)


@pytest.mark.parametrize("n,beams,keep,vocab", [(4, 32, 64, 30011), (8, 16, 32, 20000),
                                                (2, 32, 33, 9000), (1, 1, 64, 120000),
                                                (3, 24, 64, 50257)])
def test_wide_searches(n, beams, keep, vocab):
    """Many finds of many parts, most of them of a good beam or two."""
    pa.pa_clear_device_error()
    s = Search(vocab + keep, n, beams, keep, vocab, "fp32")
    s.check(s.call())
    s.scores[::beams] += 10.0
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", sorted(T))
@pytest.mark.parametrize("pad", [0, 1, 7])
def test_long_parts(dtype, pad):
    """Rows whose parts have many blocks of logits: of any values, rising, equal, all but a
    few hidden, and bad in a last block."""
    pa.pa_clear_device_error()
    s = Search(pad, 128, 4, 6, 61003, dtype, pad=pad)
    s.logits[8:12] = torch.linspace(-9, 9, 61003, device="cuda").to(T[dtype])
    s.logits[16:20] = 0.25
    s.scores[16:20] = -1.0
    s.logits[24:28] = -float("inf")
    s.logits[25, 60000:60004] = 1.0
    got = s.call()
    check_some(s, got, np.array([0, 2, 4, 6, 7, 127]))
    assert got[1][4].tolist() == [16] * 6 and got[2][4].tolist() == list(range(6))
    assert got[2][6].tolist() == [60000, 60001, 60002, 60003, -1, -1]
    assert pa.pa_get_device_error() == 0
    s.logits[33, 60990], s.logits[34, 5], s.logits[35, 61002] = (float("nan"), float("inf"),
                                                                 float("nan"))
    got = s.call()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_LOGITS
    pa.pa_clear_device_error()
    check_some(s, got, np.array([7, 8, 9]))


@pytest.mark.parametrize("pad", [0, 1, 3, 4, 5, 8])
@pytest.mark.parametrize("dtype", sorted(T))
def test_strides_and_alignments(pad, dtype):
    pa.pa_clear_device_error()
    s = Search(pad, 4, 3, 6, 1003, dtype, pad=pad)
    s.check(s.call())
    s.logits = s.logits[:, 1:]                   # (the first row misaligned too)
    s.vocab -= 1
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("masked", [0.5, 0.99, 1.0])
def test_forbidden_tokens(masked):
    pa.pa_clear_device_error()
    s = Search(11, 6, 4, 8, 700, "bf16", masked=masked)
    s.logits[5] = -float("inf")
    s.scores[9] = -float("inf")
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", sorted(T))
@pytest.mark.parametrize("vocab", [40, 3000, 50000])
def test_equal_logits(dtype, vocab):
    """Rows of nothing but ties: the lower beam, then the lower token first; equal rows at
    different alignments have equal totals."""
    pa.pa_clear_device_error()
    s = Search(12, 3, 4, 8, vocab, dtype)
    s.logits[:] = 0.5
    s.scores[:] = -1.0
    got = s.call()
    n = min(8, vocab)
    assert got[1].tolist() == [[4 * b] * 8 for b in range(3)]
    assert got[2].tolist() == [list(range(8))] * 3 and n == 8
    # (whatever the row holds, tied values among its largest too: the oracle's order)
    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        row = torch.randn(vocab, generator=g, device="cuda").to(T[dtype])
        s.logits[:] = row
        got = s.call()
        want = OS.beam_select(*s.host()[:2], 4, 8, eos=s.eos)
        assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    wide = torch.zeros((12, vocab + 1), dtype=T[dtype], device="cuda")
    wide[:, :vocab] = row
    s.logits = wide[:, :vocab]
    assert all(np.array_equal(a, b) for a, b in zip(s.call(), got))
    assert pa.pa_get_device_error() == 0


def test_few_equal_logits_above_the_rest():
    pa.pa_clear_device_error()
    s = Search(13, 2, 2, 6, 20000, "bf16")
    s.logits[:] = -3.0
    s.logits[1, 7::1000] = 4.0
    s.scores[:] = 0.0
    got = s.call()
    assert got[1][0].tolist() == [1] * 6 and got[2][0].tolist() == [7 + 1000 * i for i in range(6)]
    s.check(got)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", sorted(T))
def test_bad_logits_are_reported(bad, dtype):
    s = Search(14, 3, 2, 4, 3000, dtype)
    s.logits[1, 17] = bad
    s.logits[1, 2900] = bad
    s.logits[4] = bad
    pa.pa_clear_device_error()
    got = s.call()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_LOGITS
    s.check(got)
    s = Search(15, 3, 2, 4, 300, dtype)
    s.scores[2] = bad
    pa.pa_clear_device_error()
    got = s.call()
    assert pa.pa_get_device_error() == pa.PA_DEVERR_LOGITS
    s.check(got)
    pa.pa_clear_device_error()


def test_large_logits():
    pa.pa_clear_device_error()
    s = Search(16, 2, 3, 6, 3000, "fp32", spread=1e37)
    t = OS.totals(*s.host()[:2])
    got = s.call()
    for b in range(2):
        assert np.all(t[got[1][b], got[2][b]] >= np.sort(t[3 * b:3 * b + 3].reshape(-1))[-6])
    s = Search(17, 2, 3, 6, 3000, "fp32", spread=1e-30)
    s.check(s.call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("beams", [1, 3, 4, 32])
def test_in_place(seed, beams):
    pa.pa_clear_device_error()
    s = Search(200 + seed, 9, beams, beams, 60, "fp32", finished=0.3)
    s.scores *= 0.2
    got = s.call(in_place=True)
    s.check(got, in_place=True)
    par = got[1].reshape(-1)
    live = par >= 0
    assert np.array_equal(par[par[live]], par[live])     # parents keep their places
    assert pa.pa_get_device_error() == 0


def test_outputs_may_be_the_inputs():
    pa.pa_clear_device_error()
    s = Search(18, 50, 4, 4, 999, "bf16", finished=0.3)
    want = s.call(in_place=True)
    scores = s.scores.clone().view(50, 4)
    done = s.finished.clone().view(50, 4)
    parents, tokens = (torch.zeros((50, 4), dtype=torch.int32, device="cuda") for _ in "pt")
    pa.pa_beam_select(scores, parents, tokens, s.logits, scores, 4,
                      pa.beam_select_workspace(s.logits, 4, 4), finished=done, eos_token=s.eos,
                      finished_out=done, in_place=True)
    for a, b in zip((scores, parents, tokens, done), want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert pa.pa_get_device_error() == 0


def test_handles_replayed_on_two_streams():
    pa.pa_clear_device_error()
    made = []
    for i in range(2):
        s = Search(19 + i, 8, 4, 8, 32000, "bf16")
        out = (torch.zeros((8, 8), device="cuda"),
               *(torch.zeros((8, 8), dtype=torch.int32, device="cuda") for _ in "pt"))
        call = pa.BeamSelect(*out, s.logits, s.scores, 4)
        torch.cuda.synchronize()
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                call()
        made.append((s, out, g, st, call))
    torch.cuda.synchronize()
    for _ in range(4):
        for s, out, g, st, _ in made:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, out, *_ in made:
        s.eos = -1
        s.check([x.cpu().numpy() for x in out] + [None])
    assert pa.pa_get_device_error() == 0


def test_selection_refusals():
    s = Search(21, 2, 3, 3, 100, "fp32")
    out = (torch.zeros((2, 3), device="cuda"),
           *(torch.zeros((2, 3), dtype=torch.int32, device="cuda") for _ in "pt"))
    ws = pa.beam_select_workspace(s.logits, 3, 3)

    def call(out=out, logits=s.logits, scores=s.scores, beams=3, ws=ws, **kw):
        pa.pa_beam_select(*out, logits, scores, beams, ws, **kw)

    call()
    for kw in (dict(beams=4), dict(beams=0), dict(scores=s.scores[:5]), dict(logits=s.logits[0]),
               dict(logits=s.logits.t()), dict(logits=s.logits[:, :1].expand(6, 100)),
               dict(out=(out[0][:1], *out[1:])), dict(out=(out[0], out[1][:, :2], out[2])),
               dict(finished=torch.zeros(5, dtype=torch.bool, device="cuda"), eos_token=1),
               dict(ws=(ws[0][:16], ws[1])), dict(ws=(ws[0], ws[1][:1])),
               dict(logits=s.logits.cpu()), dict(scores=s.scores.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(logits=s.logits.double()), dict(scores=s.scores.double()),
               dict(finished=s.scores, eos_token=1)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(eos_token=100), dict(finished=s.scores > 0)):
        with pytest.raises(pa.PAError):
            call(**kw)


# ------------------------------------------------------------------ reordering

@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 16, 32])
@pytest.mark.parametrize("row,dtype", [(1, torch.int8), (3, torch.int16), (7, torch.bfloat16),
                                       (8, torch.bfloat16), (5, torch.int32), (512, torch.int32),
                                       (4099, torch.bfloat16), (5000, torch.float32),
                                       (20001, torch.uint8)])
def test_reorder(beams, row, dtype):
    pa.pa_clear_device_error()
    rng = np.random.default_rng(beams * 1000 + row)
    groups = 5
    n = groups * beams
    parents = np.arange(n) // beams * beams + rng.integers(0, beams, n)
    parents[rng.random(n) < 0.2] = -1
    states = [torch.from_numpy(rng.integers(-100, 100, (n, row))).cuda().to(dtype)
              for _ in range(3)]
    want = [torch.from_numpy(OS.reorder(s.double().cpu().numpy(), parents, beams)).to(dtype)
            for s in states]
    pa.pa_reorder_states(states, _dev(parents, np.int32), beams)
    for s, w in zip(states, want):
        assert torch.equal(s.cpu(), w)
    assert pa.pa_get_device_error() == 0


def test_reorder_cycles_strides_and_many_tensors():
    pa.pa_clear_device_error()
    parents = np.array([1, 2, 3, 0, 5, 4, 6, 6], dtype=np.int32)
    wide = torch.arange(8 * 40, dtype=torch.int32, device="cuda").view(8, 40)
    before = wide.clone()
    pa.pa_reorder_states(wide[:, 4:33], _dev(parents, np.int32), 4)
    assert torch.equal(wide[:, 4:33], before[parents.tolist()][:, 4:33])
    assert torch.equal(wide[:, :4], before[:, :4]) and torch.equal(wide[:, 33:], before[:, 33:])
    many = torch.randn((70, 8, 4, 36), device="cuda")
    before = many.clone()
    call = pa.ReorderStates(many.unbind(0), _dev(parents, np.int32), 4)
    call()
    assert torch.equal(many, before[:, parents.tolist()])
    call()                                              # once more from where it stands
    assert torch.equal(many, before[:, parents.tolist()][:, parents.tolist()])
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("beams", [4, 16])
def test_reorder_views_of_one_tensor(beams):
    """Rows of several states that alternate in one tensor."""
    pa.pa_clear_device_error()
    rng = np.random.default_rng(beams)
    parents = np.arange(48) // beams * beams + rng.integers(0, beams, 48)
    whole = torch.randn((48, 5, 36), device="cuda")
    before = whole.clone()
    views = [whole[:, i] for i in (3, 0, 4, 1)]
    pa.pa_reorder_states(views, _dev(parents, np.int32), beams)
    want = before[parents.tolist()]
    want[:, 2] = before[:, 2]
    assert torch.equal(whole, want) and pa.pa_get_device_error() == 0
    for twice in ([whole[:, 1], whole[:, 1]], [whole[:, 1:3], whole[:, 2:4]]):
        with pytest.raises(pa.PAError):
            pa.pa_reorder_states(twice, _dev(parents, np.int32), beams)
    own = _dev(parents, np.int32)
    with pytest.raises(pa.PAError):
        pa.pa_reorder_states(own.view(48, 1), own, beams)
    assert torch.equal(whole, want)


def test_reorder_bad_parents_leave_their_rows():
    x = torch.randn((6, 33), device="cuda")
    before = x.clone()
    pa.pa_clear_device_error()
    pa.pa_reorder_states(x, _dev([1, 0, 5, 9999999, 3, -2 ** 31], np.int32), 3)
    assert pa.pa_get_device_error() == pa.PA_DEVERR_PARENT
    assert torch.equal(x, before[[1, 0, 2, 3, 3, 5]])
    pa.pa_clear_device_error()


def test_reorder_past_32_bits():
    pa.pa_clear_device_error()
    x = torch.zeros((4, 1200 * 1000 * 1000), dtype=torch.uint8, device="cuda")
    x[:, -5:] = torch.arange(20, dtype=torch.uint8, device="cuda").view(4, 5)
    pa.pa_reorder_states(x, _dev([3, 1, 0, 3], np.int32), 4)
    assert x[:, -5:].cpu().tolist() == [[15, 16, 17, 18, 19], [5, 6, 7, 8, 9], [0, 1, 2, 3, 4],
                                        [15, 16, 17, 18, 19]]
    assert pa.pa_get_device_error() == 0


def test_reorder_refusals():
    x = torch.zeros((6, 8), device="cuda")
    par = _dev(np.arange(6), np.int32)
    pa.pa_reorder_states(x, par, 3)
    pa.pa_reorder_states([], par, 3)
    pa.pa_reorder_states(x[:, :0], par, 3)
    for args in ((x, par, 4), (x, par, 0), (x[:5], par, 3), ([x, x[:, :4]], par, 3),
                 (x.t(), par, 3), (x[:1].expand(6, 8), par, 3), (x.cpu(), par, 3),
                 (x, par.cpu(), 3)):
        with pytest.raises(ValueError):
            pa.pa_reorder_states(*args)
    with pytest.raises(TypeError):
        pa.pa_reorder_states(x, par.long(), 3)
