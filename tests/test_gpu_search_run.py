"""A beam search over the paged cache as an encoder-decoder server runs it: sources
in paged blocks, the beams' own tokens in a cache whose blocks they share until they
write, cross attention, selection, and the reordering of tables and states -- against
the same search in float64."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as OA
from oracle import search as OS
from oracle.allocator import BlockAllocatorModel
from oracle.bf16 import bf16_bits_to_f64
from oracle.rope import to_bf16_bits
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16, host_bits

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 4, 2)])
def test_search_over_paged_caches(d, hq, hkv):
    pa.pa_clear_device_error()
    rng = np.random.default_rng(d)
    searches, beams, vocab, steps, eos = 3, 4, 401, 24, 7
    rows = searches * beams
    scale = d ** -0.5
    # sources, written through their slots
    src = np.array([70, 5, 200], dtype=np.int32)
    nblk = -(-src // 16)
    perm = rng.permutation(int(nblk.sum()) + 2)
    stab = np.full((searches, int(nblk.max())), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(nblk.tolist()):
        stab[b, :k] = perm[at:at + k]
        at += k
    sk, sv = (normal_bf16(rng, (perm.shape[0], hkv, 16, d)) for _ in "kv")
    dsk, dsv = dev_bf16(sk), dev_bf16(sv)
    start = _dev(np.arange(searches + 1) * beams, np.int32)
    # decoder embeddings: a token's q, k, v, and the projection to the vocabulary
    emb = [normal_bf16(rng, (vocab, h, d)) for h in (hq, hkv, hkv)]
    proj = normal_bf16(rng, (2 * hq * d, vocab))
    demb, dproj = [dev_bf16(e) for e in emb], dev_bf16(proj).float()
    fproj = bf16_bits_to_f64(proj)
    nb = 64
    alloc, model = pa.BlockAllocator(nb, 16), BlockAllocatorModel(nb, 16)
    for a in (alloc, model):
        for r in range(rows):
            a.add_seq(r)
    kc, vc = (torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    scores = torch.full((searches, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0                                   # the beams are equal at first
    done = torch.zeros((searches, beams), dtype=torch.bool, device="cuda")
    history = torch.full((rows, steps), -1, dtype=torch.int32, device="cuda")
    state = torch.zeros((rows, 37), device="cuda")       # a running sum of q, as a state
    tokens = torch.full((searches, beams), 1, dtype=torch.int32, device="cuda")
    parents = torch.zeros_like(tokens)
    logits = torch.zeros((rows, vocab), device="cuda")
    cross, own = (torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda") for _ in "co")
    q = torch.zeros_like(cross)
    attend = pa.CrossAttention(cross, q, dsk, dsv, _dev(stab, np.int32), _dev(src, np.int32),
                               start, beams, scale)
    select = pa.BeamSelect(scores, parents, tokens, logits, scores, beams, finished=done,
                           eos_token=eos, finished_out=done, in_place=True)
    move = pa.ReorderStates([history], parents, beams)
    move_state = pa.ReorderStates([state], parents, beams)
    # the search in float64 keeps whole histories of its own
    told = [[1] for _ in range(rows)]
    for step in range(steps):
        tok = tokens.view(-1).long().clamp(min=0)
        q.copy_(demb[0][tok])
        slots, cow_src, cow_dst = alloc.append_slots(list(range(rows)))
        want = model.append_slots(range(rows))
        assert [w[0] for w in want] == slots.tolist()
        pairs = [(s, t) for s, t in zip(cow_src.tolist(), cow_dst.tolist()) if s >= 0]
        if pairs:
            pa.pa_copy_blocks([kc], [vc], _dev(pairs, np.int64))
        tables, ctx = alloc.block_tables(list(range(rows)), 4)
        counters = pa.step_counters(rows, hkv)
        ws = pa.splitk_workspace(rows, hq, d, 64, 64)
        pa.pa_decode_step(own, q, kc, vc, _dev(tables, np.int32), _dev(ctx, np.int32), scale,
                          key=demb[1][tok].contiguous(), value=demb[2][tok].contiguous(),
                          slot_mapping=_dev(slots, np.int64), partition_size=64, workspace=ws,
                          counters=counters)
        attend()
        state += q.float().view(rows, -1)[:, :37]
        both = torch.cat([own.view(rows, -1), cross.view(rows, -1)], 1).float()
        logits.copy_(both @ dproj * 0.3)
        # the same attention from every beam's own history
        seen = np.array([told[r] for r in range(rows)])
        for r in range(rows):
            k, v = (bf16_bits_to_f64(e[seen[r]]) for e in emb[1:])
            qr = bf16_bits_to_f64(emb[0][seen[r, -1]])
            ref = np.stack([OA.softmax_attention(qr[h], k[:, h // (hq // hkv)],
                                                 v[:, h // (hq // hkv)], scale)
                            for h in range(hq)])
            assert_close(bf16_to_f64(own[r])[None], ref[None], f"step {step} row {r}")
        ref, _ = OS.cross_attention(emb[0][seen[:, -1]], sk, sv, stab, src, [beams] * searches,
                                    scale)
        assert_close(bf16_to_f64(cross), ref, f"step {step}")
        # selection on the device's own logits
        before = scores.double().cpu().numpy().reshape(-1)
        fin = done.cpu().numpy().reshape(-1)
        host = logits.double().cpu().numpy()
        t = OS.totals(host, before, fin, eos)
        select()
        got = [x.cpu().numpy().reshape(-1) for x in (scores, parents, tokens)]
        wanted = OS.beam_select(host, before, beams, beams, fin, eos, in_place=True)
        assert np.allclose(np.sort(got[0].reshape(searches, beams)), np.sort(wanted[0]),
                           atol=2e-5, rtol=1e-6)
        for r in range(rows):
            assert got[1][r] // beams == r // beams
            assert abs(t[got[1][r], got[2][r]] - got[0][r]) < 2e-5 * (1 + abs(got[0][r]))
        move()
        move_state()
        history[:, step] = tokens.view(-1)
        for a in (alloc, model):
            a.reorder(list(range(rows)), got[1].tolist())
        told = [told[got[1][r]] + [int(got[2][r])] for r in range(rows)]
        assert list(alloc.free_list()) == model.free_list()
    h = history.cpu().numpy()
    sums = np.zeros((rows, 37))
    for r in range(rows):
        assert h[r].tolist() == told[r][1:]
        for v in told[r][:-1]:
            sums[r] += bf16_bits_to_f64(emb[0][v]).reshape(-1)[:37]
    assert np.allclose(state.cpu().numpy(), sums, atol=1e-3)
    used = nb - alloc.num_free()
    assert used < rows * 2                               # shared, not copied
    assert pa.pa_get_device_error() == 0
