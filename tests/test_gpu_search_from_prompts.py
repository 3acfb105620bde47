"""A search from its prompts on, over caches that the library's own calls fill: an
encoder's states written to their paged cache, decoder prompts written and prefilled,
cross attention of the prompts, forks, steps of the beams, and the caches read back."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as OA
from oracle import prefill as OP
from oracle import search as OS
from oracle.bf16 import bf16_bits_to_f64
from paged_kv_cache_283_gb300 import pa
from paged_kv_cache_283_gb300.inputs import normal_bf16

from gpu_helpers import assert_close, bf16_to_f64, dev_bf16

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _tables(alloc, seqs, blocks):
    tables, lens = alloc.block_tables(seqs, blocks)
    return tables, _dev(tables, np.int32), _dev(lens, np.int32)


def _slots(table, n):
    pos = np.arange(n)
    return table[pos // 16].astype(np.int64) * 16 + pos % 16


def test_search_from_prompts():
    pa.pa_clear_device_error()
    rng = np.random.default_rng(3)
    searches, beams, vocab, steps, d, hq, hkv = 3, 4, 307, 20, 128, 8, 2
    rows, scale = searches * beams, 128 ** -0.5
    src, lens = [130, 1, 47], [21, 3, 40]
    # the encoder's states, back to back, to their own cache
    enc = [normal_bf16(rng, (sum(src), hkv, d)) for _ in "kv"]
    sources = pa.BlockAllocator(16, 16, rng.permutation(16).tolist())
    for b, n in enumerate(src):
        sources.add_seq(b)
        sources.reserve(b, n)
    stab, dstab, dsrc = _tables(sources, list(range(searches)), 9)
    sk, sv = (torch.full((16, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in "kv")
    sslots = np.concatenate([_slots(stab[b], n) for b, n in enumerate(src)])
    pa.pa_reshape_and_cache(dev_bf16(enc[0]), dev_bf16(enc[1]), sk, sv, _dev(sslots, np.int64))
    host_k, host_v = (np.zeros((16, hkv, 16, d), dtype=np.uint16) for _ in "kv")
    for e, pool in zip(enc, (host_k, host_v)):
        pool[sslots // 16, :, sslots % 16] = e
    # prompts: written, prefilled and crossed, one sequence a search
    emb = [normal_bf16(rng, (vocab, h, d)) for h in (hq, hkv, hkv)]
    demb = [dev_bf16(e) for e in emb]
    proj = dev_bf16(normal_bf16(rng, (2 * hq * d, vocab))).float() * 0.3
    prompts = [rng.integers(0, vocab, n).tolist() for n in lens]
    tok = torch.tensor(sum(prompts, []), device="cuda")
    nb = 64
    alloc = pa.BlockAllocator(nb, 16)
    kc, vc = (torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    first = [b * beams for b in range(searches)]
    for r, n in zip(first, lens):
        alloc.add_seq(r)
        alloc.reserve(r, n)
    tab, dtab, dctx = _tables(alloc, first, 6)
    slots = np.concatenate([_slots(tab[b], n) for b, n in enumerate(lens)])
    q, key, value = (e[tok].contiguous() for e in demb)
    start = _dev(np.concatenate([[0], np.cumsum(lens)]), np.int32)
    pa.pa_reshape_and_cache(key, value, kc, vc, _dev(slots, np.int64))
    own, cross = torch.zeros_like(q), torch.zeros_like(q)
    pa.pa_prefill(own, q, kc, vc, dtab, dctx, start, max(lens), scale)
    work = pa.CrossWorkspace(max(lens), hq, hkv, d)      # one for every call of the stream
    pa.CrossAttention(cross, q, sk, sv, dstab, dsrc, start, max(lens), scale, work)()
    said = np.array(sum(prompts, []))
    pools = [np.zeros((nb, hkv, 16, d), dtype=np.uint16) for _ in "kv"]
    for e, pool in zip(emb[1:], pools):
        pool[slots // 16, :, slots % 16] = e[said]
    assert_close(bf16_to_f64(own), OP.prefill(emb[0][said], *pools, tab, np.array(lens),
                                              np.array(lens), scale, 16), "prefill")
    want, _ = OS.cross_attention(emb[0][said], host_k, host_v, stab, src, lens, scale)
    assert_close(bf16_to_f64(cross), want, "cross attention of the prompts")
    # one beam a search to begin with: the others fork from it and count for nothing yet
    for r in first:
        for w in range(1, beams):
            alloc.fork(r, r + w)
    last = (start[1:] - 1).long().repeat_interleave(beams)
    scores = torch.full((searches, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    parents, tokens = (torch.zeros((searches, beams), dtype=torch.int32, device="cuda")
                       for _ in "pt")
    history = torch.full((rows, steps + 1), -1, dtype=torch.int32, device="cuda")
    logits = torch.zeros((rows, vocab), device="cuda")
    out, seen = (torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda") for _ in "ab")
    qs = torch.zeros_like(out)
    at = _dev(np.arange(searches + 1) * beams, np.int32)
    select = pa.BeamSelect(scores, parents, tokens, logits, scores, beams, in_place=True)
    move = pa.ReorderStates([history], parents, beams)
    attend = pa.CrossAttention(out, qs, sk, sv, dstab, dsrc, at, beams, scale, work)
    told = [list(prompts[r // beams]) for r in range(rows)]

    def choose(a, b, step):
        logits.copy_(torch.cat([a.reshape(rows, -1), b.reshape(rows, -1)], 1).float() @ proj)
        before = scores.double().cpu().numpy().reshape(-1)
        t = OS.totals(logits.double().cpu().numpy(), before)
        select()
        move()
        history[:, step] = tokens.view(-1)
        alloc.reorder(list(range(rows)), parents.tolist())   # [searches, beams] of them
        par, new, got = (x.cpu().numpy().reshape(-1) for x in (parents, tokens, scores))
        for r in range(rows):
            assert par[r] // beams == r // beams and abs(t[par[r], new[r]] - got[r]) < 1e-4
        for b in range(searches):
            best = np.sort(t[b * beams:(b + 1) * beams].reshape(-1))[-beams:]
            assert np.abs(np.sort(got[b * beams:(b + 1) * beams]) - best).max() < 1e-4
        return [told[par[r]] + [int(new[r])] for r in range(rows)]

    told = choose(own[last], cross[last], 0)
    for step in range(1, steps + 1):
        now = tokens.view(-1).long()
        qs.copy_(demb[0][now])
        slots, cow_src, cow_dst = alloc.append_slots(list(range(rows)))
        pairs = [(a, b) for a, b in zip(cow_src.tolist(), cow_dst.tolist()) if a >= 0]
        if pairs:
            pa.pa_copy_blocks([kc], [vc], _dev(pairs, np.int64))
        tab, dtab, dctx = _tables(alloc, list(range(rows)), 6)
        pa.pa_reshape_and_cache(demb[1][now].contiguous(), demb[2][now].contiguous(), kc, vc,
                                _dev(slots, np.int64))
        pa.pa_decode(seen, qs, kc, vc, dtab, dctx, scale)
        attend()
        lines = np.array([t[-1] for t in told])
        for r in range(rows):
            k, v = (bf16_bits_to_f64(e[told[r]]) for e in emb[1:])
            x = bf16_bits_to_f64(emb[0][lines[r]])
            ref = np.stack([OA.softmax_attention(x[h], k[:, h // (hq // hkv)],
                                                 v[:, h // (hq // hkv)], scale)
                            for h in range(hq)])
            assert_close(bf16_to_f64(seen[r])[None], ref[None], f"step {step} row {r}")
        want, _ = OS.cross_attention(emb[0][lines], host_k, host_v, stab, src, [beams] * searches,
                                     scale)
        assert_close(bf16_to_f64(out), want, f"cross attention of step {step}")
        told = choose(seen, out, step)
    for r in range(rows):
        assert history[r].tolist() == told[r][lens[r // beams]:]
    # the caches hold what went in: the sources, and every beam's own tokens but the last
    ko, vo = (torch.zeros((sum(src), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pa.pa_read_cache(ko, vo, sk, sv, dstab, _dev(np.concatenate([[0], np.cumsum(src)]), np.int32),
                     max(src))
    assert torch.equal(ko, dev_bf16(enc[0])) and torch.equal(vo, dev_bf16(enc[1]))
    tab, dtab, dctx = _tables(alloc, list(range(rows)), 6)
    held = [len(t) - 1 for t in told]
    assert dctx.tolist() == held
    ko, vo = (torch.zeros((sum(held), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pa.pa_read_cache(ko, vo, kc, vc, dtab, _dev(np.concatenate([[0], np.cumsum(held)]), np.int32),
                     max(held))
    line = torch.tensor(sum((t[:-1] for t in told), []), device="cuda")
    assert torch.equal(ko, demb[1][line]) and torch.equal(vo, demb[2][line])
    assert pa.pa_get_device_error() == 0
