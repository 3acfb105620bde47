"""Cases of the operators of beam search and encoder-decoder serving over the
paged KV cache: what they compute in plain torch operations, and the calls a
user makes of the library for the same.

Operators:
  cross     attention of decoder queries (prompts, or the beams of one step,
            which share their source) to an encoder's states in a paged cache
  beam      the best continuations of a search's beams over the vocabulary
  reorder   states of the beams moved to where their parents' went, in place
  read      positions of a paged cache of any type (bf16, INT8, FP8, 4-bit)
            read back as bf16 rows, or into the slots of a bf16 cache

``own`` chooses the side: False, elementary torch operations; True, the
library's calls.  Sizes follow the library's own workloads (32 query / 8 KV
heads of 128 dims, blocks of 16 tokens) and other shapes it supports.
"""
import math
import random

import torch

own = False

BLOCK = 16
GROUP = 64  # dims that share one 4-bit scale and offset


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one short source, four beams: a latency-bound call
        {"name": "cross_one_source", "op": "cross", "seqs": 1, "hq": 8, "hkv": 8, "d": 64,
         "q_lo": 4, "q_hi": 4, "src_lo": 37, "src_hi": 37, "lens": 1},
        # a decode step of 64 searches of 4 beams
        {"name": "cross_step_64x4", "op": "cross", "seqs": 64, "hq": 32, "hkv": 8, "d": 128,
         "q_lo": 4, "q_hi": 4, "src_lo": 128, "src_hi": 2048, "lens": 2},
        # few long sources, as many KV heads as query heads
        {"name": "cross_step_long", "op": "cross", "seqs": 3, "hq": 16, "hkv": 16, "d": 64,
         "q_lo": 5, "q_hi": 5, "src_lo": 8192, "src_hi": 65536, "lens": 3},
        # decoder prompts, ragged, some sources empty
        {"name": "cross_ragged_prompts", "op": "cross", "seqs": 9, "hq": 16, "hkv": 16, "d": 64,
         "q_lo": 1, "q_hi": 700, "src_lo": 0, "src_hi": 1500, "lens": 4},
        # an 8192-token step of decoder prompts
        {"name": "cross_prompts_16x512", "op": "cross", "seqs": 16, "hq": 32, "hkv": 8, "d": 128,
         "q_lo": 512, "q_hi": 512, "src_lo": 512, "src_hi": 4096, "lens": 5},
        # one search of four beams
        {"name": "beam_one", "op": "beam", "searches": 1, "beams": 4, "keep": 8, "vocab": 32000,
         "dtype": "bf16", "masked": 0.0, "finished": 0.0, "in_place": False, "lens": 6},
        # 64 searches over a large vocabulary, twice the beams kept
        {"name": "beam_64x4", "op": "beam", "searches": 64, "beams": 4, "keep": 8,
         "vocab": 128256, "dtype": "bf16", "masked": 0.0, "finished": 0.0, "in_place": False,
         "lens": 7},
        # an odd vocabulary, 32-bit logits, forbidden tokens and finished beams
        {"name": "beam_33x5_odd", "op": "beam", "searches": 33, "beams": 5, "keep": 5,
         "vocab": 50257, "dtype": "fp32", "masked": 0.3, "finished": 0.2, "in_place": True,
         "lens": 8},
        # block tables of 64 searches: little to move
        {"name": "reorder_tables", "op": "reorder", "layers": 1, "searches": 64, "beams": 4,
         "row": 512, "dtype": "int32", "lens": 9},
        # recurrent states of 8 layers, 16 searches
        {"name": "reorder_states", "op": "reorder", "layers": 8, "searches": 16, "beams": 4,
         "row": 131072, "dtype": "fp32", "lens": 10},
        # a few odd ranges of an INT8 cache into a bf16 cache's slots
        {"name": "read_int8_slots", "op": "read", "kind": "int8", "seqs": 3, "n_lo": 1,
         "n_hi": 120, "prior_hi": 200, "hkv": 8, "d": 128, "to_slots": True, "lens": 11},
        # 16 prompts' prefixes of a 4-bit cache, for their next chunk's prefill
        {"name": "read_int4_prefixes", "op": "read", "kind": "int4", "seqs": 16, "n_lo": 512,
         "n_hi": 8192, "prior_hi": 0, "hkv": 8, "d": 128, "to_slots": False, "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "beam", "reorder", "read"])
    lens = rng.randrange(1 << 20)
    if op == "cross":
        d = rng.choice([64, 128])
        group = rng.choice([1, 2, 4, 8])
        hkv = rng.choice([h for h in (1, 2, 3, 4, 8, 16) if h * group <= 32])
        seqs = _log_int(rng, 1, 64)
        step = rng.random() < 0.5
        q_hi = rng.choice([1, 2, 3, 4, 5, 8]) if step else _log_int(rng, 1, 700)
        src = _log_int(rng, 1, 32768)
        src = min(src, (3 << 19) // (seqs * hkv * d // 64),
                  (1 << 25) // (seqs * q_hi * hkv * group // 8 + 1))
        return {"op": op, "seqs": seqs, "hq": hkv * group, "hkv": hkv, "d": d,
                "q_lo": q_hi if step else _log_int(rng, 1, q_hi), "q_hi": q_hi,
                "src_lo": rng.choice([0, max(1, src // 16)]), "src_hi": max(1, src),
                "lens": lens}
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        in_place = rng.random() < 0.4
        vocab = _log_int(rng, 2, 200000)
        searches = _log_int(rng, 1, min(64, max(1, (1 << 25) // (beams * vocab * 2))))
        return {"op": op, "searches": searches, "beams": beams,
                "keep": beams if in_place else rng.choice([beams, 2 * beams]), "vocab": vocab,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "masked": rng.choice([0.0, 0.0, 0.5, 0.999]),
                "finished": rng.choice([0.0, 0.3]), "in_place": in_place, "lens": lens}
    if op == "reorder":
        layers = rng.choice([1, 2, 5, 8])
        beams = rng.choice([2, 3, 4, 5, 8, 16])
        searches = _log_int(rng, 1, 64)
        row = _log_int(rng, 1, min(131072, (1 << 26) // (layers * beams * searches)))
        return {"op": op, "layers": layers, "searches": searches, "beams": beams, "row": row,
                "dtype": rng.choice(["fp32", "bf16", "int32"]), "lens": lens}
    n_hi = _log_int(rng, 1, 8192)
    return {"op": op, "kind": rng.choice(["bf16", "int8", "fp8", "int4"]),
            "seqs": min(_log_int(rng, 1, 64), max(1, 65536 // n_hi)),
            "n_lo": _log_int(rng, 1, n_hi), "n_hi": n_hi, "prior_hi": rng.choice([0, 100, 3000]),
            "hkv": rng.choice([1, 2, 3, 4, 8]), "d": rng.choice([64, 128]),
            "to_slots": rng.random() < 0.5, "lens": lens}


def _lens(case):
    """From the case alone: cross, (source lengths, queries); read, (first
    positions, positions read); reorder, (parents, None)."""
    rng = random.Random(case["lens"])
    n = case.get("seqs", 0)
    if case["op"] == "cross":
        return ([rng.randint(case["src_lo"], case["src_hi"]) for _ in range(n)],
                [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)])
    if case["op"] == "read":
        return ([rng.randint(0, case["prior_hi"]) for _ in range(n)],
                [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(n)])
    # each place's parent: the survivors keep theirs, the other places go to forks of them
    beams, parents = case["beams"], []
    for b in range(case["searches"]):
        alive = [w for w in range(beams) if rng.random() < 0.6] or [rng.randrange(beams)]
        parents += [b * beams + (w if w in alive else rng.choice(alive)) for w in range(beams)]
    return parents, None


# --------------------------------------------------------------- the inputs

def _tables(ctx, gen):
    """(block tables [B, MB] int32, padded with -1; blocks in the pool)."""
    nblk = [-(-c // BLOCK) for c in ctx]
    total = sum(nblk)
    nb = total + total // 4 + 1
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    mb = max(1, max(nblk))
    n = torch.tensor(nblk, device="cuda")
    j = torch.arange(mb, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + j
    return torch.where(j < n[:, None], perm[at.clamp(max=nb - 1)], -1).to(torch.int32), nb


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _codes(shape, gen):
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)


def _pool4(nb, hkv, d, gen):
    """A 4-bit pool: codes, and per token and group an offset near the least
    value and a scale near a fifteenth of the range of normal values."""
    n = (nb, hkv, BLOCK * d // GROUP)
    lo = (-2.4 + 0.3 * torch.randn(n, generator=gen, device="cuda")).to(torch.bfloat16)
    sc = (0.32 + 0.04 * torch.randn(n, generator=gen, device="cuda")).abs().to(torch.bfloat16)
    par = torch.stack([lo, sc], -1).view(torch.uint8).reshape(nb, hkv, -1)
    return torch.cat([_codes((nb, hkv, 8 * d), gen), par], -1).contiguous()


def _starts(counts):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32,
                        device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = {"device": "cuda"}
    s = {"case": case}
    if case["op"] == "cross":
        src, new = _lens(case)
        hkv, d, hq = case["hkv"], case["d"], case["hq"]
        s["tables"], nb = _tables(src, gen)
        s["source_lens"] = torch.tensor(src, dtype=torch.int32, **dev)
        s["starts"], s["max_new"] = _starts(new), max(new)
        s["q"] = _normal((sum(new), hq, d), gen)
        s["out"] = torch.zeros_like(s["q"])
        s["k_cache"], s["v_cache"] = (_normal((nb, hkv, BLOCK, d), gen) for _ in "kv")
        s["scale"] = 1.0 / math.sqrt(d)
    elif case["op"] == "beam":
        n, beams, vocab = case["searches"], case["beams"], case["vocab"]
        t = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]
        # a peaked distribution: normal values, a few tokens far above the others
        x = 2.5 * torch.randn((n * beams, vocab), generator=gen, **dev)
        row = torch.arange(n * beams, **dev)
        for _ in range(4):
            peak = torch.randint(0, vocab, (n * beams,), generator=gen, **dev)
            x[row, peak] += 8.0 * torch.rand(n * beams, generator=gen, **dev)
        if case["masked"]:
            x[torch.rand(x.shape, generator=gen, **dev) < case["masked"]] = -torch.inf
        s["logits"] = x.to(t)
        s["scores"] = -20.0 - 6.0 * torch.rand(n * beams, generator=gen, **dev)
        s["eos"] = min(2, vocab - 1)
        s["finished"] = torch.rand(n * beams, generator=gen, **dev) < case["finished"] \
            if case["finished"] else None
        shape = (n, case["keep"])
        s["out_scores"] = torch.zeros(shape, **dev)
        s["parents"], s["tokens"] = (torch.zeros(shape, dtype=torch.int32, **dev) for _ in "pt")
    elif case["op"] == "reorder":
        rows, layers = case["searches"] * case["beams"], case["layers"]
        s["parents"] = torch.tensor(_lens(case)[0], dtype=torch.int32, **dev)
        shape = (layers, rows, case["row"])
        if case["dtype"] == "int32":
            s["states"] = torch.randint(0, 1 << 20, shape, generator=gen, dtype=torch.int32, **dev)
        else:
            s["states"] = _normal(shape, gen, torch.float32 if case["dtype"] == "fp32"
                                  else torch.bfloat16)
    else:
        first, n = _lens(case)
        hkv, d, kind = case["hkv"], case["d"], case["kind"]
        s["tables"], nb = _tables([a + b for a, b in zip(first, n)], gen)
        s["first"] = torch.tensor(first, dtype=torch.int32, **dev)
        s["starts"], s["max_rows"], s["rows"] = _starts(n), max(n), sum(n)
        shape = (nb, hkv, BLOCK, d)
        if kind == "bf16":
            s["k_cache"], s["v_cache"] = (_normal(shape, gen) for _ in "kv")
        elif kind == "int4":
            s["k_cache"], s["v_cache"] = (_pool4(nb, hkv, d, gen) for _ in "kv")
        else:
            s["k_cache"], s["v_cache"] = (_codes(shape, gen) for _ in "kv")
            if kind == "int8":
                s["k_cache"], s["v_cache"] = (s[x].view(torch.int8) for x in ("k_cache",
                                                                             "v_cache"))
            else:
                for x in ("k_cache", "v_cache"):  # no cache write makes the NaN codes
                    s[x][(s[x] & 127) == 127] = 0
            s["k_scales"], s["v_scales"] = (
                0.02 + 0.01 * torch.rand((nb, hkv, BLOCK), generator=gen, **dev) for _ in "kv")
        if case["to_slots"]:
            # each sequence's rows from the start of blocks of its own
            blocks = [-(-m // BLOCK) for m in n]
            to = torch.randperm(sum(blocks), generator=gen, **dev)
            count = torch.tensor(n, **dev)
            seq = torch.repeat_interleave(torch.arange(len(n), **dev), count)
            i = torch.arange(sum(n), **dev) - s["starts"][seq]
            begin = _starts(blocks).long()
            s["slots"] = to[begin[seq] + i // BLOCK] * BLOCK + i % BLOCK
            out = (sum(blocks), hkv, BLOCK, d)
        else:
            s["slots"], out = None, (sum(n), hkv, d)
        s["k_out"], s["v_out"] = (torch.zeros(out, dtype=torch.bfloat16, **dev) for _ in "kv")
    if own:
        s["call"] = _handle(case, s)
    return s


def _handle(case, s):
    """The library's handle of one call on these buffers, as a serving program keeps it."""
    from paged_kv_cache_283_gb300 import pa
    if case["op"] == "cross":
        return pa.CrossAttention(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"],
                                 s["source_lens"], s["starts"], s["max_new"], s["scale"])
    if case["op"] == "beam":
        return pa.BeamSelect(s["out_scores"], s["parents"], s["tokens"], s["logits"],
                             s["scores"], case["beams"], finished=s["finished"],
                             eos_token=s["eos"], in_place=case["in_place"])
    if case["op"] == "reorder":
        return pa.ReorderStates(s["states"].unbind(0), s["parents"], case["beams"])
    return pa.ReadCache(s["k_out"], s["v_out"], s["k_cache"], s["v_cache"], s["tables"],
                        s["starts"], s["max_rows"], first_positions=s["first"],
                        k_scales=s.get("k_scales"), v_scales=s.get("v_scales"),
                        slot_mapping=s["slots"])


# ------------------------------------------------------------ the plain form

def _plain_cross(s):
    c = s["case"]
    hkv, d, hq = c["hkv"], c["d"], c["hq"]
    src, new = _lens(c)
    row = 0
    for b, (n, m) in enumerate(zip(src, new)):
        q = s["q"][row:row + m].float().view(m, hkv, hq // hkv, d).permute(1, 2, 0, 3)
        if n:
            blocks = s["tables"][b, :-(-n // BLOCK)].long()
            k, v = (x[blocks].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
                    for x in (s["k_cache"], s["v_cache"]))
            x = torch.matmul(q.reshape(hkv, -1, d), k.transpose(1, 2)) * s["scale"]
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(p / p.sum(-1, keepdim=True), v)
        else:
            o = torch.zeros_like(q)
        o = o.reshape(hkv, hq // hkv, m, d).permute(2, 0, 1, 3).reshape(m, hq, d)
        s["out"][row:row + m] = o.to(torch.bfloat16)
        row += m
    return s["out"]


def _keep_places(parents, beams):
    """[B, K] place of each candidate (local parents, -1: none): the first child
    of a beam keeps its parent's place, the others take the free ones in order."""
    same = parents[:, :, None] == parents[:, None, :]
    home = (parents >= 0) & ~torch.tril(same, -1).any(-1)
    at = torch.arange(beams, device="cuda")
    taken = ((parents[:, :, None] == at) & home[:, :, None]).any(1)
    free = torch.sort(torch.where(taken, at + beams, at), 1).values
    other = (torch.cumsum(~home, 1) - 1).clamp(min=0)
    return torch.where(home, parents, free.gather(1, other))


def _plain_beam(s):
    """In 64 bits: totals of different beams can lie closer than 32 tell apart."""
    c = s["case"]
    n, beams, vocab, keep = c["searches"], c["beams"], c["vocab"], c["keep"]
    x = s["logits"].double()
    top = x.amax(1, keepdim=True).clamp(min=-1e300)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    total = torch.where(x > -torch.inf, s["scores"].double()[:, None] + (x - lse), -torch.inf)
    if s["finished"] is not None:
        only = torch.full_like(total, -torch.inf)
        only[:, s["eos"]] = s["scores"].double()
        total = torch.where(s["finished"][:, None], only, total)
    total = total.view(n, beams * vocab)
    at = torch.arange(beams * vocab, device="cuda")
    best, where = [], []
    for _ in range(keep):  # the largest, of equal ones the first
        m = total.amax(1, keepdim=True)
        i = torch.where(total == m, at, beams * vocab).amin(1, keepdim=True)
        i = i.clamp(max=beams * vocab - 1)
        best.append(m)
        where.append(torch.where(m > -torch.inf, i, -1))
        total.scatter_(1, i, -torch.inf)
    best, where = torch.cat(best, 1), torch.cat(where, 1)
    parent = torch.where(where >= 0, where // vocab, -1)
    token = torch.where(where >= 0, where % vocab, -1)
    rows = torch.where(where >= 0, parent + beams * torch.arange(n, device="cuda")[:, None], -1)
    if c["in_place"]:
        place = _keep_places(parent, beams)
        best, rows, token = (torch.zeros_like(v).scatter_(1, place, v)
                             for v in (best, rows, token))
    s["out_scores"].copy_(best)
    s["parents"].copy_(rows)
    s["tokens"].copy_(token)
    return s["out_scores"], s["parents"], s["tokens"]


def _v_places(d, kind):
    """[16, d]: the byte of a V tile that holds token t's code of dim j."""
    t = torch.arange(BLOCK, device="cuda")[:, None]
    j = torch.arange(d, device="cuda")[None]
    r = j % 16
    lane = 4 * (r % 8) + (t % 8) // 2
    if kind == "int4":
        c = j // 16
        swap = (lane // 4) % 2 if d == 128 else 0 * lane
        return lane * (d // 4) + 16 * ((c // 4) ^ swap) + 4 * (c % 4) + t // 8 + 2 * (t % 2)
    w = 2 * (j // 16) + r // 8
    f = (lane // 2) % 4 if d == 128 else (lane // 4) % 2
    return lane * (d // 2) + 16 * ((w // 4) ^ f) + 4 * (w % 4) + t % 2 + 2 * (t // 8)


def _values(pool, scales, d, kind, value_pool):
    """The values that tiles [N, Hkv, ...] of a pool stand for: [N, Hkv, 16, D] in 32 bits."""
    if kind == "bf16":
        return pool.float()
    if kind == "int4":
        if value_pool:
            b = pool[..., _v_places(d, "int4").flatten()].unflatten(-1, (BLOCK, d))
            codes = torch.where(torch.arange(d, device="cuda") % 16 < 8, b & 15, b >> 4)
        else:
            b = pool[..., :8 * d].unflatten(-1, (BLOCK, d // 2))
            j = torch.arange(d, device="cuda")
            e = j % GROUP
            codes = torch.stack([b & 15, b >> 4], -1).flatten(-2)[
                ..., (d // 4) * (e // 16) + e % 16 + 16 * (j // GROUP)]
        par = pool[..., 8 * d:].contiguous().view(torch.bfloat16).float()
        par = par.unflatten(-1, (BLOCK, d // GROUP, 2)).repeat_interleave(GROUP, 3)
        return par[..., 0] + par[..., 1] * codes.float()
    codes = pool.view(torch.uint8)
    if value_pool:
        codes = codes.flatten(-2)[..., _v_places(d, kind).flatten()].unflatten(-1, (BLOCK, d))
        if kind == "int8":
            codes = codes ^ 128
    codes = codes.view(torch.int8 if kind == "int8" else torch.float8_e4m3fn).float()
    return codes * scales[..., None]


def _plain_read(s):
    c = s["case"]
    first, n = _lens(c)
    row = 0
    for b, (f, m) in enumerate(zip(first, n)):
        blocks = s["tables"][b, f // BLOCK:-(-(f + m) // BLOCK)].long()
        skip = f % BLOCK
        for cache, out, scales, vp in ((s["k_cache"], s["k_out"], s.get("k_scales"), False),
                                       (s["v_cache"], s["v_out"], s.get("v_scales"), True)):
            x = _values(cache[blocks], None if scales is None else scales[blocks], c["d"],
                        c["kind"], vp)
            x = x.transpose(1, 2).flatten(0, 1)[skip:skip + m].to(torch.bfloat16)
            if s["slots"] is None:
                out[row:row + m] = x
            else:
                at = s["slots"][row:row + m]
                out[at // BLOCK, :, at % BLOCK] = x
        row += m
    return s["k_out"], s["v_out"]


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
        if op == "cross":
            return state["out"]
        if op == "beam":
            return state["out_scores"], state["parents"], state["tokens"]
        return state["states"] if op == "reorder" else (state["k_out"], state["v_out"])
    if op == "cross":
        return _plain_cross(state)
    if op == "beam":
        return _plain_beam(state)
    if op == "read":
        return _plain_read(state)
    state["states"].copy_(state["states"][:, state["parents"].long()])
    return state["states"]


# ------------------------------------------------- in 64 bits, written apart

def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    if case["op"] == "cross":
        return _exact_cross(case, s)
    if case["op"] == "beam":
        return _exact_beam(case, s)
    if case["op"] == "read":
        return _exact_read(case, s)
    old = [x.clone() for x in s["states"].unbind(1)]
    for i, p in enumerate(_lens(case)[0]):
        s["states"][:, i] = old[p]
    return s["states"]


def _exact_cross(case, s):
    src, new = _lens(case)
    group = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    token = torch.arange(s["tables"].shape[1] * BLOCK, device="cuda")
    row = 0
    for b, (n, m) in enumerate(zip(src, new)):
        where, off = s["tables"][b].long()[token[:n] // BLOCK], token[:n] % BLOCK
        for h in range(case["hq"]) if n else ():
            k, v = (x[where, h // group, off].double() for x in (s["k_cache"], s["v_cache"]))
            w = torch.softmax(s["q"][row:row + m, h].double() @ k.T * s["scale"], -1)
            out[row:row + m, h] = w @ v
        row += m
    return out


def _exact_beam(case, s):
    n, beams, keep = case["searches"], case["beams"], case["keep"]
    logp = torch.log_softmax(s["logits"].double(), -1).nan_to_num(nan=-torch.inf,
                                                                  neginf=-torch.inf)
    scores = torch.full((n, keep), -torch.inf, dtype=torch.float64)
    parents, tokens = (torch.full((n, keep), -1, dtype=torch.int32) for _ in "pt")
    done = s["finished"].tolist() if s["finished"] is not None else [False] * (n * beams)
    for b in range(n):
        found = []  # (total, beam, token)
        for w in range(beams):
            r = b * beams + w
            start = float(s["scores"][r].double())
            if done[r]:
                found.append((start, w, s["eos"]))
                continue
            v, i = torch.sort(logp[r], descending=True, stable=True)
            v, i = v[:keep].tolist(), i[:keep].tolist()
            found += [(start + x, w, t) for x, t in zip(v, i) if x > -math.inf]
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        found = found[:keep]
        place = list(range(keep))
        if case["in_place"]:
            homes, free = set(), set(range(keep))
            for r, f in enumerate(found):
                if f[1] in free:
                    homes.add(r)
                    free.remove(f[1])
                    place[r] = f[1]
            rest = sorted(free)
            for r in range(keep):
                if r not in homes:
                    place[r] = rest.pop(0)
        for r, (x, w, t) in enumerate(found):
            scores[b, place[r]] = x
            parents[b, place[r]], tokens[b, place[r]] = b * beams + w, t
    return scores.cuda(), parents.cuda(), tokens.cuda()


def _exact_read(case, s):
    """Tile by tile: the values of every byte put where they belong."""
    d, kind = case["d"], case["kind"]
    out = []
    for cache, scales, dst, value_pool in ((s["k_cache"], s.get("k_scales"), s["k_out"], False),
                                           (s["v_cache"], s.get("v_scales"), s["v_out"], True)):
        nb, hkv = cache.shape[:2]
        if kind == "bf16":
            x = cache.double()
        elif kind == "int4":
            raw, par = cache[..., :8 * d], cache[..., 8 * d:].contiguous()
            par = par.view(torch.bfloat16).double().view(nb, hkv, BLOCK, -1, 2)
            byte = torch.arange(8 * d, device="cuda")
            x = torch.empty((nb, hkv, BLOCK, d), dtype=torch.float64, device="cuda")
            for high in (0, 1):
                if value_pool:
                    lane, rest = byte // (d // 4), byte % (d // 4)
                    run = rest // 16
                    if d == 128:
                        run = run ^ ((lane // 4) % 2)
                    c = 4 * run + rest % 16 // 4
                    t = 2 * (lane % 4) + 8 * (rest % 2) + rest % 4 // 2
                    j = 16 * c + lane // 4 + 8 * high
                else:
                    t, nib = byte // (d // 2), 2 * (byte % (d // 2)) + high
                    j = nib % (d // 4) // 16 * GROUP + nib // (d // 4) * 16 + nib % 16
                code = (raw // 16 if high else raw % 16).double()
                x[:, :, t, j] = par[:, :, t, j // GROUP, 0] + code * par[:, :, t, j // GROUP, 1]
        else:
            raw = cache.view(torch.uint8)
            if value_pool:
                byte = torch.arange(16 * d, device="cuda")
                lane, rest = byte // (d // 2), byte % (d // 2)
                f = (lane // 2) % 4 if d == 128 else (lane // 4) % 2
                w = 4 * ((rest // 16) ^ f) + rest % 16 // 4
                t = 2 * (lane % 4) + rest % 2 + 8 * (rest % 4 // 2)
                j = 16 * (w // 2) + lane // 4 + 8 * (w % 2)
                placed = torch.empty_like(raw)
                placed[:, :, t, j] = raw.flatten(-2)
                raw = placed
            if kind == "int8":
                x = raw.double() - 128 if value_pool else raw.view(torch.int8).double()
            else:
                low, e = (raw % 8).double(), (raw // 8 % 16).double()
                x = torch.where(e > 0, (8 + low) * torch.exp2(e - 10), low * 2.0 ** -9)
                x = torch.where(raw >= 128, -x, x)
            x = x * scales.double()[..., None]
        rows = []
        for b, (f, m) in enumerate(zip(*_lens(case))):
            p = torch.arange(f, f + m, device="cuda")
            rows.append(x[s["tables"][b].long()[p // BLOCK], :, p % BLOCK])
        x, rows = None, torch.cat(rows)
        if s["slots"] is None:
            out.append(rows)
        else:
            y = torch.zeros(dst.shape, dtype=torch.float64, device="cuda")
            y[s["slots"] // BLOCK, :, s["slots"] % BLOCK] = rows
            out.append(y)
    return tuple(out)


# ------------------------------------------------------------------- the work

def work(case):
    if case["op"] == "cross":
        src, new = _lens(case)
        hkv, d, hq = case["hkv"], case["d"], case["hq"]
        keys = sum(n for n, m in zip(src, new) if m)
        return {"bytes": keys * 2 * hkv * 2 * d + 2 * sum(new) * hq * d * 2 +
                4 * sum(-(-n // BLOCK) for n in src),
                "flops": 4 * sum(n * m for n, m in zip(src, new)) * hq * d}
    if case["op"] == "beam":
        rows = case["searches"] * case["beams"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * (case["vocab"] * size + 5) + case["searches"] * case["keep"] * 12,
                "flops": 3 * rows * case["vocab"]}
    if case["op"] == "reorder":
        moved = [(i, p) for i, p in enumerate(_lens(case)[0]) if i != p]
        size = case["layers"] * case["row"] * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": (len(moved) + len({p for _, p in moved})) * size +
                4 * case["searches"] * case["beams"], "flops": 0}
    rows, d = sum(_lens(case)[1]), case["d"]
    row = {"bf16": 2 * d, "int8": d + 4, "fp8": d + 4, "int4": 9 * d // 16}[case["kind"]]
    return {"bytes": rows * 2 * case["hkv"] * (row + 2 * d) + rows * (8 if case["to_slots"]
                                                                      else 0),
            "flops": 2 * rows * case["hkv"] * d}
