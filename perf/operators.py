"""Cases of the operators over the paged KV cache: what they compute in plain
torch operations, and the calls a user makes of the library for the same.

Operators:
  append    rotary position embedding of the new tokens' q and k, and the
            write of their k and v into the paged cache (bf16, INT8, FP8 or
            4-bit pools)
  decode4   one-query attention over a paged cache held in 4 bits
  step      one-query attention over a bf16 paged cache whose scores are
            capped by a tanh, biased by distance or limited to a window
  prefill   the same for chunks of new tokens, with a bidirectional prefix

``own`` chooses the side: False, elementary torch operations in 32 bits; True,
the library's calls.  Sizes follow the library's own workloads (32 query / 8
KV heads of 128 dims, blocks of 16 tokens) and other shapes it supports.
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
        # one decode step's new tokens, 64 sequences: a latency-bound call
        {"name": "append_decode_64", "op": "append", "kind": "bf16", "tokens": 64, "seqs": 64,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False, "fused_qkv": False,
         "padding": 0, "max_pos": 8192, "lens": 1},
        # an 8192-token chunked-prefill step, q / k / v slices of one projection
        {"name": "append_prefill_8192", "op": "append", "kind": "bf16", "tokens": 8192,
         "seqs": 16, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False,
         "fused_qkv": True, "padding": 0, "max_pos": 8192, "lens": 2},
        # a ragged batch into a 4-bit cache: interleaved pairs, half of the
        # dims rotated, padding tokens, far positions
        {"name": "append_int4_1009", "op": "append", "kind": "int4", "tokens": 1009, "seqs": 5,
         "hq": 16, "hkv": 4, "d": 128, "rot": 64, "interleaved": True, "fused_qkv": False,
         "padding": 23, "max_pos": 131072, "lens": 3},
        # the smallest decode: one sequence of 4 query heads
        {"name": "decode4_one", "op": "decode4", "seqs": 1, "hq": 4, "hkv": 2, "d": 64,
         "ctx_lo": 37, "ctx_hi": 37, "lens": 4},
        # an ordinary serving batch: contexts of 128 to 2048 tokens
        {"name": "decode4_batch64", "op": "decode4", "seqs": 64, "hq": 32, "hkv": 8, "d": 128,
         "ctx_lo": 128, "ctx_hi": 2048, "lens": 5},
        # a large batch of short and ragged contexts, 8 query heads a KV head
        {"name": "decode4_batch256_g8", "op": "decode4", "seqs": 256, "hq": 64, "hkv": 8,
         "d": 128, "ctx_lo": 1, "ctx_hi": 4096, "lens": 6},
        # long contexts, where keeping the cache in 4 bits matters most
        {"name": "decode4_long", "op": "decode4", "seqs": 8, "hq": 32, "hkv": 8, "d": 128,
         "ctx_lo": 8192, "ctx_hi": 131072, "lens": 7},
        # capped scores and a sliding window over an ordinary batch
        {"name": "step_cap_window", "op": "step", "seqs": 64, "hq": 32, "hkv": 8, "d": 128,
         "ctx_lo": 128, "ctx_hi": 8192, "cap": 50.0, "window": 1024, "alibi": False, "lens": 8},
        # a distance bias over long contexts, narrow heads
        {"name": "step_alibi_long", "op": "step", "seqs": 7, "hq": 32, "hkv": 16, "d": 64,
         "ctx_lo": 1000, "ctx_hi": 65536, "cap": 0.0, "window": 0, "alibi": True, "lens": 9},
        # the smallest prefill: one short prompt, whole
        {"name": "prefill_small", "op": "prefill", "seqs": 1, "hq": 8, "hkv": 2, "d": 128,
         "q_lo": 37, "q_hi": 37, "prior_hi": 0, "cap": 30.0, "window": 0, "alibi": True,
         "prefix_hi": 0, "lens": 10},
        # a ragged batch whose prompts open with a bidirectional prefix
        {"name": "prefill_prefix_ragged", "op": "prefill", "seqs": 9, "hq": 32, "hkv": 4,
         "d": 128, "q_lo": 1, "q_hi": 700, "prior_hi": 900, "cap": 0.0, "window": 1000,
         "alibi": True, "prefix_hi": 600, "lens": 11},
        # an 8192-token chunked-prefill step with capped scores
        {"name": "prefill_cap_16x512", "op": "prefill", "seqs": 16, "hq": 32, "hkv": 8, "d": 128,
         "q_lo": 512, "q_hi": 512, "prior_hi": 3584, "cap": 50.0, "window": 0, "alibi": False,
         "prefix_hi": 0, "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode4", "step", "prefill"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    lens = rng.randrange(1 << 20)
    if op == "append":
        tokens = _log_int(rng, 1, 8192)
        return {"op": op, "kind": rng.choice(["bf16", "int8", "fp8", "int4"]), "tokens": tokens,
                "seqs": _log_int(rng, 1, tokens), "hq": min(hkv, 8) * rng.choice([1, 2, 4]),
                "hkv": min(hkv, 8), "d": d, "rot": rng.choice([d, d, 32]),
                "interleaved": rng.random() < 0.5, "fused_qkv": rng.random() < 0.5,
                "padding": rng.choice([0, tokens // 7]), "max_pos": 131072, "lens": lens}
    group = rng.choice([2, 4, 8])
    hi = _log_int(rng, 1, 32768)
    lo = _log_int(rng, 1, hi)
    budget = 400000 * 8 // (hkv * max(group, 4) // 4)  # (tokens x KV heads), as the long batch
    seqs = min(_log_int(rng, 1, 256), max(1, budget // hi))
    if op == "decode4":
        return {"op": op, "seqs": seqs, "hq": hkv * group, "hkv": hkv, "d": d, "ctx_lo": lo,
                "ctx_hi": hi, "lens": lens}
    cap = rng.choice([0.0, 30.0, 50.0])
    alibi = rng.random() < 0.5
    window = rng.choice([0, _log_int(rng, 1, 8192)])
    if op == "step":
        seqs = max(1, seqs // 2)
        return {"op": op, "seqs": seqs, "hq": hkv * group, "hkv": hkv, "d": d, "ctx_lo": lo,
                "ctx_hi": hi, "cap": cap, "window": window, "alibi": alibi, "lens": lens}
    group = rng.choice([1, 2, 4, 8])
    hkv = min(hkv, 32 // group)
    q_hi = _log_int(rng, 1, 512)
    return {"op": op, "seqs": _log_int(rng, 1, 16), "hq": hkv * group, "hkv": hkv, "d": 128,
            "q_lo": _log_int(rng, 1, q_hi), "q_hi": q_hi, "prior_hi": rng.choice([0, 100, 3000]),
            "cap": cap, "window": window, "alibi": alibi, "prefix_hi": rng.choice([0, 700]),
            "lens": lens}


def _lens(case):
    """The sequences' lengths, from the case alone: (context lengths, new tokens, prefixes)."""
    rng = random.Random(case["lens"])
    if case["op"] == "append":
        n = case["tokens"] - case["padding"]
        seqs = max(1, min(case["seqs"], n))
        cuts = sorted(rng.sample(range(1, n), seqs - 1)) if seqs > 1 else []
        new = [b - a for a, b in zip([0] + cuts, cuts + [n])]
        prior = [rng.randrange(0, min(case["max_pos"], 16384) - m + 1) if m < 16384 else 0
                 for m in new]
        return [p + m for p, m in zip(prior, new)], new, []
    if case["op"] == "prefill":
        new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
        ctx = [n + rng.randint(0, case["prior_hi"]) for n in new]
        pre = [rng.randint(0, min(case["prefix_hi"], c)) for c in ctx]
        return ctx, new, pre
    ctx = [_log_int(rng, case["ctx_lo"], case["ctx_hi"]) if case["ctx_hi"] > 8 * case["ctx_lo"]
           and case["ctx_lo"] >= 1000 else rng.randint(case["ctx_lo"], case["ctx_hi"])
           for _ in range(case["seqs"])]
    return ctx, [1] * len(ctx), []


# --------------------------------------------------------------- the inputs

def _tables(ctx, hkv, gen):
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


def _pool4(nb, hkv, d, gen):
    """A 4-bit pool: codes, and per token and group an offset near the least
    value and a scale near a fifteenth of the range of normal values."""
    codes = torch.randint(0, 256, (nb, hkv, 8 * d), generator=gen, device="cuda",
                          dtype=torch.uint8)
    n = (nb, hkv, BLOCK * d // GROUP)
    lo = (-2.4 + 0.3 * torch.randn(n, generator=gen, device="cuda")).to(torch.bfloat16)
    sc = (0.32 + 0.04 * torch.randn(n, generator=gen, device="cuda")).abs().to(torch.bfloat16)
    par = torch.stack([lo, sc], -1).view(torch.uint8).reshape(nb, hkv, -1)
    return torch.cat([codes, par], -1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new, prefix = _lens(case)
    hkv, d, hq = case["hkv"], case["d"], case["hq"]
    tables, nb = _tables(ctx, hkv, gen)
    dev = {"device": "cuda"}
    s = {"case": case, "tables": tables, "ctx": torch.tensor(ctx, dtype=torch.int32, **dev)}
    if case["op"] == "append":
        T, pad = case["tokens"], case["padding"]
        if case["fused_qkv"]:
            qkv = _normal((T, hq + 2 * hkv, d), gen)
            s["q"], s["key"], s["value"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["key"], s["value"] = (_normal((T, h, d), gen) for h in (hq, hkv, hkv))
        n = torch.tensor(new, **dev)
        seq = torch.repeat_interleave(torch.arange(len(new), **dev), n)
        first = s["ctx"].long() - n
        pos = first[seq] + torch.arange(T - pad, **dev) - (torch.cumsum(n, 0) - n)[seq]
        slot = tables[seq, pos // BLOCK].long() * BLOCK + pos % BLOCK
        s["slots"] = torch.cat([slot, torch.full((pad,), -1, **dev)])
        s["positions"] = torch.cat([pos, torch.zeros(pad, dtype=torch.long, **dev)]).to(
            torch.int32)
        half = case["rot"] // 2
        freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, **dev) / half)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, **dev)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["q_out"] = torch.zeros((T, hq, d), dtype=torch.bfloat16, **dev)
        kind = case["kind"]
        if kind == "bf16":
            s["k_cache"], s["v_cache"] = (_normal((nb, hkv, BLOCK, d), gen) for _ in "kv")
        elif kind == "int4":
            s["k_cache"], s["v_cache"] = (_pool4(nb, hkv, d, gen) for _ in "kv")
        else:
            t = torch.int8 if kind == "int8" else torch.uint8
            s["k_cache"], s["v_cache"] = (
                torch.randint(0, 100, (nb, hkv, BLOCK, d), generator=gen, dtype=t, **dev)
                for _ in "kv")
            s["k_scales"], s["v_scales"] = (
                torch.rand((nb, hkv, BLOCK), generator=gen, **dev) for _ in "kv")
    else:
        T = sum(new)
        s["q"] = _normal((T, hq, d), gen)
        s["out"] = torch.zeros((T, hq, d), dtype=torch.bfloat16, **dev)
        s["scale"] = 1.0 / math.sqrt(d)
        make = _pool4 if case["op"] == "decode4" else lambda *a: _normal((nb, hkv, BLOCK, d), gen)
        s["k_cache"], s["v_cache"] = make(nb, hkv, d, gen), make(nb, hkv, d, gen)
        s["slopes"] = None
        if case.get("alibi"):
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, **dev) / hq)
        s["prefix"] = torch.tensor(prefix, dtype=torch.int32, **dev) \
            if case.get("prefix_hi") else None
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, **dev)
        s["max_new"] = max(new)
    if own:
        s["call"] = _handle(case, s, ctx)
    return s


def _handle(case, s, ctx):
    """The library's handle of one call on these buffers, as a serving program keeps it."""
    from paged_kv_cache_283_gb300 import pa
    if case["op"] == "append":
        return pa.RopeAppend(s["q_out"], s["q"], s["key"], s["value"], s["k_cache"],
                             s["v_cache"], s["slots"], s["positions"], s["cos_sin"],
                             interleaved=case["interleaved"], k_scales=s.get("k_scales"),
                             v_scales=s.get("v_scales"))
    rule = {} if case["op"] == "decode4" else {
        "softcap": case["cap"], "window": case["window"], "alibi_slopes": s["slopes"]}
    if case["op"] == "prefill":
        return pa.PrefillStep(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"],
                              s["ctx"], s["starts"], s["max_new"], s["scale"],
                              prefix_lens=s["prefix"], **rule)
    return pa.DecodeStep(None, None, s["k_cache"], s["v_cache"], None, s["q"], s["tables"],
                         s["ctx"], s["out"], s["scale"], partition_size=None,
                         host_context_lens=ctx, early_read=True, **rule)


# ------------------------------------------------------------ the plain form

def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] in 32 bits, its first `rot` dims rotated; cos / sin [T, rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else \
        (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([r, x[..., rot:]], -1)


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


def _k_places(d):
    """[d]: the nibble of a 4-bit K row that holds dim j's code."""
    j = torch.arange(d, device="cuda")
    e = j % GROUP
    return (d // 4) * (e // 16) + e % 16 + 16 * (j // GROUP)


def _quantise4(x):
    """x [T, H, D] in 32 bits: codes [T, H, D] and parameter bytes [T, H, D / 64 * 4]."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    sc = ((hi - lo) / 15.0).to(torch.bfloat16).float()
    codes = torch.where(sc > 0, torch.round((g - lo) / sc).clamp(0, 15), 0.0)
    par = torch.stack([lo.squeeze(-1).to(torch.bfloat16), sc.squeeze(-1).to(torch.bfloat16)], -1)
    return codes.flatten(-2).to(torch.uint8), par.view(torch.uint8).flatten(-2)


def _plain_append(s):
    c = s["case"]
    half = c["rot"] // 2
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, :half], cs[:, half:]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]))
    key = _rotate(s["key"].float(), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
    put = s["slots"] >= 0
    slot = s["slots"][put]
    key, value = key[put], s["value"][put]
    blk, off = slot // BLOCK, slot % BLOCK
    h = torch.arange(c["hkv"], device="cuda")
    at = (blk[:, None], h[None], off[:, None])
    kind, d = c["kind"], c["d"]
    if kind == "bf16":
        s["k_cache"][at], s["v_cache"][at] = key, value
        return s["q_out"], s["k_cache"], s["v_cache"]
    key, value = key.float(), value.float()
    tile = (blk[:, None, None], h[None, :, None])
    if kind == "int4":
        kc, kp = _quantise4(key)
        vc, vp = _quantise4(value)
        row = kc[..., torch.argsort(_k_places(d))]
        byte = torch.arange(d // 2, device="cuda")
        s["k_cache"][(*tile, (off[:, None] * (d // 2) + byte)[:, None])] = \
            row[..., 0::2] | (row[..., 1::2] << 4)
        pair = vc.unflatten(-1, (d // 16, 2, 8))
        places = _v_places(d, kind)[off].unflatten(-1, (d // 16, 2, 8))[:, :, 0].flatten(-2)
        s["v_cache"][(*tile, places[:, None])] = (pair[..., 0, :] | (pair[..., 1, :] << 4)
                                                  ).flatten(-2)
        n = d // GROUP * 4
        par = (8 * d + off[:, None] * n + torch.arange(n, device="cuda"))[:, None]
        s["k_cache"][(*tile, par)], s["v_cache"][(*tile, par)] = kp, vp
        return s["q_out"], s["k_cache"], s["v_cache"]
    top = 127.0 if kind == "int8" else 448.0
    ks, vs = key.abs().amax(-1) / top, value.abs().amax(-1) / top
    k, v = (torch.where(sc[..., None] > 0, x / sc[..., None], 0.0)
            for x, sc in ((key, ks), (value, vs)))
    if kind == "int8":
        k, v = (torch.round(x).clamp(-127, 127).to(torch.int8) for x in (k, v))
        v = (v.view(torch.uint8) ^ 128).view(torch.int8)
    else:
        k, v = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    s["k_cache"][at] = k
    s["v_cache"].flatten(-2)[(*tile, _v_places(d, kind)[off][:, None])] = v
    s["k_scales"][at], s["v_scales"][at] = ks, vs
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _values4(pool, d, value_pool):
    """The values a 4-bit pool's bytes stand for: [NB, Hkv, 16, D] in 32 bits."""
    nb, hkv = pool.shape[:2]
    if value_pool:
        b = pool[..., _v_places(d, "int4").flatten()].unflatten(-1, (BLOCK, d))
        codes = torch.where(torch.arange(d, device="cuda") % 16 < 8, b & 15, b >> 4)
    else:
        b = pool[..., :8 * d].unflatten(-1, (BLOCK, d // 2))
        codes = torch.stack([b & 15, b >> 4], -1).flatten(-2)[..., _k_places(d)]
    par = pool[..., 8 * d:].contiguous().view(torch.bfloat16).float()
    par = par.view(nb, hkv, BLOCK, d // GROUP, 2).repeat_interleave(GROUP, 3)
    return par[..., 0] + par[..., 1] * codes.float()


def _plain_attention(s):
    """Attention of every sequence's new tokens over its blocks, padded to the
    longest context and the most new tokens."""
    c = s["case"]
    hkv, d, hq = c["hkv"], c["d"], c["hq"]
    ctx, starts = s["ctx"].long(), s["starts"].long()
    blocks = s["tables"].long().clamp(min=0)
    n_ctx = blocks.shape[1] * BLOCK
    k, v = s["k_cache"], s["v_cache"]
    k, v = k[blocks], v[blocks]                      # [B, MB, Hkv, ...]
    if c["op"] == "decode4":
        k, v = (_values4(x.flatten(0, 1), d, i == 1).view(*blocks.shape, hkv, BLOCK, d)
                for i, x in enumerate((k, v)))
    k, v = (x.float().transpose(1, 2).reshape(len(ctx), hkv, n_ctx, d) for x in (k, v))
    n = starts[1:] - starts[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    there = i < n[:, None]                           # [B, M]
    row = torch.where(there, starts[:-1, None] + i, 0)
    q = s["q"][row].float().view(len(ctx), s["max_new"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (hq // hkv, -1))
    x = x * s["scale"]                               # [B, Hkv, G, M, N]
    if c.get("cap"):
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = (ctx - n)[:, None] + i                     # [B, M]
    j = torch.arange(n_ctx, device="cuda")
    away = (pos[..., None] - j)[:, None, None]       # [B, 1, 1, M, N]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(hkv, -1, 1, 1) * away.abs()
    seen = away >= 0
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][:, None, None, None, None])
    if c.get("window"):
        seen = seen & (away < c["window"])
    x = torch.where(seen, x, -torch.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = torch.where((j < ctx[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.flatten(2, 3), v).view(len(ctx), hq, s["max_new"], d).transpose(1, 2)
    s["out"][row[there]] = o[there].to(torch.bfloat16)
    return s["out"]


def run(state):
    if own:
        state["call"]()
        if state["case"]["op"] != "append":
            return state["out"]
        # pools of codes come as they are stored (whole numbers: equal or not)
        more = (state["k_scales"], state["v_scales"]) if "k_scales" in state else ()
        return (state["q_out"], state["k_cache"], state["v_cache"]) + more
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


# ------------------------------------------------- in 64 bits, written apart

def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "prefill" and case["seqs"] * case["hq"] * case["q_hi"] > 1 << 19:
        return None
    return _exact_attention(case, s)


def _exact_append(case, s):
    half, T = case["rot"] // 2, case["tokens"]
    freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    turn = torch.polar(torch.ones_like(freq), s["positions"].double()[:, None] * freq)

    def spin(x):
        x = x.double()
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = spin(s["q"])
    if case["kind"] != "bf16":
        return (q, None, None) + ((None, None) if case["kind"] != "int4" else ())
    k, v = s["k_cache"].double(), s["v_cache"].double()
    key = spin(s["key"])
    slots = s["slots"].tolist()
    real = [t for t in range(T) if slots[t] >= 0]
    blk = torch.tensor([slots[t] // BLOCK for t in real], device="cuda")
    off = torch.tensor([slots[t] % BLOCK for t in real], device="cuda")
    t = torch.tensor(real, device="cuda")
    k[blk, :, off], v[blk, :, off] = key[t], s["value"][t].double()
    return q, k, v


def _exact_values4(tiles, d, transposed):
    """Tiles [n, Hkv, 9 d] of a 4-bit pool as [n * 16, Hkv, d] values."""
    n, hkv, _ = tiles.shape
    out = torch.empty((n, hkv, BLOCK, d), dtype=torch.float64, device="cuda")
    par = tiles[..., 8 * d:].contiguous().view(torch.bfloat16).double().view(
        n, hkv, BLOCK, d // GROUP, 2)
    for j in range(d):
        if transposed:
            lane = [4 * (j % 8) + (t % 8) // 2 for t in range(BLOCK)]
            word = [(j // 64) ^ ((x // 4) % 2 if d == 128 else 0) for x in lane]
            at = [lane[t] * (d // 4) + 16 * word[t] + 4 * ((j // 16) % 4) + t // 8 + 2 * (t % 2)
                  for t in range(BLOCK)]
            high = j % 16 >= 8
        else:
            nib = (d // 4) * (j % 64 // 16) + j % 16 + 16 * (j // 64)
            at = [t * (d // 2) + nib // 2 for t in range(BLOCK)]
            high = nib % 2 == 1
        b = tiles[..., at].int()
        code = (b // 16 if high else b % 16).double()
        out[..., j] = par[..., j // 64, 0] + par[..., j // 64, 1] * code
    return out.transpose(1, 2).reshape(n * BLOCK, hkv, d)


def _exact_attention(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ctx, new, prefix = _lens(case)
    out = torch.zeros((sum(new), hq, d), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        blk = s["tables"][b, :-(-n // BLOCK)].long()
        if case["op"] == "decode4":
            K, V = (_exact_values4(s[x][blk], d, x == "v_cache") for x in ("k_cache", "v_cache"))
        else:
            K, V = (s[x][blk].double().transpose(1, 2).reshape(-1, hkv, d)
                    for x in ("k_cache", "v_cache"))
        K, V = K[:n], V[:n]
        q = s["q"][at:at + m].double()
        p = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        hidden = j > p
        if s["prefix"] is not None:
            hidden = hidden & (j >= prefix[b])
        if case.get("window"):
            hidden = hidden | (j <= p - case["window"])
        for h in range(hq):
            x = (q[:, h] @ K[:, h * hkv // hq].T) * s["scale"]
            if case.get("cap"):
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                x = x - s["slopes"][h].double() * (p - j).abs()
            x = x.masked_fill(hidden, -math.inf)
            out[at:at + m, h] = torch.softmax(x, -1) @ V[:, h * hkv // hq]
        at += m
    return out


# ------------------------------------------------------------------ the work

def work(case):
    """Bytes and operations no implementation can do without: inputs read and
    outputs written once; two operations per multiply-add of the products."""
    ctx, new, prefix = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        T, put = case["tokens"], case["tokens"] - case["padding"]
        row = {"bf16": 2 * d, "int8": d + 4, "fp8": d + 4, "int4": 9 * d // 16}[case["kind"]]
        read = T * (hq * d * 2 + 4 + 8 + case["rot"] * 4) + put * 2 * hkv * d * 2
        return {"bytes": read + T * hq * d * 2 + put * 2 * hkv * row,
                "flops": 3 * T * (hq + hkv) * case["rot"]}
    row = 9 * d // 16 if case["op"] == "decode4" else 2 * d
    window = case.get("window") or 1 << 40
    keys = pairs = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        keys += min(n, window + m - 1)
        pre = prefix[b] if case.get("prefix_hi") else 0
        for p in range(n - m, n):
            pairs += max(p + 1, pre) - max(0, p + 1 - window)
    return {"bytes": keys * 2 * hkv * row + 2 * sum(new) * hq * d * 2 +
            4 * sum(-(-n // BLOCK) for n in ctx), "flops": 4 * pairs * hq * d}
