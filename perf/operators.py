"""Timed cases of the block-summary, block-sparse decode, attention-mass and
cache-eviction operators over the paged, DCP-sharded MLA latent cache.

A case is one rank's call on its shard of the cache.  Rows are 576 values: 512
latent and 64 rope, as 576 bf16 (1,152 bytes) or as 512 e4m3 codes, four fp32
scales and 64 bf16 (656 bytes), in blocks of 64 rows behind a block table.
``run`` computes a case in elementary torch operations, or, where ``own`` is
true, through this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK, ROW, LATENT, ROPE = 64, 576, 512, 64
ROW_BYTES = {"bf16": 1152, "fp8": 656}
SUMMARY_BYTES = 608                     # 576 int8 codes, 5 fp32 scales, 12 bytes of padding
GROUPS = (0, 128, 256, 384, 512, 576)   # scale groups of a summary: four latent, one rope
SCALE = 192 ** -0.5
DEV = "cuda"


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a finished prefill of the dense workload: one of eight shards summarises its blocks
        dict(name="summary dense bf16", op="summary", kv="bf16", batch=32, lens="even", length=8192, shards=8,
             shard=3, step=False, len_seed=1),
        # the agentic length mix (median 67K tokens) after prefill, one of eight shards, fp8 rows
        dict(name="summary agentic fp8", op="summary", kv="fp8", batch=64, lens="lognormal", length=67000, shards=8,
             shard=0, step=False, len_seed=1003),
        # one decode step: only the block that took the new token is summarised again
        dict(name="summary step fp8", op="summary", kv="fp8", batch=64, lens="lognormal", length=16000, shards=1,
             shard=0, step=True, len_seed=7),
        # the smallest call: one request of 8 heads on one of two shards, where latency counts
        dict(name="blocks tiny bf16", op="blocks", kv="bf16", batch=1, heads=8, q_len=1, lens="even", length=1024,
             shards=2, shard=0, topk=4, len_seed=1),
        # 64K-token requests on one GPU, 2,048 of the rows read per step
        dict(name="blocks 64k fp8", op="blocks", kv="fp8", batch=64, heads=64, q_len=1, lens="even", length=65536,
             shards=1, shard=0, topk=32, len_seed=1),
        # speculative verification: four draft tokens of 16 heads, each with blocks of its own, ragged lengths
        dict(name="blocks draft bf16", op="blocks", kv="bf16", batch=12, heads=16, q_len=4, lens="lognormal",
             length=20000, shards=1, shard=0, topk=24, len_seed=3),
        # one million-token request, its blocks chosen among 16,384
        dict(name="blocks million fp8", op="blocks", kv="fp8", batch=1, heads=64, q_len=1, lens="even",
             length=1 << 20, shards=1, shard=0, topk=64, len_seed=1),
        # the smallest call of the accumulated weights
        dict(name="mass tiny bf16", op="mass", kv="bf16", batch=1, heads=8, q_len=1, lens="even", length=1024,
             shards=2, shard=1, decay=1.0, len_seed=1),
        # the agentic mix, one of eight shards, 64 heads, fp8 rows
        dict(name="mass agentic fp8", op="mass", kv="fp8", batch=64, heads=64, q_len=1, lens="lognormal",
             length=67000, shards=8, shard=5, decay=1.0, len_seed=1003),
        # draft tokens over bf16 rows: four causal queries of 16 heads, older weight fading
        dict(name="mass draft bf16", op="mass", kv="bf16", batch=32, heads=16, q_len=4, lens="even", length=8191,
             shards=1, shard=0, decay=0.97, len_seed=1),
        # steady state of decode: 64 rows over the budget are dropped from each request
        dict(name="evict step fp8", op="evict", kv="fp8", batch=64, lens="even", length=2112, shards=1, shard=0,
             budget=2048, sink=4, recent=256, len_seed=1),
        # after prefill: each shard of long prompts is cut to its budget
        dict(name="evict prompt bf16", op="evict", kv="bf16", batch=24, lens="lognormal", length=67000, shards=4,
             shard=2, budget=8192, sink=4, recent=2048, len_seed=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["summary", "blocks", "mass", "evict"])
    kv = rng.choice(["bf16", "fp8"])
    shards = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, kv=kv, batch=_log(rng, 1, 64), lens=rng.choice(["even", "lognormal"]), shards=shards,
             shard=rng.randrange(shards), len_seed=rng.randrange(1 << 20))
    # at most about 300 MB of this shard's rows, well below the largest listed cases
    c["length"] = max(1, min(_log(rng, 700, 262144), 300_000_000 * shards // (c["batch"] * ROW_BYTES[kv] * 2)))
    if op == "summary":
        c["step"] = rng.random() < 0.3
        if c["step"]:       # a shard that took the first request's token
            c["shard"] = (_lengths(c)[0] - 1) % shards
    if op in ("blocks", "mass"):
        c["heads"] = rng.choice([1, 8, 16, 24, 37, 64])
        c["q_len"] = rng.choice([1, 1, 2, 3]) if c["heads"] <= 16 else 1
    if op == "blocks":
        c["topk"] = _log(rng, 3, 64)
    if op == "mass":
        c["decay"] = rng.choice([0.0, 0.9, 1.0])
    if op == "evict":
        local = max(1, c["length"] // shards)
        c["budget"] = max(8, int(local * rng.uniform(0.2, 1.1)))
        c["sink"] = rng.choice([0, 1, 4])
        c["recent"] = rng.randrange(0, c["budget"] - c["sink"] + 1)
    return c


def _lengths(case):
    """Global lengths: all alike, or a lognormal mix around the case's length (sigma 1, an eighth to thrice it)."""
    if case["lens"] == "even":
        return [case["length"]] * case["batch"]
    rng, L = random.Random(case["len_seed"]), case["length"]
    return [max(1, min(3 * L, max(L // 8, int(L * math.exp(rng.gauss(0, 1)))))) for _ in range(case["batch"])]


def _local(L, s, n):
    return (L - s - 1) // n + 1 if L > s else 0


def _rows(case):
    return [_local(L, case["shard"], case["shards"]) for L in _lengths(case)]


def _visible(case):
    """This shard's rows that each (request, query) sees: query i sits at position L - q_len + i."""
    n, s, q = case["shards"], case["shard"], case["q_len"]
    return [_local(max(0, L - q + 1 + i), s, n) for L in _lengths(case) for i in range(q)]


def work(case):
    rb, rows = ROW_BYTES[case["kv"]], _rows(case)
    if case["op"] == "summary":
        if case["step"]:
            hit = [r for L, r in zip(_lengths(case), rows) if (L - 1) % case["shards"] == case["shard"]]
            read = sum((r - 1) % BLOCK + 1 for r in hit)
            blocks = len(hit)
        else:
            read, blocks = sum(rows), sum(-(-r // BLOCK) for r in rows)
        return {"bytes": read * rb + blocks * (596 + 4) + 4 * len(rows), "flops": read * ROW * 2}
    H, Q = case.get("heads", 0), case.get("q_len", 0)
    if case["op"] == "blocks":
        k, vis = case["topk"], _visible(case)
        nb = [-(-r // BLOCK) for r in rows]
        read = sum(min(v, k * BLOCK) for v in vis)
        scored = sum(-(-v // BLOCK) for v in vis)
        return {"bytes": len(vis) * H * (ROW * 2 + LATENT * 2 + 4) + sum(nb) * (596 + 4) + read * rb + len(vis) * k * 4,
                "flops": scored * H * ROW * 2 + read * H * (ROW + LATENT) * 2}
    if case["op"] == "mass":
        return {"bytes": sum(rows) * (rb + (8 if case["decay"] else 4)) + len(rows) * Q * H * (ROW * 2 + 4),
                "flops": sum(rows) * Q * H * ROW * 2}
    moved = sum(max(0, r - case["budget"]) * (case["budget"] / r) for r in rows if r)
    kept = sum(min(r, case["budget"]) for r in rows)
    return {"bytes": sum(rows) * 4 + kept * 8 + moved * 2 * rb, "flops": sum(rows) * 4}


# ----------------------------------------------------------------- inputs ----

def _quantise_rows(x):
    """fp32 [n, 576] -> 656-byte rows."""
    n = x.shape[0]
    g = x[:, :LATENT].view(n, 4, 128)
    amax = g.abs().amax(2)
    sc = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    out = torch.empty(n, 656, dtype=torch.uint8, device=x.device)
    out[:, :512] = (g / sc[:, :, None]).to(torch.float8_e4m3fn).view(n, LATENT).view(torch.uint8)
    out[:, 512:528] = sc.view(torch.uint8)
    out[:, 528:] = x[:, LATENT:].to(torch.bfloat16).view(torch.uint8)
    return out


def _pool(blocks, kv, g):
    """A pool of rows that lean towards a direction of their block, so that blocks differ in what they hold."""
    pool = torch.empty(blocks, BLOCK, ROW_BYTES[kv], dtype=torch.uint8, device=DEV)
    for b0 in range(0, blocks, 4096):
        n = min(4096, blocks - b0)
        x = torch.randn(n, BLOCK, ROW, generator=g, device=DEV)
        x += 0.5 * torch.randn(n, 1, ROW, generator=g, device=DEV)
        x = x.view(n * BLOCK, ROW)
        r = _quantise_rows(x) if kv == "fp8" else x.to(torch.bfloat16).view(torch.uint8)
        pool[b0:b0 + n] = r.view(n, BLOCK, -1)
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens, rows, B = _lengths(case), _rows(case), case["batch"]
    nb = [-(-r // BLOCK) for r in rows]
    most, total = max(1, max(nb)), max(1, sum(nb))
    perm = torch.randperm(total, generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros(B, most, dtype=torch.int32, device=DEV)
    used = torch.arange(most, device=DEV)[None] < torch.tensor(nb, device=DEV)[:, None]
    table[used] = perm[:sum(nb)]
    s = dict(case=case, cache=_pool(total, case["kv"], g), table=table, rows=rows,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    op = case["op"]
    if op == "summary":
        s["summaries"] = torch.zeros(total, SUMMARY_BYTES, dtype=torch.uint8, device=DEV)
        s["first"] = s["lens"] - 1 if case["step"] else None
        s["written"] = None
        if case["step"]:            # the blocks that hold the requests' last tokens, where this shard has them
            b = [i for i, L in enumerate(lens) if (L - 1) % case["shards"] == case["shard"]]
            k = [nb[i] - 1 for i in b]
            s["written"] = table[b, k].long()
        s["values"] = torch.empty(total if s["written"] is None else len(s["written"]), ROW, dtype=torch.bfloat16,
                                  device=DEV)
    if op in ("blocks", "mass"):
        q = torch.randn(B, case["q_len"], case["heads"], ROW, generator=g, device=DEV)
        s["q"] = (q * (0.5 + torch.rand(B, case["q_len"], case["heads"], 1, generator=g, device=DEV))).to(torch.bfloat16)
    if op == "blocks":
        s["summaries"] = torch.zeros(total, SUMMARY_BYTES, dtype=torch.uint8, device=DEV)
        _summaries(s, s["summaries"])
    if op == "mass":
        # weight gathered so far, of the size of what a few more queries bring
        s["mass"] = torch.rand(B, most * BLOCK, generator=g, device=DEV)
        s["mass"] *= 4 * case["q_len"] * case["heads"] / torch.tensor(lens, device=DEV)[:, None]
        # the weights' log-sum over all shards, as the merge gives it: here every shard weighs like this one
        lse = torch.empty(B, case["q_len"] * case["heads"], device=DEV)
        for b in range(B):
            sc = _scores(s, b, torch.float32)
            lse[b] = torch.logsumexp(sc, 1) + math.log(case["shards"])
        s["lse"] = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse)).view(B, case["q_len"], case["heads"])
    if op == "evict":
        n = most * BLOCK
        s["mass"] = torch.empty(B, n, device=DEV).exponential_(generator=g) ** 2
        s["mass"] *= torch.rand(B, n, generator=g, device=DEV) > 0.1        # weights of exactly zero among them
        s["mass_out"] = torch.zeros(B, n, device=DEV)
        s["positions_out"] = torch.zeros(B, n, dtype=torch.int32, device=DEV)
        s["rows_out"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        s["call"] = _plan(s)
    return s


# ------------------------------------------------------------- own kernels ----

def _plan(s):
    """The buffers that a program keeps from call to call."""
    from long_context_decode_mla_b200 import dcpmla
    c, (B, stride) = s["case"], s["table"].shape
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    p = dict(m=dcpmla)
    if c["op"] == "blocks":
        R = (B, c["q_len"], c["heads"])
        p["ws"] = u8(dcpmla.mla_decode_blocks_workspace_size(*R[:1], R[2], R[1], stride, c["topk"]))
        p["out"] = torch.empty(*R, LATENT, device=DEV)
        p["lse"] = torch.empty(*R, device=DEV)
        p["blocks"] = torch.empty(B, c["q_len"], c["topk"], dtype=torch.int32, device=DEV)
    elif c["op"] == "mass":
        p["ws"] = u8(dcpmla.mla_attention_mass_workspace_size(B, c["heads"], c["q_len"]))
    elif c["op"] == "evict":
        p["ws"] = u8(dcpmla.mla_cache_evict_workspace_size(B, c["budget"]))
    return p


def _run_own(s):
    c, p = s["case"], s["call"]
    m = p["m"]
    at = (c["shard"], c["shards"])
    if c["op"] == "summary":
        m.mla_block_summary(s["cache"], c["kv"], s["table"], s["lens"], *at, s["summaries"], first_positions=s["first"])
        return _summary_values(s)
    if c["op"] == "blocks":
        m.mla_decode_blocks(s["q"], s["cache"], c["kv"], s["summaries"], s["table"], s["lens"], *at, c["topk"], SCALE,
                            p["out"], p["lse"], p["ws"], out_blocks=p["blocks"], sink_blocks=1, recent_blocks=2)
        # the product that takes the attention's result works in bf16
        return {"out": p["out"].to(torch.bfloat16), "lse": p["lse"], "blocks": p["blocks"]}
    if c["op"] == "mass":
        m.mla_attention_mass(s["q"], s["cache"], c["kv"], s["table"], s["lens"], *at, SCALE, s["lse"], s["mass"],
                             p["ws"], decay=c["decay"])
        return s["mass"]
    m.mla_cache_evict(s["cache"], c["kv"], s["table"], s["lens"], *at, s["mass"], c["budget"], s["mass_out"],
                      s["rows_out"], p["ws"], positions_out=s["positions_out"], sink=c["sink"], recent=c["recent"])
    return {"cache": s["cache"], "mass": s["mass_out"], "positions": s["positions_out"], "rows": s["rows_out"]}


def _summary_values(s):
    """The means that the written codes and scales stand for (bf16 holds more bits than the codes do)."""
    rec = s["summaries"] if s["written"] is None else s["summaries"][s["written"]]
    codes, sc, out = rec.view(torch.int8), rec.view(torch.float32)[:, ROW // 4:, None], s["values"]
    torch.mul(codes[:, :LATENT].unflatten(1, (4, 128)), sc[:, :4], out=out[:, :LATENT].unflatten(1, (4, 128)))
    torch.mul(codes[:, LATENT:ROW], sc[:, 4], out=out[:, LATENT:])
    return out


# -------------------------------------------------------------- plain form ----

def _values(rows, kv, dtype=torch.float32):
    """Raw rows [..., row bytes] -> values [..., 576]."""
    if kv == "bf16":
        return rows.contiguous().view(torch.bfloat16).to(dtype)
    lat = rows[..., :512].contiguous().view(torch.float8_e4m3fn).to(dtype)
    sc = rows[..., 512:528].contiguous().view(torch.float32).to(dtype)
    rope = rows[..., 528:].contiguous().view(torch.bfloat16).to(dtype)
    lat = (lat.unflatten(-1, (4, 128)) * sc[..., None]).flatten(-2)
    return torch.cat([lat, rope], -1)


def _scores(s, b, dtype):
    """softmax scores of request b, [q_len * heads, rows], -inf where a query does not see the row."""
    c, n = s["case"], s["rows"][b]
    k = _values(s["cache"][s["table"][b, :-(-n // BLOCK)].long()].view(-1, ROW_BYTES[c["kv"]])[:n], c["kv"], dtype)
    sc = s["q"][b].to(dtype).view(-1, ROW) @ k.T * SCALE
    t = torch.arange(n, device=DEV) * c["shards"] + c["shard"]
    last = s["lens"][b] - c["q_len"] + torch.arange(c["q_len"], device=DEV)
    hidden = (t[None] > last[:, None]).repeat_interleave(c["heads"], 0)
    return sc.masked_fill(hidden, -math.inf)


def _int8(x):
    """fp32 [..., 576] -> int8-valued codes (as fp32) and the scales of the five groups."""
    codes, scales = torch.empty_like(x), x.new_empty(*x.shape[:-1], 5)
    for g in range(5):
        v = x[..., GROUPS[g]:GROUPS[g + 1]]
        amax = v.abs().amax(-1)
        sc = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
        codes[..., GROUPS[g]:GROUPS[g + 1]] = torch.round(v / sc[..., None])
        scales[..., g] = sc
    return codes, scales


def _summaries(s, out, first=None):
    """Means of every block that holds a row at or past `first`, as codes and scales, into `out`."""
    c = s["case"]
    rows = torch.tensor(s["rows"], device=DEV)
    b, k = torch.nonzero(torch.arange(s["table"].shape[1], device=DEV)[None] * BLOCK < rows[:, None], as_tuple=True)
    if first is not None:
        newest = (torch.minimum((k + 1) * BLOCK, rows[b]) - 1) * c["shards"] + c["shard"]
        b, k = b[newest >= first[b]], k[newest >= first[b]]
    for i in range(0, len(b), 8192):                        # pieces that fit the memory
        bi, ki = b[i:i + 8192], k[i:i + 8192]
        blk = s["table"][bi, ki].long()
        n = torch.clamp(rows[bi] - ki * BLOCK, max=BLOCK)
        x = _values(s["cache"][blk], c["kv"])
        x = x.masked_fill((torch.arange(BLOCK, device=DEV)[None] >= n[:, None])[..., None], 0.0)
        codes, sc = _int8(x.sum(1) / n[:, None])
        out[blk, :ROW] = codes.to(torch.int8).view(torch.uint8)
        out[blk, ROW:ROW + 20] = sc.view(torch.uint8)


def _select(s):
    """Chosen block indices [B * q_len, topk] in order, -1 behind them, and each one's rows."""
    c = s["case"]
    qc, qs = _int8(s["q"].to(torch.float32).view(-1, c["heads"], ROW))                  # [R, H, .]
    S = s["summaries"][s["table"].long()]                                             # [B, nb, 608]
    kc = S[..., :ROW].contiguous().view(torch.int8).to(torch.float32).repeat_interleave(c["q_len"], 0)
    ks = S[..., ROW:ROW + 20].contiguous().view(torch.float32).repeat_interleave(c["q_len"], 0)
    sc = 0.0
    for g in range(5):      # sums of whole numbers below 2^24: exact in fp32
        dot = qc[..., GROUPS[g]:GROUPS[g + 1]] @ kc[..., GROUPS[g]:GROUPS[g + 1]].transpose(1, 2)
        sc = sc + dot * (qs[..., g, None] * ks[:, None, :, g])
    rows = torch.tensor(_visible(c), device=DEV)
    nb, i = (rows + BLOCK - 1) // BLOCK, torch.arange(sc.shape[2], device=DEV)[None]
    sc = sc.masked_fill((i >= nb[:, None])[:, None], -math.inf)
    rank = (sc - sc.amax(2, keepdim=True)).amax(1)
    rank = rank.masked_fill((i < 1) | (i >= nb[:, None] - 2), math.inf).masked_fill(i >= nb[:, None], -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    order = order.masked_fill(order >= nb[:, None], sc.shape[2]).sort(1).values
    order = torch.cat([order, order.new_full((len(order), c["topk"] - order.shape[1]), sc.shape[2])], 1)
    n = torch.clamp(rows[:, None] - order * BLOCK, 0, BLOCK)
    return torch.where(n > 0, order, -1).to(torch.int32), n


def _attend(s, blocks, n):
    c = s["case"]
    R = blocks.shape[0]
    phys = s["table"].repeat_interleave(c["q_len"], 0).gather(1, blocks.clamp(min=0).long())
    k = _values(s["cache"][phys.long()].view(R, -1, ROW_BYTES[c["kv"]]), c["kv"])      # [R, topk * 64, 576]
    sc = s["q"].to(torch.float32).view(R, c["heads"], ROW) @ k.transpose(1, 2) * SCALE
    seen = (torch.arange(BLOCK, device=DEV)[None, None] < n[..., None]).view(R, 1, -1)
    sc = sc.masked_fill(~seen, -math.inf)
    m = sc.amax(2, keepdim=True).clamp(min=-1e30)
    p = torch.exp(sc - m)
    l = p.sum(2, keepdim=True)
    out = (p @ k[..., :LATENT]) / l.clamp(min=1e-38)
    lse = (m + torch.log(l)).squeeze(2)
    shape = (-1, c["q_len"], c["heads"])
    return {"out": out.to(torch.bfloat16).view(*shape, LATENT), "lse": lse.view(shape),
            "blocks": blocks.view(-1, c["q_len"], c["topk"])}


def _weights(s):
    c, mass = s["case"], s["mass"]
    rows = torch.tensor(s["rows"], device=DEV)
    t = torch.arange(mass.shape[1], device=DEV) * c["shards"] + c["shard"]
    last = s["lens"][:, None] - c["q_len"] + torch.arange(c["q_len"], device=DEV)[None]      # [B, q_len]
    piece = max(1, 200_000 // mass.shape[1])
    for b in range(0, len(rows), piece):                    # pieces that fit the memory
        e = min(b + piece, len(rows))
        k = _values(s["cache"][s["table"][b:e].long()].flatten(1, 2), c["kv"])
        sc = s["q"][b:e].to(torch.float32).flatten(1, 2) @ k.transpose(1, 2) * SCALE
        w = torch.exp(sc - s["lse"][b:e].flatten(1)[..., None]).unflatten(1, (c["q_len"], -1)).sum(2)
        w = w.masked_fill(t[None, None] > last[b:e, :, None], 0.0).sum(1)
        live = torch.arange(mass.shape[1], device=DEV)[None] < rows[b:e, None]
        mass[b:e] = torch.where(live, c["decay"] * mass[b:e] + w, mass[b:e])
    return mass


def _evict(s):
    c, mass = s["case"], s["mass"]
    rows = torch.tensor(s["rows"], device=DEV)[:, None]
    j = torch.arange(mass.shape[1], device=DEV)[None]
    pos = j * c["shards"] + c["shard"]
    live = j < rows
    kept_most = torch.clamp(rows, max=c["budget"])
    guarded = (pos < c["sink"]) | (pos >= s["lens"][:, None] - c["recent"])
    key = torch.where(guarded, math.inf, mass).masked_fill(~live, -math.inf)
    place = torch.sort(key, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(live).scatter_(1, place, (j < kept_most).expand_as(live).contiguous())
    moves, holes = kept & (j >= c["budget"]), ~kept & (j < kept_most)
    b, src = torch.nonzero(moves, as_tuple=True)
    _, dst = torch.nonzero(holes, as_tuple=True)           # as many, in the same order of requests
    at = lambda i: (s["table"][b, i // BLOCK].long(), i % BLOCK)  # noqa: E731
    s["cache"][at(dst)] = s["cache"][at(src)]
    stay = j < kept_most
    s["mass_out"][:] = torch.where(stay, mass, s["mass_out"])
    s["positions_out"][:] = torch.where(stay, pos.to(torch.int32), s["positions_out"])
    s["mass_out"][b, dst] = mass[b, src]
    s["positions_out"][b, dst] = pos[0, src].to(torch.int32)
    s["rows_out"][:] = kept_most[:, 0]
    return {"cache": s["cache"], "mass": s["mass_out"], "positions": s["positions_out"], "rows": s["rows_out"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "summary":
        _summaries(state, state["summaries"], state["first"])
        return _summary_values(state)
    if op == "blocks":
        return _attend(state, *_select(state))
    return _weights(state) if op == "mass" else _evict(state)


# ------------------------------------------------------------------- exact ----

def _row64(s, b, j):
    """Row values j (an index tensor) of request b in 64 bits."""
    raw = s["cache"][s["table"][b][j // BLOCK].long(), j % BLOCK]
    if s["case"]["kv"] == "bf16":
        return raw.contiguous().view(torch.bfloat16).double()
    v = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    for g, f in enumerate(raw[:, 512:528].contiguous().view(torch.float32).double().unbind(1)):
        v[:, 128 * g:128 * g + 128] *= f[:, None]
    return torch.hstack([v, raw[:, 528:].contiguous().view(torch.bfloat16).double()])


def _exact_summary(s):
    out = torch.zeros(s["cache"].shape[0], ROW, dtype=torch.float64, device=DEV)
    c = s["case"]
    for b, n in enumerate(s["rows"]):
        for k0 in range(0, -(-n // BLOCK), 2048):
            ks = [k for k in range(k0, min(k0 + 2048, -(-n // BLOCK)))
                  if s["first"] is None or (min(n, 64 * k + 64) - 1) * c["shards"] + c["shard"] >= int(s["lens"][b]) - 1]
            if not ks:
                continue
            j = (torch.tensor(ks, device=DEV)[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()
            w = (j < n).double()[:, None]
            mean = (torch.nan_to_num(_row64(s, b, j)) * w).view(-1, BLOCK, ROW).sum(1) / w.view(-1, BLOCK, 1).sum(1)
            for lo, hi in zip(GROUPS[:-1], GROUPS[1:]):
                step = mean[:, lo:hi].abs().amax(1, keepdim=True) / 127
                step[step == 0] = 1
                mean[:, lo:hi] = (mean[:, lo:hi] / step).round() * step
            out[s["table"][b, ks].long()] = mean
    return out if s["written"] is None else out[s["written"]]


def _exact_blocks(s):
    c = s["case"]
    H, out, lse = c["heads"], [], []
    S = s["summaries"].cpu().numpy()
    f32 = np.float32
    for r, n in enumerate(_visible(c)):
        b, i = divmod(r, c["q_len"])
        q = s["q"][b, i].double()
        nb = -(-n // BLOCK)
        if nb == 0:
            out.append(torch.zeros(H, LATENT, dtype=torch.float64, device=DEV))
            lse.append(torch.full((H,), -math.inf, dtype=torch.float64, device=DEV))
            continue
        rec = S[s["table"][b, :nb].long().cpu().numpy()]
        kc = rec[:, :ROW].view(np.int8).astype(np.float64)
        ks = np.ascontiguousarray(rec[:, ROW:ROW + 20]).view(f32)
        qn = s["q"][b, i].float().cpu().numpy()
        sc = np.zeros((H, nb), f32)
        for g, (lo, hi) in enumerate(zip(GROUPS[:-1], GROUPS[1:])):   # the score's 32-bit steps are its definition
            top = np.abs(qn[:, lo:hi]).max(1)
            step = np.where(top > 0, top / f32(127), f32(1)).astype(f32)
            code = np.rint(qn[:, lo:hi] / step[:, None]).astype(np.float64)
            sc = sc + (code @ kc[:, lo:hi].T).astype(f32) * (step[:, None] * ks[None, :, g])
        rank = (sc - sc.max(1, keepdims=True)).max(0)
        rank[0] = rank[max(0, nb - 2):] = np.inf
        ids = np.sort(np.lexsort((np.arange(nb), -rank))[:c["topk"]])
        j = (torch.from_numpy(ids).to(DEV)[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten()
        k = _row64(s, b, j[j < n])
        z = q @ k.T * SCALE
        out.append(torch.softmax(z, 1) @ k[:, :LATENT])
        lse.append(torch.logsumexp(z, 1))
    shape = (-1, c["q_len"], H)
    return {"out": torch.stack(out).view(*shape, LATENT), "lse": torch.stack(lse).view(shape), "blocks": None}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "summary":
        return _exact_summary(s)
    if c["op"] == "blocks":
        return _exact_blocks(s)
    if c["op"] == "mass":
        mass = s["mass"].double()
        for b, n in enumerate(s["rows"]):
            for j0 in range(0, n, 32768):
                j = torch.arange(j0, min(n, j0 + 32768), device=DEV)
                z = torch.einsum("qhd,jd->qhj", s["q"][b].double(), _row64(s, b, j)) * SCALE - s["lse"][b].double()[..., None]
                last = int(s["lens"][b]) - c["q_len"] + torch.arange(c["q_len"], device=DEV)
                see = (j * c["shards"] + c["shard"])[None] <= last[:, None]
                mass[b, j] = c["decay"] * mass[b, j] + (z.exp().sum(1) * see).sum(0)
        return mass
    out = np.zeros(s["mass"].shape)
    for b, n in enumerate(s["rows"]):
        m = s["mass"][b, :n].double().cpu().numpy()
        pos = np.arange(n) * c["shards"] + c["shard"]
        safe = (pos < c["sink"]) | (pos >= int(s["lens"][b]) - c["recent"])
        keep = np.sort(np.lexsort((np.arange(n), -m, ~safe))[:c["budget"]])
        top = min(n, c["budget"])
        free = np.setdiff1d(np.arange(top), keep)
        out[b, :top] = m[:top]
        out[b, free] = m[keep[keep >= c["budget"]]]
    return {"cache": None, "mass": torch.from_numpy(out), "positions": None, "rows": None}
