"""fp64 oracle of the block-summary, block-selection, attention-mass and
eviction operators (test infrastructure only).

Written from the operators' definitions; lengths, ownership and rows come from
the decode oracle.  The selection's score is defined by single fp32 operations
on whole-number code products, so its oracle repeats those steps in fp32.
"""
from __future__ import annotations

import numpy as np

from .mla_decode import decode_bf16, fetch_rows, local_positions

GROUPS = ((0, 128), (128, 256), (256, 384), (384, 512), (512, 576))
SUMMARY_BYTES = 608


def shard_rows(kv_cache, kv_dtype, table_row, seq_len, num_shards, shard_id):
    """float64 [n, 576] rows of one request on one shard, and their positions."""
    pos = local_positions(int(seq_len), num_shards, shard_id)
    if len(pos) == 0:
        return np.zeros((0, 576)), pos
    return fetch_rows(kv_cache, kv_dtype, table_row, pos, num_shards, 64), pos


def block_means(rows):
    """float64 means [blocks, 576] of consecutive 64-row blocks, and mean |row|."""
    n = -(-len(rows) // 64)
    cut = [rows[64 * k:64 * k + 64] for k in range(n)]
    return (np.array([c.mean(0) for c in cut]).reshape(n, 576),
            np.array([np.abs(c).mean(0) for c in cut]).reshape(n, 576))


def summary_fields(summaries):
    """codes int8 [.., 576] and scales fp32 [.., 5] of raw summaries uint8 [.., 608]."""
    s = np.ascontiguousarray(summaries)
    return s[..., :576].view(np.int8), np.ascontiguousarray(s[..., 576:596]).view(np.float32)


def quantise_query(q):
    """fp32 [H, 576] -> whole-number codes and fp32 steps [H, 5]."""
    q = np.where(np.isfinite(q), q, 0).astype(np.float32)
    codes, steps = np.zeros(q.shape), np.ones((len(q), 5), np.float32)
    for g, (a, b) in enumerate(GROUPS):
        top = np.abs(q[:, a:b]).max(1)
        up = top * (np.float32(1) / np.float32(127))
        steps[:, g] = np.where(up > 0, up, np.float32(1))
        codes[:, a:b] = np.clip(np.rint(q[:, a:b] / steps[:, g:g + 1]), -127, 127)
    return codes, steps


def block_ranks(q, summaries):
    """fp32 rank of every block (rows of `summaries`, raw) for one query token."""
    qc, qs = quantise_query(q)
    kc, ks = summary_fields(summaries)
    s = None
    for g, (a, b) in enumerate(GROUPS):
        dot = (qc[:, a:b] @ kc[:, a:b].astype(np.float64).T).astype(np.float32)
        t = dot * (qs[:, g, None] * ks[None, :, g])
        s = t if s is None else s + t
    assert s.dtype == np.float32
    return (s - s.max(1, keepdims=True)).max(0)


def block_select(q_bits, summaries, table, seq_lens, shard_id, num_shards, topk, sink, recent):
    """q_bits uint16 [B, q_len, H, 576] -> (blocks [B, q_len, topk] with -1 behind, lens [B, q_len])."""
    B, Q = q_bits.shape[:2]
    blocks, lens = np.full((B, Q, topk), -1, np.int32), np.zeros((B, Q), np.int32)
    for b in range(B):
        for i in range(Q):
            L = max(0, int(seq_lens[b]) - Q + 1 + i)
            n = len(local_positions(L, num_shards, shard_id))
            nb = -(-n // 64)
            if nb == 0:
                continue
            q = decode_bf16(q_bits[b, i]).astype(np.float32)
            rank = block_ranks(q, summaries[table[b, :nb]]).astype(np.float64)
            rank[:sink] = np.inf
            rank[max(0, nb - recent):] = np.inf
            ids = np.sort(np.argsort(-rank, kind="stable")[:topk])
            blocks[b, i, :len(ids)] = ids
            lens[b, i] = sum(min(64, n - 64 * k) for k in ids)
    return blocks, lens


def attention_mass(q_bits, kv_cache, kv_dtype, table, seq_lens, shard_id, num_shards, scale, lse,
                   mass, decay):
    """New mass (float64) and, per entry, the sum of weight times score error that fp32 can make."""
    B, Q, H = q_bits.shape[:3]
    out, err = np.array(mass, np.float64), np.zeros(mass.shape)
    for b in range(B):
        rows, pos = shard_rows(kv_cache, kv_dtype, table[b], seq_lens[b], num_shards, shard_id)
        n = len(pos)
        out[b, :n] = decay * out[b, :n] if decay else 0.0
        err[b, :n] = 2.0 ** -23 * np.abs(out[b, :n])
        for i in range(Q):
            seen = pos <= int(seq_lens[b]) - Q + i
            for h in range(H):
                if lse[b, i, h] == -np.inf:
                    continue
                q = decode_bf16(q_bits[b, i, h])
                s = scale * (rows @ q)
                w = np.where(seen, np.exp(s - lse[b, i, h]), 0.0)
                # products are exact, 576 of them are summed in fp32 (any order);
                # then a scaling, a subtraction and the exponential; q values below
                # 2^-9 of the head's largest may lose bits below 2^-17 of it
                mag = np.abs(scale) * (np.abs(rows) @ np.abs(q))
                small = np.abs(scale) * np.abs(rows).sum(1) * np.abs(q).max() * 2.0 ** -17
                e = 576 * 2.0 ** -24 * mag + small * (kv_dtype == "fp8") \
                    + 2.0 ** -22 * (np.abs(s) + abs(lse[b, i, h]) + 1)
                out[b, :n] += w
                err[b, :n] += w * e
        err[b, :n] += 2.0 ** -24 * Q * H * out[b, :n]
    return out, err


def evict_plan(mass, positions, length, budget, sink, recent):
    """One request: mass [n], positions [n] -> (moves [(src, dst)], new order of old rows)."""
    n = len(mass)
    if n <= budget:
        return [], list(range(n))
    safe = (positions < sink) | (positions >= length - recent)
    order = sorted(range(n), key=lambda j: (not safe[j], 0 if safe[j] else 1 if np.isnan(mass[j]) else 0,
                                            0.0 if safe[j] or np.isnan(mass[j]) else -float(mass[j]), j))
    kept = set(order[:budget])
    holes = [j for j in range(budget) if j not in kept]
    movers = [j for j in range(budget, n) if j in kept]
    new = list(range(budget))
    for s, d in zip(movers, holes):
        new[d] = s
    return list(zip(movers, holes)), new


def cache_evict(kv_cache, table, seq_lens, rows, shard_id, num_shards, mass, positions, budget, sink,
                recent, mass_out, positions_out):
    """Whole batch: (cache, mass_out, positions_out, rows_out) after the eviction."""
    cache, mo, po = kv_cache.copy(), mass_out.copy(), positions_out.copy()
    ro = np.zeros(len(seq_lens), np.int32)
    for b, L in enumerate(seq_lens):
        n = len(local_positions(int(L), num_shards, shard_id)) if rows is None else int(rows[b])
        pos = np.arange(n) * num_shards + shard_id if positions is None else positions[b, :n]
        moves, new = evict_plan(mass[b, :n], pos, int(L), budget, sink, recent)
        for s, d in moves:
            cache[table[b, d // 64], d % 64] = kv_cache[table[b, s // 64], s % 64]
        mo[b, :len(new)] = mass[b, new]
        po[b, :len(new)] = pos[new]
        ro[b] = len(new)
    return cache, mo, po, ro
