"""Decode over chosen blocks holds the precision that its two terms of P give it.

The bounds are counted from the inputs, and each test shows on the CPU that the
form with one term less, or with the leading term cut instead of rounded, is
outside them.
"""
import numpy as np
import pytest
import torch

import oracle
from long_context_decode_mla_b200 import dcpmla
from long_context_decode_mla_b200 import workload as wl
from oracle import block_cache as ob

pytestmark = pytest.mark.gpu

SCALE = wl.SOFTMAX_SCALE


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dcpmla.lib()
    torch.cuda.set_device(0)


def _decode(p, kv, topk, splits=0):
    """Decode over the chosen blocks of one shard: O, LSE (float64) and the blocks."""
    d = p.to("cuda")
    B, H = d.q.shape[:2]
    S = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, kv, d.block_tables[0], d.seq_lens, 0, 1, S)
    ws = torch.zeros(dcpmla.mla_decode_blocks_workspace_size(B, H, 1, d.block_tables.shape[2], topk, splits),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(B, H, 512, device="cuda"), torch.empty(B, H, device="cuda")
    blocks = torch.empty(B, topk, dtype=torch.int32, device="cuda")
    dcpmla.mla_decode_blocks(d.q, d.kv_cache, kv, S, d.block_tables[0], d.seq_lens, 0, 1, topk, SCALE, out, lse, ws,
                             blocks, 1, 1, splits)
    assert int(ws[:4].view(torch.int32).item()) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), blocks.cpu().numpy()


def _bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("heads,splits", [(16, 0), (64, 1), (16, 5), (1, 1)])
@pytest.mark.parametrize("grow", [0.0, 0.25])
def test_bf16_rows_keep_both_terms_of_p(heads, splits, grow):
    """Requests of one to nine tiles, so that the second term's buffer is used again and again, with scores that
    grow from tile to tile, so that O is rescaled in between."""
    lens, topk = [576, 300, 129, 64, 40, 7], 9
    p = wl.make_problem("dense", num_shards=1, batch=len(lens), heads=heads, seq_len=lens, seed=41)
    for b, L in enumerate(lens):
        for k in range(-(-L // 64)):
            rows = p.kv_cache[int(p.block_tables[0, b, k])].view(torch.bfloat16)
            rows.copy_((rows.float() * (1 + grow * k)).to(torch.bfloat16))
    ni = p.numpy_inputs()
    out, lse, _ = _decode(p, "bf16", topk, splits)
    caught = 0
    for b, L in enumerate(lens):
        rows, _ = ob.shard_rows(ni["kv_cache"], "bf16", ni["block_tables"][0, b], L, 1, 0)
        q = oracle.decode_bf16(ni["q"][b])
        want, wl_ = oracle.attention_with_lse(q, rows, SCALE)
        # A score is 36 sums of 16 exact products, added one after the other; each addition cuts at most 2^-23 of
        # what it adds up.  Then one product with the scale, whose constant is rounded too, and one difference.
        prod = q[:, None, :] * rows[None]
        part = prod.reshape(heads, L, 36, 16)
        before = np.abs(np.cumsum(part.sum(3), 2) - part.sum(3))
        s = SCALE * prod.sum(2)
        e = SCALE * 2.0 ** -23 * (before + np.abs(part).sum(3)).sum(2) + 2.0 ** -22 * np.abs(s)
        # P: the exponential 2^-22, its two bf16 terms 2^-17; O: eight additions a tile as above; the sum of P: 32
        # additions and one a tile; pieces of a request are weighed and added in fp32
        tiles = -(-L // 64)
        c = 2.0 ** -22 + 2.0 ** -17 + 8 * tiles * 2.0 ** -23 + (32 + tiles) * 2.0 ** -24 + 2.0 ** -20
        w = np.exp(s - wl_[:, None])
        tol = (w * (e + (w * e).sum(1, keepdims=True) + c)) @ np.abs(rows[:, :512])
        assert (np.abs(out[b] - want) <= tol).all(), (b, (np.abs(out[b] - want) / tol).max())
        assert (np.abs(lse[b] - wl_) <= (w * e).sum(1) + c + 2.0 ** -21 * np.abs(s).max(1)).all()
        # one term only, each tile relative to its own largest score
        one = np.empty_like(w)
        for t in range(tiles):
            top = s[:, 64 * t:64 * t + 64].max(1, keepdims=True)
            one[:, 64 * t:64 * t + 64] = _bf16(np.exp(s[:, 64 * t:64 * t + 64] - top)) * np.exp(top - wl_[:, None])
        caught += bool((np.abs(one @ rows[:, :512] - want) > tol).any())
    assert caught >= len(lens) - 1


def _e4m3(x):
    return x.to(torch.float8_e4m3fn).float()


def _p_terms(p16, rounded):
    """Sum of the two e4m3 terms of fp16 values: the leading one with 4 significant bits, and what it leaves."""
    bits = p16.view(torch.int16).int() & 0xFFFF
    hi = ((bits + (0x40 if rounded else 0)) & 0xFF80).to(torch.int16).view(torch.float16)
    return _e4m3(hi.float()) + _e4m3((p16.float() - hi.float()).half().float())


def test_fp8_rows_round_the_leading_term_of_p():
    """Requests of one tile, where P is known from the inputs: the RMS error lies below the geometric mean of what a
    rounded and what a cut leading term make of that P."""
    lens, H = [8, 16, 11, 20, 13, 9, 17, 16] * 4, 32
    p = wl.make_problem("agentic", num_shards=1, batch=len(lens), heads=H, seq_len=lens, seed=31)
    ni = p.numpy_inputs()
    out, _, _ = _decode(p, "fp8", 2)
    err, total, got = {False: 0.0, True: 0.0}, 0.0, 0.0
    for b, L in enumerate(lens):
        rows, _ = ob.shard_rows(ni["kv_cache"], "fp8", ni["block_tables"][0, b], L, 1, 0)
        raw = p.kv_cache[int(p.block_tables[0, b, 0]), :L]
        sc = raw[:, 512:528].contiguous().view(torch.float32)
        codes = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
        q = oracle.decode_bf16(ni["q"][b])
        want, _ = oracle.attention_with_lse(q, rows, SCALE)
        s = SCALE * (q @ rows.T)
        w = torch.from_numpy(np.exp(s - s.max(1, keepdims=True)))
        for g in range(4):
            top, cols = sc[:, g].max(), slice(128 * g, 128 * g + 128)
            p16 = (w.half().float() * (sc[:, g] * (8 / top)).half().float()).half()
            for r in err:
                o = (_p_terms(p16, r).double() @ codes[:, cols]) * (top / 8) / w.sum(1, keepdim=True)
                err[r] += float(((o - torch.from_numpy(want[:, cols])) ** 2).sum())
        total += (want ** 2).sum()
        got += ((out[b] - want) ** 2).sum()
    cut, rounded = np.sqrt(err[False] / total), np.sqrt(err[True] / total)
    assert cut > 1.6 * rounded
    assert np.sqrt(got / total) <= np.sqrt(cut * rounded), (np.sqrt(got / total), cut, rounded)


@pytest.mark.parametrize("rows,factors", [(4032, (1,)), (1000, (1,)), (4032, (1, 3)), (2050, (1, 3, 9, 27)),
                                          (2050, (27, 9, 3, 1)), (3000, (1, 1.9, 0.2))])
def test_fp8_rows_that_weigh_little_are_not_lost(rows, factors):
    """A choice of thousands of rows: what e4m3 cuts off below its smallest step adds up over them.  The RMS error
    lies below the geometric mean of what P in a frame of 28 and in one of 8 leaves, with the running maximum as
    one CTA moves it and the scales' reference as the blocks' scales (times the factors in turn) raise it."""
    B, H = 4, 8
    p = wl.make_problem("agentic", num_shards=1, batch=B, heads=H, seq_len=[rows] * B, seed=77)
    for b in range(B):
        for t in range(-(-rows // 64)):
            sc = p.kv_cache[int(p.block_tables[0, b, t]), :, 512:528]
            sc.copy_((sc.contiguous().view(torch.float32) * factors[t % len(factors)]).view(torch.uint8))
    ni = p.numpy_inputs()
    out, _, _ = _decode(p, "fp8", -(-rows // 64), 1)
    err, total, got = {(28.0, 2.0): 0.0, (8.0, 4.0): 0.0}, 0.0, 0.0
    for b in range(B):
        k, _ = ob.shard_rows(ni["kv_cache"], "fp8", ni["block_tables"][0, b], rows, 1, 0)
        raw = p.kv_cache[p.block_tables[0, b].long()].view(-1, 656)[:rows]
        sc = raw[:, 512:528].contiguous().view(torch.float32)
        codes = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
        q = oracle.decode_bf16(ni["q"][b])
        want, lse = oracle.attention_with_lse(q, k, SCALE)
        s = SCALE / np.log(2.0) * (q @ k.T)
        used, m = np.empty_like(s), np.full(H, -np.inf)
        for t in range(0, rows, 64):
            top = s[:, t:t + 64].max(1)
            m = np.where(top > m + 3.0, top, m)
            used[:, t:t + 64] = m[:, None]
        w = torch.from_numpy(np.exp2(s - used)).half().float()
        back = torch.from_numpy(np.exp2(used - lse[:, None] / np.log(2.0)))
        for g in range(4):
            cols = slice(128 * g, 128 * g + 128)
            for norm, slack in err:
                ref, r = torch.empty(rows), 0.0
                for t in range(0, rows, 64):
                    top = float(sc[t:t + 64, g].max())
                    r = top if top > slack * r else r
                    ref[t:t + 64] = r
                p16 = (w * (sc[:, g] * (norm / ref)).half().float()).half()
                o = (_p_terms(p16, True).double() * back * (ref / norm)) @ codes[:, cols]
                err[norm, slack] += float(((o - torch.from_numpy(want[:, cols])) ** 2).sum())
        total += (want ** 2).sum()
        got += ((out[b] - want) ** 2).sum()
    fine, coarse = np.sqrt(err[28.0, 2.0] / total), np.sqrt(err[8.0, 4.0] / total)
    # few rows carry a softmax of large scores, and then the frames differ little: there the model alone, with scores
    # up to 3e-4 off (36 additions that cut 2^-23 of sums up to 27 * 17, times the scale, twice)
    limit = np.sqrt(fine * coarse) if coarse > 1.2 * fine else np.hypot(fine, 3e-4)
    assert coarse > 1.2 * fine or max(factors) > 1
    assert np.sqrt(got / total) <= limit, (np.sqrt(got / total), fine, coarse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_call_repeats_itself(kv):
    """The same call gives the same bits, whatever the order in which its CTAs run."""
    lens = [9000, 500, 64, 1, 3000]
    p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=1, batch=5, heads=24, seq_len=lens, seed=8)
    first = _decode(p, kv, 8)
    for _ in range(3):
        for a, b in zip(first, _decode(p, kv, 8)):
            assert np.array_equal(a, b)
