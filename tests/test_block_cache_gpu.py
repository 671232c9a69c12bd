"""GPU parity of block summaries, block-sparse decode, attention mass and
eviction against their fp64 oracles.

Selections and evictions are whole numbers and must be equal; means, weights
and attention are held to bounds that count roundings.  Rows past a request's
end and unused table entries hold junk (NaN codes, indices outside the pool),
and outputs start from a marker that must survive where nothing is written.
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
NAME = {"fp8": "agentic", "bf16": "dense"}
RAGGED = [1000, 1, 0, 64, 65, 63, 4097, 130]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dcpmla.lib()
    torch.cuda.set_device(0)


def _problem(lens, N, kv, heads=16, q_len=1, seed=5):
    """A ragged problem whose absent rows are NaN junk and whose unused table entries lie outside the pool."""
    p = wl.make_problem(NAME[kv], num_shards=N, batch=len(lens), heads=heads * q_len, seq_len=lens, seed=seed)
    for s in range(N):
        for b, L in enumerate(lens):
            n = len(oracle.local_positions(L, N, s))
            nb = -(-n // 64)
            if n % 64:
                p.kv_cache[int(p.block_tables[s, b, nb - 1]), n % 64:] = 0xFF
            p.block_tables[s, b, nb:] = 1 << 30
    p.q = p.q.view(len(lens), q_len, heads, 576)
    return p, p.numpy_inputs(), p.to("cuda")


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _flag(ws):
    return int(ws[:4].view(torch.int32).item())


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _summaries(d, s, N, out=None, first=None):
    out = torch.full((d.kv_cache.shape[0], 608), 0xAB, dtype=torch.uint8, device="cuda") if out is None else out
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, d.kv_dtype, d.block_tables[s], d.seq_lens, s, N, out, first, flags)
    assert int(flags.item()) == 0
    return out


# ------------------------------------------------------------- summaries ----

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("N", [1, 3])
def test_summary_is_the_mean(kv, N):
    p, ni, d = _problem(RAGGED, N, kv)
    for s in range(N):
        got = _summaries(d, s, N).cpu().numpy()
        written = np.zeros(len(got), bool)
        codes, scales = ob.summary_fields(got)
        for b, L in enumerate(RAGGED):
            rows, _ = ob.shard_rows(ni["kv_cache"], kv, ni["block_tables"][s, b], L, N, s)
            means, mags = ob.block_means(rows)
            for k in range(len(means)):
                blk = ni["block_tables"][s, b, k]
                written[blk] = True
                # 64 values summed in fp32 (an fp8 value's product is fused), one division
                tol = 68 * 2.0 ** -24 * mags[k]
                for g, (lo, hi) in enumerate(ob.GROUPS):
                    sc = float(scales[blk, g])
                    top = np.abs(means[k, lo:hi]).max()
                    assert abs(sc * 127 - top) <= tol[lo:hi].max() + 2.0 ** -22 * top
                    off = np.abs(codes[blk, lo:hi] * sc - means[k, lo:hi])
                    assert (off <= sc * (0.5 + 2.0 ** -15) + tol[lo:hi]).all()
                assert not got[blk, 596:].any()
        assert (got[~written] == 0xAB).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("N", [1, 2])
def test_summary_of_the_newest_blocks_only(kv, N):
    """Written again from a position on: those blocks as in a full pass, the others untouched."""
    p, ni, d = _problem(RAGGED, N, kv)
    first = [999, 0, 0, 63, 0, 63, 300, 500]
    for s in range(N):
        full = _summaries(d, s, N).cpu().numpy()
        part = _summaries(d, s, N, first=_i32(first)).cpu().numpy()
        due = np.zeros(len(full), bool)
        for b, L in enumerate(RAGGED):
            pos = oracle.local_positions(L, N, s)
            due[ni["block_tables"][s, b, np.unique(np.nonzero(pos >= first[b])[0] // 64)]] = True
        assert np.array_equal(part[due], full[due])
        assert (part[~due] == 0xAB).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_summary_of_zeros_and_of_values_that_are_not_finite(kv):
    p, ni, _ = _problem([64, 70], 1, kv)
    blk = p.block_tables[0]
    p.kv_cache[int(blk[0, 0])] = 0
    row = p.kv_cache[int(blk[1, 1])]          # six rows are present
    if kv == "bf16":
        row.view(torch.bfloat16)[3, 7] = float("inf")
        row.view(torch.bfloat16)[2, 520] = float("nan")
    else:
        row[3, 7] = 0x7F                      # the NaN code
        row[2, 528:].view(torch.bfloat16)[8] = float("nan")
    d = p.to("cuda")
    codes, scales = ob.summary_fields(_summaries(d, 0, 1).cpu().numpy())
    assert not codes[int(blk[0, 0])].any() and (scales[int(blk[0, 0])] == 1).all()
    c, s = codes[int(blk[1, 1])], scales[int(blk[1, 1])]
    assert c[7] == 0 and c[520] == 0 and np.isfinite(s).all() and np.abs(c[:128]).max() == 127


def test_summary_flags_bad_entries():
    p, ni, d = _problem([200, 100], 1, "fp8")
    d.block_tables[0, 0, 1] = -3
    d.seq_lens[1] = 10 ** 6
    out = torch.full((d.kv_cache.shape[0], 608), 0xAB, dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, "fp8", d.block_tables[0], d.seq_lens, 0, 1, out, None, flags)
    assert int(flags.item()) == dcpmla.FLAG_BAD_BLOCK | dcpmla.FLAG_BAD_LENGTH


# -------------------------------------------------------------- selection ----

def _select(d, S, s, N, heads, q_len, topk, sink, recent):
    B, stride = d.block_tables.shape[1:]
    table = torch.full((B, q_len, topk), -7, dtype=torch.int32, device="cuda")
    blocks, lens = table.clone(), torch.full((B, q_len), -7, dtype=torch.int32, device="cuda")
    ws = _ws(dcpmla.mla_block_select_workspace_size(B, heads, q_len, stride))
    dcpmla.mla_block_select(d.q, S, d.block_tables[s], d.seq_lens, s, N, topk, table, lens, ws, blocks, sink, recent)
    return blocks.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), _flag(ws)


@pytest.mark.parametrize("heads,q_len", [(1, 1), (8, 3), (37, 1), (64, 1), (64, 2)])
@pytest.mark.parametrize("N,topk,sink,recent", [(1, 4, 1, 1), (3, 5, 0, 2), (2, 100, 3, 1), (1, 1, 0, 1)])
def test_selection_equals_the_oracle(heads, q_len, N, topk, sink, recent):
    lens = [1000, 1, 0, 64, 65, 8200, 130, 12007]
    p, ni, d = _problem(lens, N, "fp8", heads, q_len)
    for s in range(N):
        S = _summaries(d, s, N)
        blocks, table, n, flag = _select(d, S, s, N, heads, q_len, topk, sink, recent)
        want, wn = ob.block_select(ni["q"], S.cpu().numpy(), ni["block_tables"][s], lens, s, N, topk, sink, recent)
        assert flag == 0
        assert np.array_equal(blocks, want) and np.array_equal(n, wn)
        for b in range(len(lens)):
            t = ni["block_tables"][s, b]
            assert np.array_equal(table[b], np.where(want[b] >= 0, t[np.maximum(want[b], 0)], -1))


@pytest.mark.parametrize("stride", [129, 4097, 20001])
def test_selection_over_long_tables(stride):
    """Summaries drawn directly: one tile and a block, and tables that a whole cluster works on."""
    g = torch.Generator().manual_seed(stride)
    S = torch.zeros(stride, 608, dtype=torch.uint8)
    S[:, :576] = torch.randint(0, 256, (stride, 576), generator=g, dtype=torch.uint8)
    S[:, 576:596] = (torch.rand(stride, 5, generator=g) + 0.1).view(torch.uint8)
    S[:, :576][S[:, :576] == 128] = 0                # codes lie in -127..127
    lens = [64 * stride, 64 * stride - 63, 64 * stride // 2 + 1]
    q = torch.randn(3, 1, 24, 576, generator=g).to(torch.bfloat16)
    table = torch.stack([torch.randperm(stride, generator=g) for _ in lens]).to(torch.int32)
    d = wl.DecodeProblem(q.cuda(), None, "fp8", table[None].cuda(), _i32(lens), 1)
    blocks, _, n, flag = _select(d, S.cuda(), 0, 1, 24, 1, 70, 2, 3)
    want, wn = ob.block_select(q.view(torch.int16).numpy().view(np.uint16), S.numpy(), table.numpy(), lens, 0, 1,
                               70, 2, 3)
    assert flag == 0 and np.array_equal(blocks, want) and np.array_equal(n, wn)


def test_selection_ties_go_to_the_lowest_block():
    """All summaries alike, all zero, and alike in pairs."""
    nb = 300
    S = torch.zeros(nb, 608, dtype=torch.uint8)
    S[:, 576:596] = torch.ones(nb, 5).view(torch.uint8)
    S[100:200, 3] = 9                                 # a hundred blocks alike, better or worse than the rest
    table = torch.arange(nb, dtype=torch.int32).repeat(2, 1)
    q = torch.zeros(2, 1, 4, 576)
    q[0, 0, :, 3], q[1, 0, :, 3] = 1.0, -1.0
    d = wl.DecodeProblem(q.to(torch.bfloat16).cuda(), None, "fp8", table[None].cuda(), _i32([64 * nb] * 2), 1)
    blocks, _, _, _ = _select(d, S.cuda(), 0, 1, 4, 1, 12, 1, 1)
    assert blocks[0, 0].tolist() == [0] + list(range(100, 110)) + [299]
    assert blocks[1, 0].tolist() == list(range(11)) + [299]


def test_selection_flags_bad_entries_and_ranks_them_last():
    lens = [64 * 9, 64 * 3]
    p, ni, d = _problem(lens, 1, "fp8", 8)
    S = _summaries(d, 0, 1)
    d.block_tables[0, 0, 4] = d.kv_cache.shape[0]
    blocks, _, n, flag = _select(d, S, 0, 1, 8, 1, 8, 1, 1)
    assert flag == dcpmla.FLAG_BAD_BLOCK
    assert blocks[0, 0].tolist() == [0, 1, 2, 3, 5, 6, 7, 8] and n.tolist() == [[512], [192]]
    d.seq_lens[1] = 10 ** 7
    assert _select(d, S, 0, 1, 8, 1, 8, 1, 1)[3] & dcpmla.FLAG_BAD_LENGTH


# ------------------------------------------------------ block-sparse decode ----

def _chosen_attention(ni, kv, s, N, lens, blocks):
    B, Q, H = ni["q"].shape[:3]
    out, lse = np.zeros((B, Q, H, 512)), np.full((B, Q, H), -np.inf)
    for b in range(B):
        for i in range(Q):
            L = max(0, lens[b] - Q + 1 + i)
            rows, pos = ob.shard_rows(ni["kv_cache"], kv, ni["block_tables"][s, b], L, N, s)
            pick = np.isin(np.arange(len(pos)) // 64, blocks[b, i][blocks[b, i] >= 0])
            if pick.any():
                out[b, i], lse[b, i] = oracle.attention_with_lse(oracle.decode_bf16(ni["q"][b, i]), rows[pick], SCALE)
    return out, lse


def _check_attention(out, lse, want, wlse, kv):
    """The decode kernels' own bounds: 2e-3 / 2e-2 of max|O|, LSE 1e-4 / 1e-3."""
    fin = np.isfinite(wlse)
    assert np.array_equal(fin, np.isfinite(lse)) and not out[~fin].any()
    assert np.abs(out - want).max() <= (2e-3 if kv == "bf16" else 2e-2) * np.abs(want).max()
    assert np.abs(lse[fin] - wlse[fin]).max() <= (1e-4 if kv == "bf16" else 1e-3)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,q_len,N,topk", [(8, 1, 1, 3), (64, 1, 2, 6), (16, 4, 2, 4), (37, 2, 1, 200)])
def test_decode_over_chosen_blocks(kv, heads, q_len, N, topk):
    lens = [1000, 2, 0, 64, 65, 5000, 130]
    p, ni, d = _problem(lens, N, kv, heads, q_len)
    B, stride = len(lens), d.block_tables.shape[2]
    ws = _ws(dcpmla.mla_decode_blocks_workspace_size(B, heads, q_len, stride, topk))
    for s in range(N):
        S = _summaries(d, s, N)
        out = torch.empty(B, q_len, heads, 512, device="cuda")
        lse = torch.empty(B, q_len, heads, device="cuda")
        blocks = torch.empty(B, q_len, topk, dtype=torch.int32, device="cuda")
        dcpmla.mla_decode_blocks(d.q, d.kv_cache, kv, S, d.block_tables[s], d.seq_lens, s, N, topk, SCALE, out, lse,
                                 ws, blocks, 1, 1)
        want, _ = ob.block_select(ni["q"], S.cpu().numpy(), ni["block_tables"][s], lens, s, N, topk, 1, 1)
        assert np.array_equal(blocks.cpu().numpy(), want) and _flag(ws) == 0
        ro, rl = _chosen_attention(ni, kv, s, N, lens, want)
        _check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ro, rl, kv)


# ---------------------------------------------------------- attention mass ----

def _mass(d, ni, kv, s, N, heads, q_len, lse, mass, decay, splits=0):
    B = len(ni["seq_lens"])
    ws = _ws(dcpmla.mla_attention_mass_workspace_size(B, heads, q_len))
    dcpmla.mla_attention_mass(d.q, d.kv_cache, kv, d.block_tables[s], d.seq_lens, s, N, SCALE, lse, mass, ws, decay,
                              splits)
    assert _flag(ws) == 0
    return mass


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,q_len,N,decay", [(8, 1, 1, 1.0), (64, 1, 2, 0.0), (37, 1, 3, 0.5), (16, 4, 1, 1.0),
                                                 (16, 7, 2, 0.9), (1, 1, 1, 0.0), (64, 3, 1, 0.0)])
def test_mass_is_the_attention_weight(kv, heads, q_len, N, decay):
    lens = [500, 1, 0, 64, 65, 2100, 129, 3]
    p, ni, d = _problem(lens, N, kv, heads, q_len)
    _, _, _, rl = oracle.dcp_decode_multi(ni["q"], ni["kv_cache"], kv, ni["block_tables"], ni["seq_lens"], N, SCALE)
    lse = torch.as_tensor(rl, dtype=torch.float32, device="cuda")
    g = np.random.default_rng(3)
    total = np.zeros((len(lens), q_len, heads))
    for s in range(N):
        width = d.block_tables.shape[2] * 64
        m0 = g.random((len(lens), width)).astype(np.float32)
        start = torch.as_tensor(m0, device="cuda")
        if decay == 0.0:
            start.fill_(float("nan"))
        got = _mass(d, ni, kv, s, N, heads, q_len, lse, start.clone(), decay)
        want, err = ob.attention_mass(ni["q"], ni["kv_cache"], kv, ni["block_tables"][s], lens, s, N, SCALE,
                                      lse.double().cpu().numpy(), m0, decay)
        again = _mass(d, ni, kv, s, N, heads, q_len, lse, start.clone(), decay, splits=5)
        x = got.double().cpu().numpy()
        for b, L in enumerate(lens):
            n = len(oracle.local_positions(L, N, s))
            assert (np.abs(x[b, :n] - want[b, :n]) <= err[b, :n]).all(), (b, np.abs(x[b, :n] - want[b, :n]).max())
            tail, first = got[b, n:], start[b, n:]
            assert torch.equal(tail.isnan(), first.isnan()) and torch.equal(tail.nan_to_num(), first.nan_to_num())
            assert torch.equal(again[b, :n], got[b, :n])          # whatever the number of CTAs


def test_mass_of_all_rows_sums_to_the_heads():
    """The weights of one query's head sum to one over all shards."""
    lens, N, H = [3000, 200], 2, 64
    p, ni, d = _problem(lens, N, "fp8", H)
    dec = dcpmla.DcpDecoder(2, H, N)
    d.q = d.q.view(2, H, 576)
    dec.step(d)
    total = torch.zeros(2, dtype=torch.float64, device="cuda")
    for s in range(N):
        m = torch.zeros(2, d.block_tables.shape[2] * 64, device="cuda")
        total += _mass(d, ni, "fp8", s, N, H, 1, dec.out_lse, m, 1.0).double().sum(1)
    # each weight is off by its score's and the LSE's error (1e-5) at most
    assert (total - H).abs().max().item() <= 2e-5 * H


def test_mass_with_empty_queries_and_bad_entries():
    lens, H = [200, 300], 8
    p, ni, d = _problem(lens, 1, "bf16", H)
    lse = torch.full((2, 1, H), float("-inf"), device="cuda")
    lse[0, 0, 0] = 3.0
    m = torch.ones(2, d.block_tables.shape[2] * 64, device="cuda")
    _mass(d, ni, "bf16", 0, 1, H, 1, lse, m, 1.0)
    assert (m[1] == 1).all() and (m[0, :200] >= 1).all() and (m[0, 200:] == 1).all()
    d.block_tables[0, 0, 1] = -1
    ws = _ws(dcpmla.mla_attention_mass_workspace_size(2, H))
    short = torch.ones(2, 250, device="cuda")
    dcpmla.mla_attention_mass(d.q, d.kv_cache, "bf16", d.block_tables[0], d.seq_lens, 0, 1, SCALE, lse, short, ws, 0.0)
    assert _flag(ws) == dcpmla.FLAG_BAD_BLOCK | dcpmla.FLAG_BAD_LENGTH
    assert (short[0, 64:128] == 1).all() and (short[1] == 0).all()


# --------------------------------------------------------------- eviction ----

def _masses(B, width, seed):
    g = np.random.default_rng(seed)
    m = (g.exponential(size=(B, width)) ** 2).astype(np.float32)
    m[g.random((B, width)) < 0.2] = 0.0
    m[g.random((B, width)) < 0.2] = 1.5                 # many ties
    m[:, ::97] = np.nan
    m[:, 5::89] = np.inf
    return m


def _evict(d, kv, s, N, mass, budget, sink, recent, rows=None, positions=None, alias=False, keep_positions=True):
    B = len(mass)
    cache = d.kv_cache.clone()
    m = torch.as_tensor(mass, device="cuda")
    pos = None if positions is None else _i32(positions)
    mo = m if alias else torch.full_like(m, -5.0)
    po = (pos if alias and pos is not None else torch.full(m.shape, -9, dtype=torch.int32, device="cuda"))
    ro = torch.full((B,), -3, dtype=torch.int32, device="cuda")
    ws = _ws(dcpmla.mla_cache_evict_workspace_size(B, budget))
    dcpmla.mla_cache_evict(cache, kv, d.block_tables[s], d.seq_lens, s, N, m, budget, mo, ro, ws,
                           None if rows is None else _i32(rows), pos, po if keep_positions else None, sink, recent)
    return cache.cpu().numpy(), mo.cpu().numpy(), po.cpu().numpy(), ro.cpu().numpy(), _flag(ws)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("N,budget,sink,recent", [(1, 64, 4, 16), (2, 100, 0, 0), (3, 1, 0, 1), (1, 333, 0, 333),
                                                  (1, 4999, 1, 5), (1, 100000, 2, 2)])
def test_eviction_equals_the_oracle(kv, N, budget, sink, recent):
    lens = [1000, 1, 0, 64, 65, 5000, 130]
    p, ni, d = _problem(lens, N, kv, 1)
    for s in range(N):
        mass = _masses(len(lens), d.block_tables.shape[2] * 64, s)
        got = _evict(d, kv, s, N, mass, budget, sink, recent)
        want = ob.cache_evict(ni["kv_cache"], ni["block_tables"][s], lens, None, s, N, mass, None, budget, sink,
                              recent, np.full_like(mass, -5.0), np.full(mass.shape, -9, np.int32))
        assert got[4] == 0
        for x, y in zip(got, want):
            assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f")


@pytest.mark.parametrize("length,budget", [(20000, 7001), (8193, 8192), (70001, 100)])
def test_eviction_of_long_requests(length, budget):
    """Requests that a whole cluster picks from, beside short ones."""
    lens = [length, 700, length - 4099]
    p, ni, d = _problem(lens, 1, "fp8", 1)
    mass = _masses(3, d.block_tables.shape[2] * 64, length)
    got = _evict(d, "fp8", 0, 1, mass, budget, 3, 50, keep_positions=False)
    want = ob.cache_evict(ni["kv_cache"], ni["block_tables"][0], lens, None, 0, 1, mass, None, budget, 3, 50,
                          np.full_like(mass, -5.0), np.full(mass.shape, -9, np.int32))
    assert got[4] == 0 and (got[2] == -9).all()
    for x, y in zip(got[:2] + got[3:4], want[:2] + want[3:4]):
        assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f")


@pytest.mark.parametrize("alias", [False, True])
def test_second_eviction_goes_by_rows_and_positions(alias):
    lens, N, s = [900, 640, 50], 2, 1
    p, ni, d = _problem(lens, N, "fp8", 1)
    g = np.random.default_rng(0)
    mass = _masses(3, d.block_tables.shape[2] * 64, 8)
    pos = np.stack([g.permutation(mass.shape[1]) for _ in lens]).astype(np.int32) * N + s
    rows = [300, 128, 25]
    got = _evict(d, "fp8", s, N, mass, 128, 5, 64, rows, pos, alias)
    mo, po = (mass, pos) if alias else (np.full_like(mass, -5.0), np.full(mass.shape, -9, np.int32))
    want = ob.cache_evict(ni["kv_cache"], ni["block_tables"][s], lens, rows, s, N, mass, pos, 128, 5, 64, mo, po)
    assert got[4] == 0
    for x, y in zip(got, want):
        assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f")


def test_eviction_clips_and_flags_bad_lengths_and_entries():
    p, ni, d = _problem([640, 640], 1, "fp8", 1)
    mass = np.arange(1280, dtype=np.float32).reshape(2, 640)      # the last 128 rows of each stay
    d.block_tables[0, 0, 8] = 1 << 29
    cache, mo, _, ro, flag = _evict(d, "fp8", 0, 1, mass, 128, 0, 0, rows=[640, 10 ** 6])
    assert flag == dcpmla.FLAG_BAD_BLOCK | dcpmla.FLAG_BAD_LENGTH and ro.tolist() == [128, 128]
    t, old = ni["block_tables"][0], ni["kv_cache"]
    assert np.array_equal(cache[t[1, :2]], old[t[1, 8:10]])
    assert np.array_equal(cache[t[0, 1]], old[t[0, 9]]) and np.array_equal(cache[t[0, 0]], old[t[0, 0]])
    assert mo[0, :128].tolist() == mass[0, 512:].tolist()


# --------------------------------------------------------------- together ----

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_serving_run(kv):
    """Decode steps as a server runs them on two shards: append the step's token, bring the last blocks'
    summaries up to date, decode over chosen blocks, merge, add the weights, then evict and decode what
    stays, the shards' caches now of their own lengths."""
    N, H, topk, budget = 2, 16, 3, 150
    lens = [700, 66, 401]
    p, ni, d = _problem([L + 8 for L in lens], N, kv, H)
    B, stride = len(lens), d.block_tables.shape[2]
    d.q = d.q.view(B, H, 576)
    d.seq_lens = _i32(lens)
    cache = ni["kv_cache"].copy()
    d.block_summaries = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    mass = [torch.zeros(B, stride * 64, device="cuda") for _ in range(N)]
    for s in range(N):
        _summaries(d, s, N, out=d.block_summaries)
    dec = dcpmla.DcpDecoder(B, H, N, block_topk=topk, max_blocks=stride)
    mws = _ws(dcpmla.mla_attention_mass_workspace_size(B, H))
    g = torch.Generator().manual_seed(2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    want_mass = [np.zeros((B, stride * 64)) for _ in range(N)]
    want_err = [np.zeros((B, stride * 64)) for _ in range(N)]
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    with torch.cuda.stream(stream):
        graph = None
        for step in range(3):
            lat = torch.randn(B, 512, generator=g).to(torch.bfloat16)
            rope = torch.randn(B, 64, generator=g).to(torch.bfloat16)
            q = torch.randn(B, H, 576, generator=g).to(torch.bfloat16)
            d.q.copy_(q)
            at = [L + step for L in lens]
            d.seq_lens.copy_(_i32([a + 1 for a in at]))
            first = _i32(at)
            for s in range(N):
                dcpmla.mla_kv_append(lat.cuda(), rope.cuda(), first, _i32(range(B)), d.block_tables[s], s, N,
                                     d.kv_cache, kv)
                cache, _ = oracle.kv_append(cache, kv, bits(lat), bits(rope), np.array(at, np.int32),
                                            np.arange(B, dtype=np.int32), ni["block_tables"][s], s, N)
                _summaries(d, s, N, out=d.block_summaries, first=first)
            if graph is None:
                graph = dec.capture(d)
            graph.replay()
            for s in range(N):
                dcpmla.mla_attention_mass(d.q, d.kv_cache, kv, d.block_tables[s], d.seq_lens, s, N, SCALE,
                                          dec.out_lse, mass[s], mws)
            # the oracle's step, by the summaries that the GPU keeps
            S, nil = d.block_summaries.cpu().numpy(), [a + 1 for a in at]
            parts, lses = [], []
            for s in range(N):
                blocks, _ = ob.block_select(bits(q)[:, None], S, ni["block_tables"][s], nil, s, N, topk, 1, 1)
                assert np.array_equal(dec.blocks[s].cpu().numpy(), blocks)
                o, l = _chosen_attention(dict(ni, q=bits(q)[:, None], kv_cache=cache), kv, s, N, nil, blocks)
                parts.append(o[:, 0])
                lses.append(l[:, 0])
            ro, rl = oracle.dcp_merge(np.array(parts), np.array(lses))
            _check_attention(dec.out.double().cpu().numpy(), dec.out_lse.double().cpu().numpy(), ro, rl, kv)
            for s in range(N):
                want_mass[s], e = ob.attention_mass(bits(q)[:, None], cache, kv, ni["block_tables"][s], nil, s, N, SCALE,
                                                    dec.out_lse.double().cpu().numpy()[:, None], want_mass[s], 1.0)
                want_err[s] += e
        assert np.array_equal(d.kv_cache.cpu().numpy(), cache) and dec.flags() == 0 and _flag(mws) == 0
        rows = []
        for s in range(N):
            got = mass[s].cpu().numpy()
            assert (np.abs(got - want_mass[s]) <= want_err[s]).all()
            rows.append(torch.empty(B, dtype=torch.int32, device="cuda"))
            ws = _ws(dcpmla.mla_cache_evict_workspace_size(B, budget))
            pos = torch.zeros(B, stride * 64, dtype=torch.int32, device="cuda")
            dcpmla.mla_cache_evict(d.kv_cache, kv, d.block_tables[s], d.seq_lens, s, N, mass[s], budget, mass[s],
                                   rows[s], ws, positions_out=pos, sink=2, recent=20)
            kept, mo, po, ro_ = ob.cache_evict(cache, ni["block_tables"][s], nil, None, s, N, got, None, budget, 2, 20,
                                               got, np.zeros(got.shape, np.int32))
            cache = kept
            assert np.array_equal(rows[s].cpu().numpy(), ro_) and np.array_equal(pos.cpu().numpy(), po)
            assert np.array_equal(mass[s].cpu().numpy(), mo)
        assert np.array_equal(d.kv_cache.cpu().numpy(), cache)
        # what stays: every shard is a cache of rows_out rows by itself
        dws = _ws(dcpmla.mla_decode_workspace_size(B, H))
        parts, lses = torch.empty(N, B, H, 512, device="cuda"), torch.empty(N, B, H, device="cuda")
        out, lse = torch.empty(B, H, 512, device="cuda"), torch.empty(B, H, device="cuda")
        ref = []
        for s in range(N):
            dcpmla.mla_decode_partial(d.q, d.kv_cache, kv, d.block_tables[s], rows[s], 0, 1, None, SCALE, parts[s],
                                      lses[s], dws)
            ref.append(oracle.mla_decode_partial(bits(q), cache, kv, ni["block_tables"][s], rows[s].cpu().numpy(), 0, 1,
                                                 SCALE))
        dcpmla.dcp_merge(parts, lses, out, lse)
        ro, rl = oracle.dcp_merge(np.array([r[0] for r in ref]), np.array([r[1] for r in ref]))
        _check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ro, rl, kv)
