"""Block summaries, block-sparse decode, attention mass and eviction where their
schedules can go wrong: more requests than a launch looks at together, one CTA
for all of them, every kernel choice, calls on two streams at once, and captured
steps replayed on new inputs.
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


def _u8(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _small_requests(B, kv, heads, seed, longest=200):
    """B requests of 0..longest rows, all tables over one small pool of blocks (requests share them)."""
    g = torch.Generator().manual_seed(seed)
    blocks = 40
    pool = wl.random_kv_pool(blocks, kv, seed)
    table = torch.randint(0, blocks, (B, -(-longest // 64)), generator=g, dtype=torch.int32)
    lens = torch.randint(0, longest + 1, (B,), generator=g, dtype=torch.int32)
    lens[:4] = torch.tensor([0, 1, 64, longest])
    q = torch.randn(B, heads, 576, generator=g).to(torch.bfloat16)
    return pool, table, lens, q


def _bits(q):
    return q.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,splits", [(700, 0), (700, 1), (300, 2)])
def test_mass_of_many_small_requests(kv, B, splits):
    H = 3
    pool, table, lens, q = _small_requests(B, kv, H, B + splits)
    lse = torch.full((B, H), 4.0, device="cuda")
    mass = torch.full((B, 256), -2.0, device="cuda")
    ws = _u8(dcpmla.mla_attention_mass_workspace_size(B, H))
    dcpmla.mla_attention_mass(q.cuda(), pool.cuda(), kv, table.cuda(), lens.cuda(), 0, 1, SCALE, lse, mass, ws, 0.0,
                              splits)
    assert int(ws[:4].view(torch.int32).item()) == 0
    want, err = ob.attention_mass(_bits(q)[:, None], pool.numpy(), kv, table.numpy(), lens.numpy(), 0, 1, SCALE,
                                  lse.double().cpu().numpy()[:, None], np.full((B, 256), -2.0), 0.0)
    got = mass.double().cpu().numpy()
    assert (np.abs(got - want) <= err).all()
    assert (got[np.arange(256)[None] >= lens.numpy()[:, None]] == -2.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_mass_of_one_head(kv):
    """One head's weights keep their relative error: no other head's, and no sum over rows, averages it away."""
    B, n = 64, 64
    pool = wl.random_kv_pool(B, kv, 71)
    q = torch.randn(B, 1, 576, generator=torch.Generator().manual_seed(72)).to(torch.bfloat16)
    table = torch.arange(B, dtype=torch.int32)[:, None].contiguous()
    z = np.stack([oracle.decode_rows(pool[b].numpy(), kv) @ q[b, 0].double().numpy() for b in range(B)]) * SCALE
    lse = torch.from_numpy(np.log(np.exp(z).sum(1))).float()[:, None]
    mass = torch.zeros(B, n, device="cuda")
    ws = _u8(dcpmla.mla_attention_mass_workspace_size(B, 1))
    dcpmla.mla_attention_mass(q.cuda(), pool.cuda(), kv, table.cuda(), _i32([n] * B), 0, 1, SCALE, lse.cuda(), mass,
                              ws, 0.0)
    want = np.exp(z - lse.double().numpy())
    off = mass.cpu().double().numpy() / want - 1
    # a weight's relative error is its exponent's error: the scores' and the log-sum's sizes are below 16, so six
    # fp32 additions and two constants add 2^-25 * 16 each at most, 0.6 of that in the mean square
    assert np.sqrt((off ** 2).mean()) <= np.sqrt(8) * 0.6 * 16 * 2.0 ** -25


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_summaries_of_many_requests(kv):
    """More requests than one look at the lengths covers; each block belongs to one of them."""
    B = 1500
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 65, (B,), generator=g, dtype=torch.int32)
    pool = wl.random_kv_pool(B, kv, 3)
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None].contiguous()
    S = torch.full((B, 608), 0xAB, dtype=torch.uint8, device="cuda")
    dcpmla.mla_block_summary(pool.cuda(), kv, table.cuda(), lens.cuda(), 0, 1, S)
    codes, scales = ob.summary_fields(S.cpu().numpy())
    for b in range(B):
        blk, n = int(table[b, 0]), int(lens[b])
        if n == 0:
            assert (S[blk].cpu().numpy() == 0xAB).all()
            continue
        rows = oracle.decode_rows(pool[blk, :n].numpy(), kv)
        mean, mag = rows.mean(0), np.abs(rows).mean(0)
        for i, (lo, hi) in enumerate(ob.GROUPS):
            off = np.abs(codes[blk, lo:hi] * float(scales[blk, i]) - mean[lo:hi])
            assert (off <= scales[blk, i] * (0.5 + 2.0 ** -15) + 68 * 2.0 ** -24 * mag[lo:hi]).all()


@pytest.mark.parametrize("B,q_len", [(700, 1), (260, 2)])
def test_selection_of_many_queries(B, q_len):
    pool, table, lens, _ = _small_requests(B, "fp8", 1, 9, longest=700)
    H = 5
    q = torch.randn(B, q_len, H, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    S = torch.zeros(40, 608, dtype=torch.uint8)
    g = torch.Generator().manual_seed(2)
    S[:, :576] = torch.randint(0, 127, (40, 576), generator=g, dtype=torch.uint8)
    S[:, 576:596] = (torch.rand(40, 5, generator=g) + 0.1).view(torch.uint8)
    topk = 4
    t = torch.empty(B, q_len, topk, dtype=torch.int32, device="cuda")
    b, n = torch.empty_like(t), torch.empty(B, q_len, dtype=torch.int32, device="cuda")
    ws = _u8(dcpmla.mla_block_select_workspace_size(B, H, q_len, table.shape[1]))
    dcpmla.mla_block_select(q.cuda(), S.cuda(), table.cuda(), lens.cuda(), 0, 1, topk, t, n, ws, b, 1, 1)
    want, wn = ob.block_select(_bits(q), S.numpy(), table.numpy(), lens.numpy(), 0, 1, topk, 1, 1)
    assert np.array_equal(b.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)


def _crowded_selection(B=48, H=16, stride=1024):
    """Ranks so close together that one rounding of a step more or less changes the choice."""
    g = torch.Generator().manual_seed(31)
    q = torch.randn(B, 1, H, 576, generator=g).to(torch.bfloat16)
    S = torch.zeros(stride, 608, dtype=torch.uint8)
    S[:, :576] = torch.randint(0, 256, (stride, 576), generator=g).to(torch.uint8)
    S[:, 576:596] = (torch.rand(stride, 5, generator=g) * 0.01 + 0.01).view(torch.uint8)
    table = torch.arange(stride, dtype=torch.int32).repeat(B, 1)
    lens = torch.full((B,), stride * 64, dtype=torch.int32)
    return q, S, table, lens


def test_selection_of_close_ranks():
    q, S, table, lens = _crowded_selection()
    B, stride = table.shape
    topk = stride // 2
    t = torch.empty(B, 1, topk, dtype=torch.int32, device="cuda")
    b, n = torch.empty_like(t), torch.empty(B, 1, dtype=torch.int32, device="cuda")
    ws = _u8(dcpmla.mla_block_select_workspace_size(B, q.shape[2], 1, stride))
    dcpmla.mla_block_select(q.cuda(), S.cuda(), table.cuda(), lens.cuda(), 0, 1, topk, t, n, ws, b, 1, 1)
    want, _ = ob.block_select(_bits(q), S.numpy(), table.numpy(), lens.numpy(), 0, 1, topk, 1, 1)
    assert np.array_equal(b.cpu().numpy(), want)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_summary_scale_is_one_multiplication(kv):
    """64 equal bf16 values (fp8 rows: the rope) have an exact mean: scale = largest one * fp32(1/127), no division."""
    n = 64
    pool = wl.random_kv_pool(n, kv, 17)
    pool[:] = pool[:, :1]
    S = _u8(n * 608).view(n, 608)
    dcpmla.mla_block_summary(pool.cuda(), kv, _i32(np.arange(n)[None]), _i32([n * 64]), 0, 1, S)
    _, scales = ob.summary_fields(S.cpu().numpy())
    rows = oracle.decode_rows(pool[:, 0].numpy(), kv).astype(np.float32)
    top = np.stack([np.abs(rows[:, lo:hi]).max(1) for lo, hi in ob.GROUPS], 1)
    if kv == "fp8":
        top, scales = top[:, 4:], scales[:, 4:]
    up = top * (np.float32(1) / np.float32(127))
    assert (up != top / np.float32(127)).any() and np.array_equal(scales, up)


def test_eviction_of_many_requests():
    B, budget = 600, 40
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 129, (B,), generator=g, dtype=torch.int32)
    pool = wl.random_kv_pool(2 * B, "fp8", 3)
    table = torch.randperm(2 * B, generator=g).to(torch.int32).view(B, 2)
    mass = torch.rand(B, 128, generator=g)
    cache, m = pool.cuda(), mass.cuda()
    mo, ro = torch.full_like(m, -1.0), torch.empty(B, dtype=torch.int32, device="cuda")
    ws = _u8(dcpmla.mla_cache_evict_workspace_size(B, budget))
    dcpmla.mla_cache_evict(cache, "fp8", table.cuda(), lens.cuda(), 0, 1, m, budget, mo, ro, ws, sink=1, recent=5)
    want = ob.cache_evict(pool.numpy(), table.numpy(), lens.numpy(), None, 0, 1, mass.numpy(), None, budget, 1, 5,
                          np.full((B, 128), -1.0, np.float32), np.zeros((B, 128), np.int32))
    assert np.array_equal(cache.cpu().numpy(), want[0]) and np.array_equal(mo.cpu().numpy(), want[1])
    assert np.array_equal(ro.cpu().numpy(), want[3])


@pytest.mark.parametrize("kv,impl", [("bf16", "simt"), ("bf16", "tc"), ("bf16", "tc16"), ("fp8", "simt"), ("fp8", "tc"),
                                     ("fp8", "tc16")])
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_block_sparse_decode_on_every_kernel(kv, impl, splits):
    """With every block chosen it is dense decode, whichever kernel runs it; with fewer the choice is the same."""
    lens, H = [900, 64, 3, 0], 12
    p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=1, batch=4, heads=H, seq_len=lens, seed=6)
    ni, d = p.numpy_inputs(), p.to("cuda")
    S = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, kv, d.block_tables[0], d.seq_lens, 0, 1, S)
    stride = d.block_tables.shape[2]
    ref = {}
    for topk in (stride, 3):
        ws = _u8(dcpmla.mla_decode_blocks_workspace_size(4, H, 1, stride, topk, splits))
        out, lse = torch.empty(4, H, 512, device="cuda"), torch.empty(4, H, device="cuda")
        blocks = torch.empty(4, topk, dtype=torch.int32, device="cuda")
        dcpmla.mla_decode_blocks(d.q, d.kv_cache, kv, S, d.block_tables[0], d.seq_lens, 0, 1, topk, SCALE, out, lse, ws,
                                 blocks, 1, 1, splits, impl)
        assert int(ws[:4].view(torch.int32).item()) == 0
        ref[topk] = (out.double().cpu().numpy(), lse.double().cpu().numpy(), blocks.cpu().numpy())
    o, l = oracle.mla_decode_partial(ni["q"], ni["kv_cache"], kv, ni["block_tables"][0], ni["seq_lens"], 0, 1, SCALE)
    # the decode kernels' bounds; the fp16-operand kernel's LSE over fp8 rows 5e-3
    tol_o, tol_l = (2e-3, 1e-4) if kv == "bf16" else (2e-2, 5e-3 if impl == "tc16" else 1e-3)
    got_o, got_l, _ = ref[stride]
    fin = np.isfinite(l)
    assert np.array_equal(fin, np.isfinite(got_l))
    assert np.abs(got_o - o).max() <= tol_o * np.abs(o).max() and np.abs(got_l[fin] - l[fin]).max() <= tol_l
    want, _ = ob.block_select(ni["q"][:, None], S.cpu().numpy(), ni["block_tables"][0], lens, 0, 1, 3, 1, 1)
    assert np.array_equal(ref[3][2], want[:, 0])


def test_two_calls_at_once():
    """Two streams, a workspace each, the same inputs: each call's result is that of a call alone."""
    lens, H, topk, budget = [6000, 4100, 9000], 16, 8, 500
    p = wl.make_problem("agentic", num_shards=1, batch=3, heads=H, seq_len=lens, seed=2)
    d = p.to("cuda")
    stride = d.block_tables.shape[2]
    S = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, "fp8", d.block_tables[0], d.seq_lens, 0, 1, S)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for k in range(3):       # the third set is the one that runs alone
        g = torch.Generator(device="cuda").manual_seed(5)
        sets.append(dict(
            out=torch.empty(3, H, 512, device="cuda"), lse=torch.empty(3, H, device="cuda"),
            blocks=torch.empty(3, topk, dtype=torch.int32, device="cuda"), cache=d.kv_cache.clone(),
            mass=torch.rand(3, stride * 64, generator=g, device="cuda"), rows=torch.empty(3, dtype=torch.int32,
                                                                                         device="cuda"),
            w1=_u8(dcpmla.mla_decode_blocks_workspace_size(3, H, 1, stride, topk)),
            w2=_u8(dcpmla.mla_attention_mass_workspace_size(3, H)),
            w3=_u8(dcpmla.mla_cache_evict_workspace_size(3, budget))))
    torch.cuda.synchronize()

    def run(s, stream):
        dcpmla.mla_decode_blocks(d.q, s["cache"], "fp8", S, d.block_tables[0], d.seq_lens, 0, 1, topk, SCALE, s["out"],
                                 s["lse"], s["w1"], s["blocks"], 1, 2, stream=stream)
        dcpmla.mla_attention_mass(d.q, s["cache"], "fp8", d.block_tables[0], d.seq_lens, 0, 1, SCALE, s["lse"], s["mass"],
                                  s["w2"], stream=stream)
        dcpmla.mla_cache_evict(s["cache"], "fp8", d.block_tables[0], d.seq_lens, 0, 1, s["mass"], budget, s["mass"],
                               s["rows"], s["w3"], sink=2, recent=50, stream=stream)

    for k in range(2):
        run(sets[k], streams[k])
    torch.cuda.synchronize()
    run(sets[2], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for k in range(2):
        for name in ("out", "lse", "blocks", "cache", "mass", "rows"):
            assert torch.equal(sets[k][name], sets[2][name]), (k, name)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_step_follows_its_inputs(kv):
    """A captured step (summaries of the newest blocks, choice, decode, weights, eviction) replayed on other
    lengths, queries and masses gives what the calls give."""
    H, topk, budget, B = 16, 4, 300, 2
    p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=1, batch=B, heads=H, seq_len=[3000, 2500],
                        seed=4)
    d = p.to("cuda")
    stride = d.block_tables.shape[2]
    fresh = d.kv_cache.clone()

    def buffers():
        return dict(S=torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda"),
                    out=torch.zeros(B, H, 512, device="cuda"), lse=torch.zeros(B, H, device="cuda"),
                    blocks=torch.zeros(B, topk, dtype=torch.int32, device="cuda"),
                    mass=torch.zeros(B, stride * 64, device="cuda"), pos=torch.zeros(B, stride * 64, dtype=torch.int32,
                                                                                     device="cuda"),
                    rows=torch.zeros(B, dtype=torch.int32, device="cuda"), cache=fresh.clone(),
                    w=[_u8(dcpmla.mla_decode_blocks_workspace_size(B, H, 1, stride, topk)),
                       _u8(dcpmla.mla_attention_mass_workspace_size(B, H)),
                       _u8(dcpmla.mla_cache_evict_workspace_size(B, budget))])

    q, lens, first = d.q.clone(), d.seq_lens.clone(), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(s):
        t = d.block_tables[0]
        dcpmla.mla_block_summary(s["cache"], kv, t, lens, 0, 1, s["S"], first)
        dcpmla.mla_decode_blocks(q, s["cache"], kv, s["S"], t, lens, 0, 1, topk, SCALE, s["out"], s["lse"], s["w"][0],
                                 s["blocks"])
        dcpmla.mla_attention_mass(q, s["cache"], kv, t, lens, 0, 1, SCALE, s["lse"], s["mass"], s["w"][1])
        dcpmla.mla_cache_evict(s["cache"], kv, t, lens, 0, 1, s["mass"], budget, s["mass"], s["rows"], s["w"][2],
                               positions_out=s["pos"], sink=1, recent=10)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = buffers(), buffers()
    with torch.cuda.stream(side):
        step(a)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(a)
    for k, new in enumerate(([3000, 2500], [65, 2499], [0, 1], [2000, 64])):
        g = torch.Generator(device="cuda").manual_seed(k)
        q.copy_(torch.randn(B, H, 576, generator=g, device="cuda"))
        lens.copy_(_i32(new))
        for s in (a, b):
            s["cache"].copy_(fresh)
            s["mass"].copy_(torch.rand(B, stride * 64, generator=g.manual_seed(k), device="cuda"))
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for name in ("S", "out", "lse", "blocks", "mass", "pos", "rows", "cache"):
            assert torch.equal(a[name], b[name]), (k, name)
        assert a["rows"].tolist() == [min(n, budget) for n in new]


def test_a_device_that_is_not_current_is_refused():
    """Tensors in host memory among device ones are turned down before any pointer is passed on."""
    p = wl.make_problem("agentic", num_shards=1, batch=1, heads=4, seq_len=[100], seed=1)
    d = p.to("cuda")
    S = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="cuda device"):
        dcpmla.mla_block_summary(d.kv_cache, "fp8", p.block_tables[0], d.seq_lens, 0, 1, S)
    with pytest.raises(ValueError, match="must be contiguous"):
        dcpmla.mla_block_summary(d.kv_cache, "fp8", d.block_tables[0], d.seq_lens, 0, 1, S[:, :600])
