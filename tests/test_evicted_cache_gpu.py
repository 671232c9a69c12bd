"""Evicted caches that go on being used: tokens appended behind the kept rows,
summaries, choice, decode, weights and further evictions in place, and draft
tokens over shards that no longer hold their share of the positions.

What the calls leave to the caller is done here as the header states it: after
an eviction every summary of the request is written again, and an appended row
gets mass 0 and its token's position before it is weighed.
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


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _flag(ws):
    return int(ws[:4].view(torch.int32).item())


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _bits(t):
    return t.view(torch.int16).numpy().view(np.uint16)


class _Caches:
    """Requests over N shards, on the GPU through the calls and beside it in the oracle's arrays."""

    def __init__(self, kv, N, H, lens, room, seed):
        self.kv, self.N, self.H, self.B = kv, N, H, len(lens)
        p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=N, batch=self.B, heads=H,
                            seq_len=[L + room for L in lens], seed=seed)
        self.tables, d = p.block_tables.numpy(), p.to("cuda")
        self.cache, self.t = d.kv_cache, d.block_tables
        self.ref = p.kv_cache.numpy().copy()
        self.stride = self.t.shape[2]
        self.lens = np.array(lens)                         # global lengths
        self.g = torch.Generator().manual_seed(seed)
        n = self.stride * 64
        self.mass = [torch.rand(self.B, n, generator=self.g).cuda() for _ in range(N)]
        self.pos = [torch.full((self.B, n), -77, dtype=torch.int32, device="cuda") for _ in range(N)]
        self.rows = [None] * N                             # rows held, once evicted
        self.S = torch.zeros(self.cache.shape[0], 608, dtype=torch.uint8, device="cuda")
        self.want = [m.double().cpu().numpy() for m in self.mass]
        self.err = [np.zeros((self.B, n)) for _ in range(N)]
        self.ref_pos, self.ref_rows = [None] * N, [None] * N

    def evict(self, budget, sink, recent):
        """In place, by rows and positions from the second time on; then all summaries anew."""
        L = _i32(self.lens)
        ws = _ws(dcpmla.mla_cache_evict_workspace_size(self.B, budget))
        for s in range(self.N):
            got = self.mass[s].cpu().numpy()
            live = [len(oracle.local_positions(int(x), self.N, s)) for x in self.lens] if self.rows[s] is None \
                else self.ref_rows[s]
            for b in range(self.B):
                off = np.abs(got[b, :live[b]] - self.want[s][b, :live[b]])
                assert (off <= self.err[s][b, :live[b]]).all()
            out = torch.empty(self.B, dtype=torch.int32, device="cuda")
            dcpmla.mla_cache_evict(self.cache, self.kv, self.t[s], L, s, self.N, self.mass[s], budget, self.mass[s], out,
                                   ws, rows=self.rows[s], positions=None if self.rows[s] is None else self.pos[s],
                                   positions_out=self.pos[s], sink=sink, recent=recent)
            old = np.full(got.shape, -77, np.int32) if self.ref_pos[s] is None else self.ref_pos[s]
            self.ref, mo, po, ro = ob.cache_evict(self.ref, self.tables[s], self.lens, self.ref_rows[s], s, self.N, got,
                                                  self.ref_pos[s], budget, sink, recent, got, old)
            self.rows[s], self.ref_rows[s], self.ref_pos[s] = out, ro, po
            assert np.array_equal(out.cpu().numpy(), ro) and np.array_equal(self.mass[s].cpu().numpy(), mo)
            assert np.array_equal(self.pos[s].cpu().numpy(), po)
            self.want[s], self.err[s] = mo.astype(np.float64), np.zeros(mo.shape)
            dcpmla.mla_block_summary(self.cache, self.kv, self.t[s], out, 0, 1, self.S)
        assert _flag(ws) == 0 and np.array_equal(self.cache.cpu().numpy(), self.ref)

    def append(self):
        """One token a request: behind the kept rows of the shard that owns it."""
        lat = torch.randn(self.B, 512, generator=self.g).to(torch.bfloat16)
        rope = torch.randn(self.B, 64, generator=self.g).to(torch.bfloat16)
        token = _i32(self.lens)
        for s in range(self.N):
            own = token % self.N == s
            at = torch.where(own, self.rows[s], -1).to(torch.int32)
            dcpmla.mla_kv_append(lat.cuda(), rope.cuda(), at, _i32(range(self.B)), self.t[s], 0, 1, self.cache, self.kv)
            # the appended row starts without weight, at its token's position
            k = self.rows[s].long()[:, None]
            self.mass[s].scatter_(1, k, torch.where(own[:, None], 0.0, self.mass[s].gather(1, k)))
            self.pos[s].scatter_(1, k, torch.where(own[:, None], token[:, None], self.pos[s].gather(1, k)))
            before = self.rows[s]
            self.rows[s] = before + own.to(torch.int32)
            dcpmla.mla_block_summary(self.cache, self.kv, self.t[s], self.rows[s], 0, 1, self.S, before)
            self.ref, _ = oracle.kv_append(self.ref, self.kv, _bits(lat), _bits(rope), at.cpu().numpy(),
                                           np.arange(self.B, dtype=np.int32), self.tables[s], 0, 1)
            for b in range(self.B):
                if self.lens[b] % self.N == s:
                    j = self.ref_rows[s][b]
                    self.want[s][b, j], self.err[s][b, j], self.ref_pos[s][b, j] = 0.0, 0.0, self.lens[b]
                    self.ref_rows[s] = self.ref_rows[s] + (np.arange(self.B) == b).astype(np.int32)
        self.lens = self.lens + 1
        assert np.array_equal(self.cache.cpu().numpy(), self.ref)

    def seen(self, s, b, queries, i):
        """Places of the rows of shard s that query i of `queries` newest tokens sees, by their positions."""
        return np.nonzero(self.ref_pos[s][b, :self.ref_rows[s][b]] <= self.lens[b] - queries + i)[0]

    def values(self, s, b):
        """All rows of request b on shard s, in their order."""
        return ob.shard_rows(self.ref, self.kv, self.tables[s][b], self.ref_rows[s][b], 1, 0)[0]

    def summaries_are_current(self):
        fresh = torch.zeros_like(self.S)
        for s in range(self.N):
            dcpmla.mla_block_summary(self.cache, self.kv, self.t[s], self.rows[s], 0, 1, fresh)
            for b in range(self.B):
                used = self.tables[s][b, :-(-int(self.ref_rows[s][b]) // 64)]
                assert torch.equal(fresh[used], self.S[used])

    def check(self, out, lse, want, wlse):
        """The decode kernels' own bounds."""
        tol = (2e-3, 1e-4) if self.kv == "bf16" else (2e-2, 1e-3)
        assert np.abs(out.double().cpu().numpy() - want).max() <= tol[0] * np.abs(want).max()
        assert np.abs(lse.double().cpu().numpy() - wlse).max() <= tol[1]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("N", [1, 2])
def test_evicted_caches_are_appended_to_weighed_and_evicted_again(kv, N):
    H, topk, decay = 8, 3, 0.9
    c = _Caches(kv, N, H, [700, 66, 401], 12, 3)
    B = c.B
    parts, lses = torch.empty(N, B, H, 512, device="cuda"), torch.empty(N, B, H, device="cuda")
    out, lse = torch.empty(B, H, 512, device="cuda"), torch.empty(B, H, device="cuda")
    blocks = torch.empty(B, topk, dtype=torch.int32, device="cuda")
    dws = _ws(dcpmla.mla_decode_blocks_workspace_size(B, H, 1, c.stride, topk))
    mws = _ws(dcpmla.mla_attention_mass_workspace_size(B, H))
    for budget in (200, 197, 90):
        c.evict(budget, 2, 20)
        for _ in range(4):
            c.append()
            q = torch.randn(B, H, 576, generator=c.g).to(torch.bfloat16)
            o64, l64 = np.zeros((N, B, H, 512)), np.full((N, B, H), -np.inf)
            for s in range(N):
                dcpmla.mla_decode_blocks(q.cuda(), c.cache, kv, c.S, c.t[s], c.rows[s], 0, 1, topk, SCALE, parts[s],
                                         lses[s], dws, blocks)
                want, _ = ob.block_select(_bits(q)[:, None], c.S.cpu().numpy(), c.tables[s], c.ref_rows[s], 0, 1, topk,
                                          1, 1)
                assert np.array_equal(blocks.cpu().numpy(), want[:, 0])
                for b in range(B):
                    k = c.values(s, b)
                    pick = np.isin(np.arange(len(k)) // 64, want[b, 0])
                    o64[s, b], l64[s, b] = oracle.attention_with_lse(oracle.decode_bf16(_bits(q)[b]), k[pick], SCALE)
            dcpmla.dcp_merge(parts, lses, out, lse)
            c.check(out, lse, *oracle.dcp_merge(o64, l64))
            for s in range(N):
                dcpmla.mla_attention_mass(q.cuda(), c.cache, kv, c.t[s], c.rows[s], 0, 1, SCALE, lse, c.mass[s], mws,
                                          decay)
                c.want[s], e = ob.attention_mass(_bits(q)[:, None], c.ref, kv, c.tables[s], c.ref_rows[s], 0, 1, SCALE,
                                                 lse.double().cpu().numpy()[:, None], c.want[s], decay)
                c.err[s] = decay * c.err[s] + e
        c.summaries_are_current()
    assert _flag(dws) == 0 and _flag(mws) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("N", [1, 2, 3])
def test_draft_tokens_over_evicted_shards(kv, N):
    """Each (request, draft) is a request of its own, of as many rows as that draft sees on the shard: the kept
    ones and the drafts up to it that the shard owns."""
    H, Q, topk, decay = 8, 3, 2, 0.5
    c = _Caches(kv, N, H, [700, 66, 401], 8, 5)
    B = c.B
    c.evict(150, 2, 20)
    held = [r.clone() for r in c.rows]
    first = c.lens.copy()
    for _ in range(Q):
        c.append()
    q = torch.randn(B, Q, H, 576, generator=c.g).to(torch.bfloat16)
    flat = q.view(B * Q, H, 576).cuda()
    lens, tables = [], []
    for s in range(N):
        t = _i32(first)[:, None] + torch.arange(Q, device="cuda", dtype=torch.int32)[None]
        lens.append((held[s][:, None] + torch.cumsum(t % N == s, 1)).to(torch.int32).contiguous())      # [B, Q]
        tables.append(c.t[s].repeat_interleave(Q, 0).contiguous())
        for b in range(B):
            for i in range(Q):
                assert np.array_equal(c.seen(s, b, Q, i), np.arange(int(lens[s][b, i])))
    R = B * Q
    parts, lses = torch.empty(N, R, H, 512, device="cuda"), torch.empty(N, R, H, device="cuda")
    out, lse = torch.empty(R, H, 512, device="cuda"), torch.empty(R, H, device="cuda")
    ws = _ws(dcpmla.mla_decode_workspace_size(R, H))
    bws = _ws(dcpmla.mla_decode_blocks_workspace_size(R, H, 1, c.stride, topk))
    blocks = torch.empty(R, topk, dtype=torch.int32, device="cuda")
    for chosen in (True, False):
        o64, l64 = np.zeros((N, R, H, 512)), np.full((N, R, H), -np.inf)
        for s in range(N):
            n = lens[s].view(R)
            if chosen:
                dcpmla.mla_decode_blocks(flat, c.cache, kv, c.S, tables[s], n, 0, 1, topk, SCALE, parts[s], lses[s], bws,
                                         blocks)
                want, _ = ob.block_select(_bits(q).reshape(R, 1, H, 576), c.S.cpu().numpy(), tables[s].cpu().numpy(),
                                          n.cpu().numpy(), 0, 1, topk, 1, 1)
                assert np.array_equal(blocks.cpu().numpy(), want[:, 0])
            else:
                dcpmla.mla_decode_partial(flat, c.cache, kv, tables[s], n, 0, 1, None, SCALE, parts[s], lses[s], ws)
            for b in range(B):
                for i in range(Q):
                    seen = c.seen(s, b, Q, i)
                    if chosen:
                        seen = seen[np.isin(seen // 64, want[b * Q + i, 0])]
                    o64[s, b * Q + i], l64[s, b * Q + i] = oracle.attention_with_lse(
                        oracle.decode_bf16(_bits(q)[b, i]), c.values(s, b)[seen], SCALE)
        dcpmla.dcp_merge(parts, lses, out, lse)
        c.check(out, lse, *oracle.dcp_merge(o64, l64))
    # the weights: a call a draft, the newest first (it sees every row, so its call carries the decay)
    mws = _ws(dcpmla.mla_attention_mass_workspace_size(B, H))
    wl64 = lse.view(B, Q, H).double().cpu().numpy()
    for s in range(N):
        for i in reversed(range(Q)):
            d = decay if i == Q - 1 else 1.0
            dcpmla.mla_attention_mass(q[:, i].contiguous().cuda(), c.cache, kv, c.t[s], lens[s][:, i].contiguous(), 0, 1,
                                      SCALE, lse.view(B, Q, H)[:, i].contiguous(), c.mass[s], mws, d)
        got = c.mass[s].double().cpu().numpy()
        for b in range(B):
            n, k = c.ref_rows[s][b], c.values(s, b)
            want, err = decay * c.want[s][b, :n], np.zeros(n)
            for i in range(Q):
                see = np.zeros(n, bool)
                see[c.seen(s, b, Q, i)] = True
                qi = oracle.decode_bf16(_bits(q)[b, i])
                z = SCALE * (qi @ k.T)
                w = np.where(see, np.exp(z - wl64[b, i][:, None]), 0.0)
                # as in the oracle of the weights: 576 exact products summed in fp32, small values of q cut at 2^-17
                # of the largest in fp8, then the scale, a difference and the exponential
                e = 576 * 2.0 ** -24 * SCALE * (np.abs(qi) @ np.abs(k).T) + 2.0 ** -22 * (np.abs(z)
                                                                                         + np.abs(wl64[b, i][:, None]) + 1)
                if kv == "fp8":
                    e += SCALE * np.abs(k).sum(1) * np.abs(qi).max(1, keepdims=True) * 2.0 ** -17
                want += w.sum(0)
                err += (w * e).sum(0)
            err += 2.0 ** -23 * (want + 1)
            assert (np.abs(got[b, :n] - want) <= err).all()
    if N == 1:
        # one shard holds every draft: the batched form sees the same
        mo, ml = torch.empty(B, Q * H, 512, device="cuda"), torch.empty(B, Q * H, device="cuda")
        dcpmla.mla_decode_partial_multi(q.cuda(), c.cache, kv, c.t[0], c.rows[0], 0, 1, SCALE, mo, ml,
                                        _ws(dcpmla.mla_decode_workspace_size(B, Q * H)))
        c.check(mo.view(R, H, 512), ml.view(R, H), *oracle.dcp_merge(o64, l64))
    assert _flag(ws) == 0 and _flag(bws) == 0 and _flag(mws) == 0
