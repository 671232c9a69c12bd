"""Host-side refusals of the block-summary, block-sparse decode, attention-mass
and eviction calls: every case is turned down before a launch, so none needs a
GPU; and the binding's checks of the tensors it passes on as pointers."""
import ctypes

import numpy as np
import pytest
import torch

from long_context_decode_mla_b200 import dcpmla
from oracle import block_cache as ob

OK, EINVAL, EUNSUP, EWS, EALIGN = 0, -1, -2, -3, -4
P = 1 << 20          # a 16-byte aligned address that is never followed
BIG = 1 << 40

SUMMARY = dict(kv=P, dtype=1, nb=10, bs=64, table=P, stride=4, lens=P, first=None, batch=2, shard=0, n=1, out=P,
               flags=None, stream=None)
SELECT = dict(q=P, s=P, nb=10, bs=64, table=P, stride=4, lens=P, batch=2, heads=8, q_len=1, shard=0, n=1, topk=4, sink=1,
              recent=1, blocks=None, out=P, olens=P, ws=P, wsb=BIG, stream=None)
DECODE = dict(q=P, kv=P, dtype=1, s=P, nb=10, bs=64, table=P, stride=4, lens=P, batch=2, heads=8, q_len=1, shard=0, n=1,
              topk=4, sink=1, recent=1, scale=0.1, out=P, lse=P, blocks=None, ws=P, wsb=BIG, splits=4, impl=0,
              stream=None)
MASS = dict(q=P, kv=P, dtype=1, nb=10, bs=64, table=P, stride=4, lens=P, batch=2, heads=8, q_len=1, shard=0, n=1,
            scale=0.1, lse=P, decay=1.0, mass=P, mstride=256, ws=P, wsb=BIG, splits=4, stream=None)
EVICT = dict(kv=P, dtype=1, nb=10, bs=64, table=P, stride=4, lens=P, rows=None, batch=2, shard=0, n=1, mass=P, pos=None,
             mstride=256, budget=100, sink=1, recent=9, mo=P, po=None, ro=2 * P, ws=P, wsb=BIG, stream=None)
CALLS = {"mla_block_summary": SUMMARY, "mla_block_select": SELECT, "mla_decode_blocks": DECODE,
         "mla_attention_mass": MASS, "mla_cache_evict": EVICT}


def _refused(fn, **change):
    args = dict(CALLS[fn])
    assert set(change) <= set(args), change
    args.update(change)
    return getattr(dcpmla.lib(), fn)(*args.values())


SHARED = [(dict(n=0), EINVAL), (dict(shard=-1), EINVAL), (dict(shard=1), EINVAL), (dict(batch=-1), EINVAL),
          (dict(nb=0), EINVAL), (dict(stride=0), EINVAL), (dict(bs=0), EINVAL), (dict(bs=32), EUNSUP),
          (dict(table=None), EINVAL), (dict(lens=None), EINVAL)]
CACHE = [(dict(dtype=2), EINVAL), (dict(kv=None), EINVAL), (dict(kv=P + 8), EALIGN)]
QUERY = [(dict(heads=0), EINVAL), (dict(heads=65), EUNSUP), (dict(q_len=0), EINVAL), (dict(q_len=65), EINVAL),
         (dict(q=None), EINVAL), (dict(q=P + 2), EALIGN)]
WORK = [(dict(ws=None), EWS), (dict(wsb=256), EWS), (dict(ws=P + 4), EALIGN)]
CHOICE = [(dict(topk=0), EINVAL), (dict(sink=-1), EINVAL), (dict(recent=0), EINVAL), (dict(sink=3, recent=2), EINVAL),
          (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), EINVAL), (dict(stride=400000), EUNSUP),
          (dict(batch=70000), EUNSUP), (dict(batch=2000, q_len=64), EUNSUP), (dict(s=None), EINVAL),
          (dict(s=P + 4), EALIGN)]
NUMBERS = [(dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(splits=-1), EINVAL)]
REFUSED = {
    "mla_block_summary": SHARED + CACHE + [(dict(out=None), EINVAL), (dict(out=P + 8), EALIGN)],
    "mla_block_select": SHARED + QUERY + WORK + CHOICE + [(dict(out=None), EINVAL), (dict(olens=None), EINVAL)],
    "mla_decode_blocks": SHARED + CACHE + QUERY + WORK + CHOICE + NUMBERS + [
        (dict(out=None), EINVAL), (dict(lse=None), EINVAL), (dict(out=P + 4), EALIGN), (dict(impl=9), EINVAL),
        (dict(impl=0x102), EINVAL)],
    "mla_attention_mass": SHARED + CACHE + QUERY + WORK + NUMBERS + [
        (dict(lse=None), EINVAL), (dict(mass=None), EINVAL), (dict(mstride=0), EINVAL), (dict(decay=-0.5), EINVAL),
        (dict(decay=float("nan")), EINVAL)],
    "mla_cache_evict": SHARED + CACHE + WORK + [
        (dict(mass=None), EINVAL), (dict(mo=None), EINVAL), (dict(ro=None), EINVAL), (dict(rows=2 * P), EINVAL),
        (dict(lens=P + 16, ro=P + 16), EINVAL),
        (dict(budget=0), EINVAL), (dict(sink=-1), EINVAL), (dict(recent=-1), EINVAL),
        (dict(sink=50, recent=51), EINVAL), (dict(mstride=0), EINVAL), (dict(batch=70000), EUNSUP),
        (dict(stride=1 << 20, mstride=1 << 26), EUNSUP)],
}


@pytest.mark.parametrize("fn,change,code", [(f, c, r) for f, cases in REFUSED.items() for c, r in cases])
def test_refused(fn, change, code):
    assert _refused(fn, **change) == code


@pytest.mark.parametrize("fn", sorted(CALLS))
def test_an_empty_batch_is_no_work(fn):
    assert _refused(fn, batch=0) == OK


def test_workspace_sizes():
    L, n = dcpmla.lib(), ctypes.c_size_t(0)
    assert L.mla_block_select_workspace_size(1, 65, 1, 4, ctypes.byref(n)) == EUNSUP
    assert L.mla_block_select_workspace_size(1, 8, 1, 4, None) == EINVAL
    assert L.mla_decode_blocks_workspace_size(1, 8, 1, 4, 0, 1, ctypes.byref(n)) == EINVAL
    assert L.mla_attention_mass_workspace_size(-1, 8, 1, ctypes.byref(n)) == EINVAL
    assert L.mla_cache_evict_workspace_size(1, 0, ctypes.byref(n)) == EINVAL
    assert dcpmla.mla_cache_evict_workspace_size(4, 1000) >= 256 + 2 * 4 * 1000 * 4
    assert dcpmla.mla_decode_blocks_workspace_size(4, 8, 2, 100, 16, 8) > \
        dcpmla.mla_block_select_workspace_size(4, 8, 2, 100) + dcpmla.mla_decode_workspace_size(8, 8, 8)


def test_the_binding_checks_what_it_passes_on():
    q = torch.zeros(2, 8, 576, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kv, S = torch.zeros(3, 64, 656, dtype=torch.uint8), torch.zeros(3, 608, dtype=torch.uint8)
    ws, out, lse = torch.zeros(64, dtype=torch.uint8), torch.zeros(2, 8, 512), torch.zeros(2, 8)
    mass = torch.zeros(2, 256)
    good = dict(summary=lambda **k: dcpmla.mla_block_summary(kv, "fp8", k.get("t", t), k.get("n", n), 0, 1, k.get("S", S)),
                decode=lambda **k: dcpmla.mla_decode_blocks(k.get("q", q), kv, "fp8", k.get("S", S), k.get("t", t),
                                                            k.get("n", n), 0, 1, 4, 0.1, k.get("out", out), lse, ws),
                mass=lambda **k: dcpmla.mla_attention_mass(k.get("q", q), kv, "fp8", k.get("t", t), k.get("n", n), 0, 1,
                                                           0.1, k.get("lse", lse), k.get("mass", mass), ws),
                evict=lambda **k: dcpmla.mla_cache_evict(kv, "fp8", k.get("t", t), k.get("n", n), 0, 1,
                                                         k.get("mass", mass), 8, mass, n.clone(), ws))
    bad = dict(t=t.long(), n=n.long(), S=torch.zeros(3, 600, dtype=torch.uint8), q=q.float(), out=out[:, :4],
               lse=lse.double(), mass=torch.zeros(256, 2).T)
    used = dict(summary="tnS", decode=["t", "n", "S", "q", "out"], mass=["t", "n", "q", "lse", "mass"],
                evict=["t", "n", "mass"])
    for fn, names in used.items():
        for name in names:
            with pytest.raises(ValueError, match="must"):
                good[fn](**{name: bad[name]})
        with pytest.raises(ValueError, match="cuda device"):      # host memory goes to no kernel
            good[fn]()
    with pytest.raises(ValueError, match="must"):                   # a cache of fewer blocks than it is said to have
        dcpmla.mla_block_summary(kv, "bf16", t, n, 0, 1, S)
    with pytest.raises(ValueError, match="max_blocks"):
        dcpmla.DcpDecoder(2, 8, 1, block_topk=4, device="cpu")


# ----------------------------------------------------------- oracle pins ----

def test_oracle_ranks_by_the_distance_to_the_best_block():
    """Two heads of very different scale: each keeps its own best block first."""
    S = np.zeros((3, 608), np.uint8)
    S[:, 576:596] = np.ones((3, 5), np.float32).view(np.uint8)
    S[0, 0], S[1, 1], S[2, 2] = 100, 100, 50
    q = np.zeros((2, 576), np.float32)
    q[0, 0], q[1, 1] = 1000.0, 0.5
    r = ob.block_ranks(q, S)
    assert r[0] == 0 and r[1] == 0 and r[2] == -50.0


def test_oracle_eviction_fills_freed_places_in_order():
    mass = np.array([1, 9, 2, np.nan, 8, 7, 0, 9], np.float32)
    moves, new = ob.evict_plan(mass, np.arange(8), 8, 4, 0, 0)
    assert moves == [(4, 0), (5, 2), (7, 3)] and new == [4, 1, 5, 7]
    moves, new = ob.evict_plan(mass, np.arange(8), 8, 4, 1, 2)
    assert moves == [(6, 2), (7, 3)] and new == [0, 1, 6, 7]


def test_oracle_mass_sums_to_one_over_a_request():
    g = np.random.default_rng(0)
    rows = g.standard_normal((1, 64, 576)).astype(np.float32)
    cache = (rows.view(np.uint32) >> 16).astype(np.uint16).view(np.uint8).reshape(1, 64, 1152)
    q = (g.standard_normal((1, 1, 2, 576)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    k = ob.decode_bf16(cache.view(np.uint16).reshape(64, 576))
    s = 0.1 * ob.decode_bf16(q[0, 0]) @ k[:50].T
    lse = np.log(np.exp(s).sum(1))[None, None]
    m, e = ob.attention_mass(q, cache, "bf16", np.zeros((1, 1), int), [50], 0, 1, 0.1, lse, np.zeros((1, 64)), 1.0)
    assert abs(m.sum() - 2) < 1e-12 and not m[0, 50:].any() and e.max() < 1e-3
