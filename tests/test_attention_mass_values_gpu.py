"""Attention mass where its arithmetic can go wrong without a wrong sum: queries
that saw nothing, values that are not finite, log-sum-exps far from the scores,
and more CTAs than there are tiles.
"""
import numpy as np
import pytest
import torch

from long_context_decode_mla_b200 import dcpmla
from long_context_decode_mla_b200 import workload as wl
from oracle import block_cache as ob

pytestmark = pytest.mark.gpu

SCALE = wl.SOFTMAX_SCALE
LENS = [130, 64, 1]
ROPE = 520                   # a rope value: bf16 in both row types


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dcpmla.lib()
    torch.cuda.set_device(0)


def _case(kv, heads, q_len, seed=3):
    """Cache, table, lengths (CPU tensors) and queries of three requests."""
    p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=1, batch=len(LENS), heads=heads * q_len,
                        seq_len=LENS, seed=seed)
    return p, p.q.view(len(LENS), q_len, heads, 576).clone()


def _value(row, kv, d):
    """View of rope value d of one raw row."""
    return (row.view(torch.bfloat16)[d:d + 1] if kv == "bf16" else row[528:].view(torch.bfloat16)[d - 512:d - 511])


def _mass(p, q, kv, lse, start, decay=1.0, splits=0, scale=SCALE):
    B, Q, H = q.shape[:3]
    m = start.clone().cuda()
    ws = torch.zeros(dcpmla.mla_attention_mass_workspace_size(B, H, Q), dtype=torch.uint8, device="cuda")
    dcpmla.mla_attention_mass(q.cuda(), p.kv_cache.cuda(), kv, p.block_tables[0].cuda(), p.seq_lens.cuda(), 0, 1, scale,
                              lse.cuda(), m, ws, decay, splits)
    assert int(ws[:4].view(torch.int32).item()) == 0
    return m.cpu()


def _oracle(p, q, kv, lse, start, decay=1.0):
    bits = q.view(torch.int16).numpy().view(np.uint16)
    return ob.attention_mass(bits, p.kv_cache.numpy(), kv, p.block_tables[0].numpy(), LENS, 0, 1, SCALE,
                             lse.double().numpy(), start.numpy(), decay)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,q_len", [(3, 1), (64, 1), (8, 2), (40, 3)])
def test_a_query_that_saw_nothing_adds_nothing_whatever_it_holds(kv, heads, q_len):
    p, q = _case(kv, heads, q_len)
    lse = torch.full((len(LENS), q_len, heads), 4.0)
    lse[:, :, 0], lse[1] = -np.inf, -np.inf
    start = torch.rand(len(LENS), 192, generator=torch.Generator().manual_seed(1))
    want, err = _oracle(p, q, kv, lse, start)
    plain = _mass(p, q, kv, lse, start)
    assert (np.abs(plain.double().numpy() - want) <= err).all()
    for junk in (float("nan"), float("inf"), -float("inf")):
        bad = q.clone()
        bad[:, :, 0], bad[1] = junk, junk
        assert torch.equal(_mass(p, bad, kv, lse, start), plain)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,q_len", [(3, 1), (64, 1), (8, 2)])
def test_a_row_that_scores_minus_infinity_weighs_nothing(kv, heads, q_len):
    """A row's infinity reaches its own weights only, and there as the heads' scores say: exp(-inf) = 0."""
    p, q = _case(kv, heads, q_len)
    q[..., ROPE] = q[..., ROPE].abs() + 0.25
    lse = torch.full((len(LENS), q_len, heads), 4.0)
    start = torch.rand(len(LENS), 192, generator=torch.Generator().manual_seed(2))
    want, err = _oracle(p, q, kv, lse, start)
    b, j = 0, 70
    _value(p.kv_cache[int(p.block_tables[0, b, j // 64]), j % 64], kv, ROPE)[0] = -float("inf")
    got = _mass(p, q, kv, lse, start)
    assert got[b, j] == start[b, j]
    want[b, j] = start[b, j]
    assert (np.abs(got.double().numpy() - want) <= err).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_row_of_nan_is_nan_for_those_who_saw_it_only(kv):
    p, q = _case(kv, 4, 1)
    b, j = 0, 3
    _value(p.kv_cache[int(p.block_tables[0, b, 0]), j], kv, ROPE)[0] = float("nan")
    start = torch.ones(len(LENS), 192)
    seen = _mass(p, q, kv, torch.full((len(LENS), 1, 4), 4.0), start)
    assert torch.isnan(seen[b, j]) and int(torch.isnan(seen).sum()) == 1
    assert torch.equal(_mass(p, q, kv, torch.full((len(LENS), 1, 4), -np.inf), start), start)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [SCALE, 0.1, 1.0, -0.07])
def test_a_log_sum_far_above_the_scores_leaves_nothing(kv, scale):
    """exp(score - lse) is zero from some 200 on, up to the largest finite log-sum."""
    p, q = _case(kv, 5, 1)
    start = torch.rand(len(LENS), 192, generator=torch.Generator().manual_seed(5))
    # products of 576 values of about 1 stay below 200, so that exp() of these differences underflows
    for far in (1e3, 3e8, 1.3e9, 7.7e9, 1e12, 3.3e19, 2.2e30, 1.9e38, 3.4e38, np.inf):
        lse = torch.full((len(LENS), 1, 5), far)
        assert torch.equal(_mass(p, q, kv, lse, start, scale=scale), start), far


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("splits", [6, 149, 1 << 20, (1 << 31) - 1])
def test_any_number_of_ctas(kv, splits):
    """More CTAs than tiles, up to the largest int: the same bits as one CTA."""
    p, q = _case(kv, 7, 2)
    lse = torch.full((len(LENS), 2, 7), 4.0)
    start = torch.rand(len(LENS), 192, generator=torch.Generator().manual_seed(6))
    assert torch.equal(_mass(p, q, kv, lse, start, splits=splits), _mass(p, q, kv, lse, start, splits=1))
