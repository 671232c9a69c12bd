"""Blocks are ranked by what the softmax makes of their scores: with a negative
softmax scale the lowest products come first.
"""
import numpy as np
import pytest
import torch

import oracle
from long_context_decode_mla_b200 import dcpmla
from long_context_decode_mla_b200 import workload as wl
from oracle import block_cache as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dcpmla.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kv,impl", [("bf16", "auto"), ("bf16", "tc16"), ("fp8", "auto"), ("fp8", "simt")])
@pytest.mark.parametrize("scale", [0.07, -0.07, -1e-30, 0.0])
def test_choice_follows_the_sign_of_the_scale(kv, impl, scale):
    lens, H, topk = [2500, 400, 64, 1], 6, 4
    p = wl.make_problem("agentic" if kv == "fp8" else "dense", num_shards=1, batch=4, heads=H, seq_len=lens, seed=23)
    ni, d = p.numpy_inputs(), p.to("cuda")
    S = torch.zeros(d.kv_cache.shape[0], 608, dtype=torch.uint8, device="cuda")
    dcpmla.mla_block_summary(d.kv_cache, kv, d.block_tables[0], d.seq_lens, 0, 1, S)
    ws = torch.zeros(dcpmla.mla_decode_blocks_workspace_size(4, H, 1, d.block_tables.shape[2], topk), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty(4, H, 512, device="cuda"), torch.empty(4, H, device="cuda")
    blocks = torch.empty(4, topk, dtype=torch.int32, device="cuda")
    dcpmla.mla_decode_blocks(d.q, d.kv_cache, kv, S, d.block_tables[0], d.seq_lens, 0, 1, topk, scale, out, lse, ws,
                             blocks, 1, 1, impl=impl)
    bits = ni["q"] ^ 0x8000 if scale < 0 else ni["q"]
    want, _ = ob.block_select(bits[:, None], S.cpu().numpy(), ni["block_tables"][0], lens, 0, 1, topk, 1, 1)
    assert np.array_equal(blocks.cpu().numpy(), want[:, 0]) and int(ws[:4].view(torch.int32).item()) == 0
    for b, L in enumerate(lens):
        rows, pos = ob.shard_rows(ni["kv_cache"], kv, ni["block_tables"][0, b], L, 1, 0)
        pick = np.isin(np.arange(len(pos)) // 64, want[b, 0])
        o, l = oracle.attention_with_lse(oracle.decode_bf16(ni["q"][b]), rows[pick], scale)
        # the decode kernels' own bounds
        assert np.abs(out[b].double().cpu().numpy() - o).max() <= (2e-3 if kv == "bf16" else 2e-2) * np.abs(o).max()
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= (1e-4 if kv == "bf16" else 1e-3)
