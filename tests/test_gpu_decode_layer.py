"""The example's decoder layer on the GPU: a step gives the same bits as its operators called one by one in their
unfused forms, for every cache format, and a context grown by single steps is the one attended to."""
import os
import sys

import pytest
import torch

import weight_only_fp4_amd as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "nvfp4"])
def test_steps_match_the_separate_operators(kind):
    import decode_layer as example
    B, page, n = 3, 16, 40
    layer = example.DecoderLayer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, experts=8, topk=2, width=128)
    width = -(-n // page)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, width).to(DEV)
    cache, plain = (example.new_cache(layer, B * width, page, kind) for _ in range(2))
    ws = nv.workspace(nv.paged_attention_workspace_bytes(B, 8, 2, 64, width * page), DEV)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    rows = torch.arange(B, device=DEV)
    for t in range(n):
        x, r = torch.randn((2, B, 512), generator=gen, device=DEV).to(torch.bfloat16)
        pos = torch.full((B,), t, dtype=torch.int32, device=DEV)
        slots = table[rows, t // page] * page + t % page
        out, res = layer.step(x, r, pos, cache, slots, table, pos + 1, ws)
        # the residual's addition, the norm, the rotation and the write by themselves
        added = (x.float() + r.float()).to(torch.bfloat16)
        h, none = nv.rms_norm(added, layer.norm1)
        assert none is None
        qkv = nv.gemm(h, layer.qkv, layer.qkv_rows, 512, layer.qkv_scale).view(B, 12, 64)
        q, k = nv.rope(qkv[:, :8], pos, layer.inv_freq), nv.rope(qkv[:, 8:10], pos, layer.inv_freq)
        nv.kv_write(k, qkv[:, 10:], plain["k"], plain["v"], slots, k_scale=plain["k_scale"], v_scale=plain["v_scale"])
        o = nv.paged_attention(q, plain["k"], plain["v"], table, pos + 1, k_scale=plain["k_scale"], v_scale=plain["v_scale"])
        y = nv.gemm(o.view(B, 512), layer.o, 512, 512, layer.o_scale)
        want, want_res = layer.experts_half(y, added)
        assert torch.equal(out, want) and torch.equal(res, want_res), t
    assert torch.equal(cache["k"].view(torch.uint8), plain["k"].view(torch.uint8))
    assert torch.equal(cache["v"].view(torch.uint8), plain["v"].view(torch.uint8))
    assert torch.isfinite(out.float()).all()
