"""A whole decode step of the example on the GPU: page tables, a layer with adapters, the experts in one call, the head and
the next token, prompts first; captured and replayed it gives the same bits as its operators called one by one, whose
own results are held to their definitions."""
import os
import sys

import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["bf16", "nvfp4"])
def test_prompts_then_captured_steps(kind):
    import decode_layer as example
    B, page, steps = 5, 16, 12
    layer = example.DecoderLayer(hidden=512, q_heads=8, kv_heads=2, head_dim=64, experts=8, topk=2, width=128)
    layer.add_adapters(3, 8)
    head = example.Head(1000, 512)
    prompts = [7, 0, 33, 16, 1]
    width = 5
    rng = np.random.default_rng(5)
    free = rng.permutation(B * width)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    adapter = ints([0, -1, 2, 2, 1])

    def start():
        """The prompts' keys and values in a cache of their own, and a step after them."""
        cache = example.new_cache(layer, B * width, page, kind)
        table, lengths, pages, used = ints(np.zeros((B, width))), ints([0] * B), ints(free), ints([0])
        plan = nv.kv_plan(lengths, ints(prompts), table, pages, used, page, sum(prompts) + 3)
        gen = torch.Generator(device=DEV)
        gen.manual_seed(9)
        k, v = torch.randn((2, sum(prompts) + 3, 2, 64), generator=gen, device=DEV).to(torch.bfloat16)
        nv.kv_write(k, v, cache["k"], cache["v"], plan.slots, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
        step = example.Step(layer, head, cache, table, plan.lengths.clone(), pages[int(plan.head):].clone(), page, adapter)
        step.tokens.copy_(ints([3, 1, 4, 1, 5]))
        return step, plan

    step, plan = start()
    want = ref.plan([0] * B, prompts, np.zeros((B, width)), free, 0, page, sum(prompts) + 3)
    assert np.array_equal(plan.slots.cpu().numpy(), want[0]) and np.array_equal(plan.lengths.cpu().numpy(), prompts)
    us = torch.rand((steps, B), generator=torch.Generator().manual_seed(1)).to(DEV)
    # warm-up and capture on a state of its own, then back to the start
    keep = [t.clone() for t in (step.lengths, step.used, step.tokens, step.table, step.cache["k"], step.cache["v"])]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step()
    for t, old in zip((step.lengths, step.used, step.tokens, step.table, step.cache["k"], step.cache["v"]), keep):
        t.copy_(old)
    plain, _ = start()
    lengths, table, used = list(prompts), want[6], 0
    rest = free[int(want[5][0]):]
    for i in range(steps):
        step.u.copy_(us[i])
        plain.u.copy_(us[i])
        graph.replay()
        tokens = plain.tokens.clone()
        p = nv.kv_plan(plain.lengths, plain.new, plain.table, plain.free_pages, plain.used, page, B)
        slots, positions, requests, after, offsets, used_now, table = ref.plan(lengths, [1] * B, table, rest, used, page, B)
        for g, w in zip((*p, plain.table), (slots, positions, requests, after, offsets, used_now, table)):
            assert np.array_equal(g.cpu().numpy(), w)
        lengths, used = after, int(used_now[0])
        plain.lengths.copy_(p.lengths)
        plain.used.copy_(p.head)
        x = head.embedding[tokens.long()]
        a, r = layer.attention(x, torch.zeros_like(x), p.positions, plain.cache, p.slots, plain.table, p.lengths,
                               plain.workspace, adapter)
        y, r = layer.experts_half(a, r)
        out = head.logits(y, r)
        got = nv.sample(out, us[i], plain.temperature, plain.top_k, plain.top_p)
        plain.tokens.copy_(got)
        torch.cuda.synchronize()
        assert torch.equal(logits, out) and torch.equal(step.tokens, got), i
        assert torch.equal(step.lengths, p.lengths) and torch.equal(step.table, plain.table)
        rows, t, tp = out.double().cpu().numpy(), np.float32(0.8).astype(float), np.float32(0.95).astype(float)
        for b in range(B):
            assert int(got[b]) == ref.sample_row(rows[b], float(us[i, b]), t, 50, tp)[0]
    assert torch.isfinite(out.float()).all()
    # the adapters count: without them the attention half's output is another one, but for the sequence that has none
    bare, _ = layer.attention(x, torch.zeros_like(x), p.positions, plain.cache, p.slots, plain.table, p.lengths,
                              plain.workspace)
    assert torch.equal(bare[1], a[1]) and not any(torch.equal(bare[i], a[i]) for i in (0, 2, 3, 4))
