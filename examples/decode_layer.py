#!/usr/bin/env python3
"""One decoder layer serving one new token per sequence, and the step around it, every operator from this package:

    page tables and slots -> norm (+ residual) -> FP4 QKV projection (+ adapters) -> rotary positions + cache write ->
    paged attention -> FP4 output projection (+ adapters) -> norm (+ residual) -> FP4 experts -> norm -> FP4 LM head ->
    the next token

    python examples/decode_layer.py [--batch 16] [--context 4096] [--cache nvfp4|e4m3|bf16] [--adapters 0] [--steps 64]

Weights and contexts are random; the step is captured in one HIP graph and replayed, the lengths, pages, positions and
tokens advancing in device memory.  Prints the time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_fp4_amd as nv

CACHE_DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "nvfp4": torch.uint8}


def fp4_weight(n, k, gen, experts=None):
    """Random canonical NVFP4 weights (codes, scales) with outputs of about the inputs' size, and the global scale."""
    shape = (n, k) if experts is None else (experts, n, k)
    codes = torch.randint(0, 256, (*shape[:-1], k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0x30, 0x40, (*shape[:-1], k // 16), generator=gen, device="cuda", dtype=torch.uint8)
    # E2M1 values have a root mean square of 2.9, these scale bytes of 1.1
    return codes, scales, torch.full((experts or 1,), 0.31 / k ** 0.5, device="cuda")


class DecoderLayer:
    def __init__(self, hidden=2048, q_heads=32, kv_heads=4, head_dim=128, experts=128, topk=8, width=768, theta=1e6,
                 seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.experts, self.topk, self.width = experts, topk, width
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(torch.bfloat16)
                                  for _ in range(2))
        self.qkv_rows = (q_heads + 2 * kv_heads) * head_dim
        c, s, self.qkv_scale = fp4_weight(self.qkv_rows, hidden, gen)
        self.qkv = nv.repack(c, s)
        c, s, self.o_scale = fp4_weight(hidden, q_heads * head_dim, gen)
        self.o = nv.repack(c, s)
        self.router = (torch.randn((experts, hidden), generator=gen, device="cuda") / hidden ** 0.5).to(torch.bfloat16)
        c, s, self.fc1_scale = fp4_weight(2 * width, hidden, gen, experts)
        self.fc1 = nv.repack_gated(c, s)
        c, s, self.fc2_scale = fp4_weight(hidden, width, gen, experts)
        self.fc2 = nv.repack(c, s)
        pairs = torch.arange(head_dim // 2, dtype=torch.float64)
        self.inv_freq = (theta ** (-2.0 * pairs / head_dim)).float().cuda()

    def add_adapters(self, n, rank, seed=1):
        """n random low-rank adapters beside the QKV and the output projection."""
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        pair = lambda rows, cols: tuple(  # noqa: E731
            (torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5).to(torch.bfloat16)
            for s in ((n, rank, cols), (n, rows, rank)))
        self.qkv_lora = pair(self.qkv_rows, self.hidden)
        self.o_lora = pair(self.hidden, self.q_heads * self.head_dim)
        self.lora_scale = torch.full((n,), 0.5, device="cuda")

    def adapted(self, y, x, lora, adapter):
        """y with the rows' adapters added in place (adapter int32 [B], or None)."""
        return y if adapter is None else nv.lora_add(y, x, *lora, adapter, scale=self.lora_scale, out=y)

    def attention(self, x, residual, positions, cache, slots, table, lengths, workspace, adapter=None):
        """The attention half: x, residual [B, hidden] -> (its output, the residual with x added)."""
        B, hq, hk, d = x.shape[0], self.q_heads, self.kv_heads, self.head_dim
        h, residual = nv.rms_norm(x, self.norm1, residual=residual)
        qkv = nv.gemm(h, self.qkv, self.qkv_rows, self.hidden, self.qkv_scale)
        qkv = self.adapted(qkv, h, getattr(self, "qkv_lora", None), adapter).view(B, hq + 2 * hk, d)
        q = nv.rope_kv_write(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], positions, self.inv_freq, cache["k"],
                             cache["v"], slots, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
        o = nv.paged_attention(q, cache["k"], cache["v"], table, lengths, k_scale=cache["k_scale"],
                               v_scale=cache["v_scale"], workspace_buf=workspace)
        o = o.view(B, hq * d)
        y = nv.gemm(o, self.o, self.hidden, hq * d, self.o_scale)
        return self.adapted(y, o, getattr(self, "o_lora", None), adapter), residual

    def experts_half(self, x, residual):
        h, residual = nv.rms_norm(x, self.norm2, residual=residual)
        weights, ids = torch.topk(torch.softmax((h @ self.router.t()).float(), -1), self.topk)
        weights = (weights / weights.sum(-1, keepdim=True)).contiguous()
        ids = ids.to(torch.int32)
        # a decoding batch: the whole layer in one call, which is faster while experts have few rows
        if x.shape[0] <= 64 and 2 * ids.numel() <= 3 * self.experts:
            return nv.moe_layer(h, ids, weights, self.fc1, self.fc2, self.experts, self.width, self.fc1_scale,
                                self.fc2_scale), residual
        offsets, row_token, token_row = nv.moe_route(ids, self.experts)
        a = nv.moe_fc1(h, row_token, offsets, self.fc1, self.experts, self.width, self.hidden, self.fc1_scale)
        y = nv.grouped_gemm(a, offsets, self.fc2, self.experts, self.hidden, self.width, self.fc2_scale)
        return nv.moe_combine(y, token_row, weights), residual

    def step(self, x, residual, positions, cache, slots, table, lengths, workspace, adapter=None):
        """lengths counts the new tokens: their keys and values are written before they are attended to."""
        x, residual = self.attention(x, residual, positions, cache, slots, table, lengths, workspace, adapter)
        return self.experts_half(x, residual)


class Head:
    """Embedding, last norm and FP4 LM head."""

    def __init__(self, vocab, hidden, seed=2):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.vocab, self.hidden = vocab, hidden
        self.embedding = torch.randn((vocab, hidden), generator=gen, device="cuda").to(torch.bfloat16)
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
        c, s, self.scale = fp4_weight(vocab, hidden, gen)
        self.weight = nv.repack(c, s)
        self.scale *= 3   # logits whose distribution has peaks

    def logits(self, x, residual):
        h, _ = nv.rms_norm(x, self.norm, residual=residual)
        return nv.gemm(h, self.weight, self.vocab, self.hidden, self.scale)


class Step:
    """One token for each of B sequences: its page and slot, a layer, the head, the next token.  All of a step's state is
    device memory that the step itself advances, so that a captured one replays."""

    def __init__(self, layer, head, cache, table, lengths, free_pages, page, adapter=None, temperature=0.8, top_k=50,
                 top_p=0.95):
        B, dev = table.shape[0], "cuda"
        self.layer, self.head, self.cache, self.table, self.page, self.adapter = layer, head, cache, table, page, adapter
        self.lengths, self.free_pages = lengths, free_pages
        self.new = torch.ones(B, dtype=torch.int32, device=dev)
        self.used = torch.zeros(1, dtype=torch.int32, device=dev)
        self.tokens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.u = torch.zeros(B, device=dev)
        self.temperature, self.top_p = torch.full((B,), temperature, device=dev), torch.full((B,), top_p, device=dev)
        self.top_k = torch.full((B,), top_k, dtype=torch.int32, device=dev)
        rows = [torch.empty(n, dtype=torch.int32, device=dev) for n in (B, B, B, B + 1)]
        # the lengths and the next free page's place are written over what they were
        self.plan = nv.KvPlan(*rows[:3], self.lengths, rows[3], self.used)
        self.workspace = nv.workspace(nv.paged_attention_workspace_bytes(
            B, layer.q_heads, layer.kv_heads, layer.head_dim, table.shape[1] * page), dev)

    def __call__(self):
        """Reads tokens and u (fresh random numbers), writes the next tokens over the tokens; returns the logits."""
        p = nv.kv_plan(self.lengths, self.new, self.table, self.free_pages, self.used, self.page, self.table.shape[0],
                       out=self.plan)
        x = self.head.embedding[self.tokens.long()]
        x, residual = self.layer.step(x, torch.zeros_like(x), p.positions, self.cache, p.slots, self.table, p.lengths,
                                      self.workspace, self.adapter)
        logits = self.head.logits(x, residual)
        nv.sample(logits, self.u, self.temperature, self.top_k, self.top_p, out=self.tokens)
        return logits


def new_cache(layer, pages, page_size, kind):
    k, v = nv.kv_cache(pages, layer.kv_heads, page_size, layer.head_dim, CACHE_DTYPES[kind])
    scale = None if kind == "bf16" else torch.full((layer.kv_heads,), 0.02, device="cuda")
    return {"k": k, "v": v, "k_scale": scale, "v_scale": scale}


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--context", type=int, default=4096)
    p.add_argument("--page", type=int, default=16)
    p.add_argument("--cache", choices=sorted(CACHE_DTYPES), default="nvfp4")
    p.add_argument("--adapters", type=int, default=0, help="low-rank adapters, one sequence in two with one of them")
    p.add_argument("--vocab", type=int, default=32000)
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    torch.manual_seed(0)
    layer = DecoderLayer()
    width = -(-(a.context + a.steps + 8) // a.page)
    pages = a.batch * width
    free = torch.randperm(pages, device="cuda").to(torch.int32)
    table = torch.zeros((a.batch, width), dtype=torch.int32, device="cuda")
    cache = new_cache(layer, pages, a.page, a.cache)
    # the context: random keys and values, written as a prompt's chunk is
    lengths = torch.zeros(a.batch, dtype=torch.int32, device="cuda")
    plan = nv.kv_plan(lengths, torch.full_like(lengths, a.context), table, free, torch.zeros_like(lengths[:1]), a.page,
                      a.batch * a.context)
    for slots in plan.slots.split(8192):
        k, v = torch.randn((2, len(slots), layer.kv_heads, layer.head_dim), device="cuda").to(torch.bfloat16)
        nv.kv_write(k, v, cache["k"], cache["v"], slots, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
    adapter = None
    if a.adapters:
        layer.add_adapters(a.adapters, 16)
        rows = torch.arange(a.batch, device="cuda")
        adapter = torch.where(rows % 2 == 0, rows // 2 % a.adapters, -1).to(torch.int32)
    step = Step(layer, Head(a.vocab, layer.hidden), cache, table, plan.lengths, free[int(plan.head):], a.page, adapter)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    began = time.perf_counter()
    n = a.steps - 1
    for _ in range(n):
        step.u.uniform_()
        graph.replay()
    torch.cuda.synchronize()
    print(f"{a.batch} sequences of about {a.context} tokens, {a.cache} cache: {(time.perf_counter() - began) / n * 1e6:.1f} us "
          f"a step of one layer and the head, logits finite: {bool(torch.isfinite(logits.float()).all())}")


if __name__ == "__main__":
    main()
