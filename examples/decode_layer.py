#!/usr/bin/env python3
"""One decoder layer serving one new token per sequence, every operator from this package:

    norm (+ residual) -> FP4 QKV projection -> rotary positions + cache write -> paged attention -> FP4 output
    projection -> norm (+ residual) -> routing -> FP4 experts (fused FC1, FC2) -> combine

    python examples/decode_layer.py [--batch 16] [--context 4096] [--cache nvfp4|e4m3|bf16] [--steps 64]

Weights and contexts are random; the step is captured in one HIP graph and replayed, the lengths, positions and slots
advancing in device memory.  Prints the time of a step.
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

    def attention(self, x, residual, positions, cache, slots, table, lengths, workspace):
        """The attention half: x, residual [B, hidden] -> (its output, the residual with x added)."""
        B, hq, hk, d = x.shape[0], self.q_heads, self.kv_heads, self.head_dim
        h, residual = nv.rms_norm(x, self.norm1, residual=residual)
        qkv = nv.gemm(h, self.qkv, self.qkv_rows, self.hidden, self.qkv_scale).view(B, hq + 2 * hk, d)
        q = nv.rope_kv_write(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], positions, self.inv_freq, cache["k"],
                             cache["v"], slots, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
        o = nv.paged_attention(q, cache["k"], cache["v"], table, lengths, k_scale=cache["k_scale"],
                               v_scale=cache["v_scale"], workspace_buf=workspace)
        return nv.gemm(o.view(B, hq * d), self.o, self.hidden, hq * d, self.o_scale), residual

    def experts_half(self, x, residual):
        h, residual = nv.rms_norm(x, self.norm2, residual=residual)
        weights, ids = torch.topk(torch.softmax((h @ self.router.t()).float(), -1), self.topk)
        weights = (weights / weights.sum(-1, keepdim=True)).contiguous()
        offsets, row_token, token_row = nv.moe_route(ids.to(torch.int32), self.experts)
        a = nv.moe_fc1(h, row_token, offsets, self.fc1, self.experts, self.width, self.hidden, self.fc1_scale)
        y = nv.grouped_gemm(a, offsets, self.fc2, self.experts, self.hidden, self.width, self.fc2_scale)
        return nv.moe_combine(y, token_row, weights), residual

    def step(self, x, residual, positions, cache, slots, table, lengths, workspace):
        """lengths counts the new tokens: their keys and values are written before they are attended to."""
        x, residual = self.attention(x, residual, positions, cache, slots, table, lengths, workspace)
        return self.experts_half(x, residual)


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
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    torch.manual_seed(0)
    layer = DecoderLayer()
    width = -(-(a.context + a.steps + 8) // a.page)
    pages = a.batch * width
    table = torch.randperm(pages, device="cuda").to(torch.int32).view(a.batch, width)
    cache = new_cache(layer, pages, a.page, a.cache)
    # the context: random keys and values, written as a prompt's chunk is
    t = torch.arange(a.context, device="cuda")
    for b in range(a.batch):
        slots = (table[b, t // a.page] * a.page + (t % a.page)).to(torch.int32)
        k, v = torch.randn((2, a.context, layer.kv_heads, layer.head_dim), device="cuda").to(torch.bfloat16)
        nv.kv_write(k, v, cache["k"], cache["v"], slots, k_scale=cache["k_scale"], v_scale=cache["v_scale"])
    x, residual = torch.randn((2, a.batch, layer.hidden), device="cuda").to(torch.bfloat16)
    positions = torch.full((a.batch,), a.context, dtype=torch.int32, device="cuda")
    slots, lengths = torch.empty_like(positions), torch.empty_like(positions)
    workspace = nv.workspace(nv.paged_attention_workspace_bytes(a.batch, layer.q_heads, layer.kv_heads, layer.head_dim,
                                                                width * a.page), "cuda")
    rows = torch.arange(a.batch, device="cuda")

    def step():
        slots.copy_(table[rows, (positions // a.page).long()] * a.page + positions % a.page)
        lengths.copy_(positions + 1)
        out, res = layer.step(x, residual, positions, cache, slots, table, lengths, workspace)
        positions.add_(1)
        return out, res

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    began = time.perf_counter()
    n = a.steps - 1
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{a.batch} sequences of about {a.context} tokens, {a.cache} cache: {(time.perf_counter() - began) / n * 1e6:.1f} us "
          f"a layer and step, outputs finite: {bool(torch.isfinite(out.float()).all())}")


if __name__ == "__main__":
    main()
