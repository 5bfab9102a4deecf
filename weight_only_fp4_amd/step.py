"""What a decode step runs around and between its layers' linears and attention: page tables and slots from the requests'
lengths, low-rank adapters beside a shared projection, the expert layer of a few tokens in one call, and the choice of
the next token.  Signatures only, as in ``attention``: the checks are compiled (``csrc/binding_step.h``), the operators
and their formulas are declared in ``include/nvfp4_w4a16.h``.  Arguments of the wrong type, shape or device raise
``ValueError``, a refusal by the library ``Nvfp4Error``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MOE_SILU_GLU, lib
from . import attention as _attention

__all__ = ["KvPlan", "kv_plan", "lora_add", "lora_workspace_bytes", "moe_layer", "moe_layer_workspace_bytes", "sample",
           "sample_workspace_bytes"]


def _bytes(name, *sizes):
    n = int(getattr(lib(), name)(*sizes))
    if n < 0:
        raise ValueError(lib().nvfp4_last_error().decode())
    return n


# ------------------------------------------------------------------- plan --

class KvPlan(NamedTuple):
    """What ``kv_plan`` gives, all int32: of each row of the step its ``slots``, ``positions`` and ``requests`` (-1, 0, -1
    where it has none); of each request its ``lengths`` with the new tokens; ``offsets`` [requests + 1], the first row
    of each request (its last new token is row offsets[b + 1] - 1); ``head`` [1], the next free page's place."""
    slots: torch.Tensor
    positions: torch.Tensor
    requests: torch.Tensor
    lengths: torch.Tensor
    offsets: torch.Tensor
    head: torch.Tensor


def kv_plan(cached, new, page_table, free_pages, free_head, page_size, tokens, out=None):
    """Page tables, slots and positions of a step's new tokens.  cached, new int32 [B]: tokens that each request has in
    the cache and brings; page_table int32 [B, max_pages], completed in place with pages from free_pages int32 [F], from
    place free_head int32 [1] on; tokens: the step's rows, which hold the requests' new tokens one request after another.
    The slots go to ``rope_kv_write`` or ``kv_write``, the positions to ``rope``, page_table and lengths to
    ``paged_attention``.  A request whose pages or rows do not fit gets no page and no slots, and keeps its cached length.
    out: a KvPlan (or six tensors) to write to, whose lengths may be cached itself and its head free_head."""
    return KvPlan(*(_attention._binding or _attention._native()).kv_plan(cached, new, page_table, free_pages, free_head,
                                                                         page_size, tokens, out))


# ------------------------------------------------------------------- lora --

def lora_workspace_bytes(tokens, K, N, rank):
    """Bytes of ``workspace`` a lora_add call needs."""
    return _bytes("nvfp4_lora_workspace_bytes", tokens, K, N, rank)


def lora_add(y, x, a, b, adapter, scale=None, out=None, workspace_buf=None):
    """y + scale[i] * (x a[i]^T) b[i]^T of each row, i = adapter of the row: y [T, N], x [T, K], a [L, r, K], b [L, N, r]
    bf16 or fp16, adapter int32 [T] (rows with an index outside [0, L) stay as y), scale fp32 [L] (None: 1); r a multiple
    of 8 up to 128.  out may be y.  workspace_buf: ``workspace(lora_workspace_bytes(...), device)``, made per call if not
    given."""
    return (_attention._binding or _attention._native()).lora_add(y, x, a, b, adapter, scale, out, workspace_buf)


# -------------------------------------------------------------------- moe --

def moe_layer_workspace_bytes(tokens, topk, E, H, I):
    """Bytes of ``workspace`` a moe_layer call needs."""
    return _bytes("nvfp4_moe_layer_workspace_bytes", tokens, topk, E, H, I)


def moe_layer(x, topk_ids, topk_weights, w1, w2, E, I, g1=None, g2=None, divisor=False, activation=MOE_SILU_GLU,
              pre_scale1=None, pre_scale2=None, mxfp4=False, out=None, workspace_buf=None):
    """The whole expert layer of up to 64 tokens (512 (token, slot) pairs) in two launches: x [T, H] bf16 or fp16,
    topk_ids int32 and topk_weights fp32 [T, k] (ids outside [0, E) add nothing), w1 from ``repack_gated`` (MOE_SILU_GLU)
    or ``repack`` (MOE_RELU2), w2 from ``repack``, g1 and g2 fp32 [E]; mxfp4: blobs of the MXFP4 repacks and no g1, g2.
    pre_scale1 [H], pre_scale2 [I]: the products' pre-quant scales.  Nothing else is rounded to 16 bits than X' and the output.
    workspace_buf: ``workspace(moe_layer_workspace_bytes(...), device)``, reusable by moe_layer calls of any sizes on one
    stream; made per call if not given.  More tokens: ``moe_route``, ``moe_fc1``, ``grouped_gemm``, ``moe_combine``."""
    return (_attention._binding or _attention._native()).moe_layer(x, topk_ids, topk_weights, w1, w2, E, I, g1, g2,
                                                                   divisor, activation, pre_scale1, pre_scale2, mxfp4,
                                                                   out, workspace_buf)


# ----------------------------------------------------------------- sample --

def sample_workspace_bytes(rows, vocab):
    """Bytes of ``workspace`` a sample call needs."""
    return _bytes("nvfp4_sample_workspace_bytes", rows, vocab)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, return_logprobs=False, out=None,
           workspace_buf=None):
    """One token a row, int32 [B], from logits [B, V] bf16, fp16 or fp32 and given random numbers u fp32 [B] in [0, 1);
    every setting is a tensor [B] or None: temperature fp32 (0: the largest logit), top_k int32 (0: off), top_p fp32 (1:
    off), min_p fp32 (0: off).  The filters keep the most likely tokens, of equal logits those of lower index; the token is
    the first kept one, by index, whose cumulative weight exceeds u times the total.  A row of -inf gives -1.
    return_logprobs: also the tokens' log probabilities among those kept, fp32 [B].  workspace_buf:
    ``workspace(sample_workspace_bytes(...), device)``, made per call if not given."""
    return (_attention._binding or _attention._native()).sample(logits, u, temperature, top_k, top_p, min_p,
                                                                return_logprobs, out, workspace_buf)
