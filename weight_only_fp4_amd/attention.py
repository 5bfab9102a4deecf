"""The attention half of a decoder layer: root-mean-square norm, rotary positions, the paged key-value cache and the
attention of one new token per sequence.  Signatures only: the checks and the marshalling are compiled
(``csrc/binding.cpp``), the operators and their formulas are declared in ``include/nvfp4_w4a16.h``.  Arguments of the
wrong type, shape or device raise ``ValueError``, a refusal by the library ``Nvfp4Error``.

Caches are 4-d tensors [pages, heads, page_size, row], one for the keys and one for the values, in the format their
dtype names: bf16 / fp16 (the activations' type), float8_e4m3fn, or uint8 for NVFP4 (row = 9 * head_dim / 16; a (page,
head) block holds its tokens' codes, then their group scales).  ``kv_cache`` allocates them; any page and head strides
of whole 16-byte steps are taken, so a permuted view of another order works too (NVFP4 blocks are contiguous).
"""
from __future__ import annotations

import os

import torch

from . import Nvfp4Error, lib

__all__ = ["rms_norm", "rms_norm_fp8", "rope", "rope_pair_axis", "kv_cache", "kv_write", "rope_kv_write", "kv_read",
           "paged_attention", "paged_attention_workspace_bytes"]

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_attention.so")
_binding = None


def _native():
    """Load the compiled binding (never builds; see weight_only_fp4_amd.build)."""
    global _binding
    if _binding is None:
        lib()   # its own message if the library is missing
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: build it with `python -m weight_only_fp4_amd.build`")
        from . import _attention
        _attention.set_error(Nvfp4Error)
        _binding = _attention
    return _binding


# ------------------------------------------------------------------- norm --

def rms_norm(x, weight, eps=1e-6, residual=None, out=None, residual_out=None):
    """y = RNE16(h * rsqrt(mean(h^2) + eps) * weight) of each row, h = RNE16(x + residual) or x.  x [T, N] bf16 or fp16.
    Returns (y, h); h is None without a residual, and its tensor residual_out may be ``residual`` itself."""
    return (_binding or _native()).rms_norm(x, weight, eps, residual, out, None, residual_out, False)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, out=None, scales=None, residual_out=None):
    """The norm with an 8-bit output: (codes float8_e4m3fn [T, N], scales fp32 [T], h); a value is code * scale, each
    row's scale its largest absolute value / 448."""
    return (_binding or _native()).rms_norm(x, weight, eps, residual, out, scales, residual_out, True)


# ----------------------------------------------------------------- rotary --

def rope_pair_axis(sections, interleaved=False, device="cuda"):
    """The axis of every rotated pair as int32 [sum(sections)]: axis a takes sections[a] pairs, consecutive ones, or
    (interleaved) every len(sections)-th pair from pair a on while its section lasts, the first axis the rest."""
    total, n = sum(sections), len(sections)
    if not interleaved:
        axis = [a for a, s in enumerate(sections) for _ in range(s)]
    else:
        axis = [0] * total
        for a in range(1, n):
            for i in range(a, min(total, sections[a] * n), n):
                axis[i] = a
    return torch.tensor(axis, dtype=torch.int32, device=device)


def rope(x, positions, inv_freq, pair_axis=None, interleaved=False, out=None):
    """Rotary positions: x [T, H, D] bf16 or fp16, its first 2 * len(inv_freq) columns turned in pairs (i, i + R/2), or
    (2i, 2i+1) with interleaved; positions int32 [T] or [axes, T], inv_freq fp32 [R/2], pair_axis int32 [R/2] (the axis
    whose position turns a pair; ``rope_pair_axis``).  out may be x."""
    return (_binding or _native()).rope(x, positions, inv_freq, pair_axis, interleaved, out)


# ------------------------------------------------------------------ cache --

def kv_cache(pages, heads, page_size, head_dim, dtype, device="cuda"):
    """(k_cache, v_cache), zero-filled: dtype bf16 or fp16, float8_e4m3fn, or uint8 for NVFP4."""
    if dtype not in (torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.uint8):
        raise ValueError("cache dtype must be bf16, fp16, float8_e4m3fn or uint8 (NVFP4)")
    row = head_dim * 9 // 16 if dtype == torch.uint8 else head_dim
    return tuple(torch.zeros((pages, heads, page_size, row), dtype=dtype, device=device) for _ in range(2))


def kv_write(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None):
    """Quantises (by the caches' dtype) and writes k, v [T, heads, D] to rows slots int32 [T] of the cache, row s of the
    cache being token s % page_size of page s // page_size; tokens with a negative slot are skipped, the others' slots
    distinct.  k_scale, v_scale: fp32 [heads], the values' scales in an 8- or 4-bit cache (None: 1)."""
    (_binding or _native()).kv_append(None, k, v, None, None, None, False, k_cache, v_cache, slots, k_scale, v_scale,
                                      None)


def rope_kv_write(q, k, v, positions, inv_freq, k_cache, v_cache, slots, k_scale=None, v_scale=None, pair_axis=None,
                  interleaved=False, out=None):
    """One launch for a step's new tokens: q [T, Hq, D] and k rotated as ``rope`` does, k and v written as ``kv_write``
    does.  Returns the rotated queries (out may be q)."""
    if q is None:
        raise ValueError("q must be a bf16 or fp16 tensor")
    return (_binding or _native()).kv_append(q, k, v, positions, inv_freq, pair_axis, interleaved, k_cache, v_cache, slots,
                                             k_scale, v_scale, out)


def kv_read(k_cache, v_cache, slots, dtype=None, k_scale=None, v_scale=None, out=None):
    """(k, v) [T, heads, D] of dtype (default: a 16-bit cache's own, bf16 otherwise): rows slots int32 [T] of the cache,
    zeros for a slot outside it.  out: an optional (k, v) pair to write to."""
    if dtype is not None and dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype must be bf16 or fp16")
    k, v = out or (None, None)
    return (_binding or _native()).kv_read(k_cache, v_cache, slots, None if dtype is None else dtype == torch.float16,
                                           k_scale, v_scale, k, v)


# -------------------------------------------------------------- attention --

def paged_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_tokens):
    """Bytes of ``workspace`` a paged_attention call needs; max_tokens = page-table width * page_size."""
    n = int(lib().nvfp4_paged_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_tokens))
    if n < 0:
        raise ValueError(lib().nvfp4_last_error().decode())
    return n


def paged_attention(q, k_cache, v_cache, page_table, lengths, scale=None, k_scale=None, v_scale=None, window=0,
                    out=None, return_lse=False, workspace_buf=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the cached tokens of each sequence, token t of
    sequence b in page page_table[b, t // page_size] (int32 [B, max_pages]), lengths int32 [B] tokens (0: the output is
    0).  scale defaults to 1 / sqrt(D); window > 0: the last ``window`` tokens only.  Returns out [B, Hq, D], or (out,
    lse fp32 [B, Hq]).  workspace_buf: ``workspace(paged_attention_workspace_bytes(...), device)``, reusable by calls
    of any sizes on one stream; made per call if not given.  Batches of more than 2048 sequences are not split over their
    lengths: very long ones are better called for in smaller batches."""
    return (_binding or _native()).paged_attention(q, k_cache, v_cache, page_table, lengths, scale, k_scale, v_scale,
                                                   window, out, return_lse, workspace_buf)
