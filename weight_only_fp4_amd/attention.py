"""The attention half of a decoder layer: root-mean-square norm, rotary positions, the paged key-value cache and the
attention of one new token per sequence.  Argument marshalling only; the operators and their formulas are declared in
``include/nvfp4_w4a16.h``.

Caches are 4-d tensors [pages, heads, page_size, row], one for the keys and one for the values, in the format their
dtype names: bf16 / fp16 (the activations' type), float8_e4m3fn, or uint8 for NVFP4 (row = 9 * head_dim / 16; a (page,
head) block holds its tokens' codes, then their group scales).  ``kv_cache`` allocates them; any page and head strides
of whole 16-byte steps are taken, so a permuted view of another order works too (NVFP4 blocks are contiguous).
"""
from __future__ import annotations

import math
import struct

import torch

from . import _ACT_DTYPES, _check, _dev, lib, workspace

__all__ = ["rms_norm", "rms_norm_fp8", "rope", "rope_pair_axis", "kv_cache", "kv_write", "rope_kv_write", "kv_read",
           "paged_attention", "paged_attention_workspace_bytes"]

_KV_FORMATS = {torch.bfloat16: 0, torch.float16: 0, torch.float8_e4m3fn: 1, torch.uint8: 2}
_KV_STRUCT, _ROPE_STRUCT = struct.Struct("PPPP7q4i"), struct.Struct("PPPq4i")


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _act(name, t, ndim, device=None):
    """An activation tensor (bf16 or fp16) on the GPU with unit stride in its last dim; its dtype."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _ACT_DTYPES:
        raise ValueError(f"{name} must be a bf16 or fp16 tensor")
    _dev(name, t, None, ndim)
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.dtype


def _same(name, t, dtype, shape, device):
    """t must be a `dtype` tensor of `shape` on `device` with unit stride in its last dim."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dim")
    return t


def _vector(name, t, dtype, n, device):
    _same(name, t, dtype, (n,), device)
    return t


def _ld(t):
    """Leading dimension of a 2-d tensor (a single row's stride is of no account)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _steps(t):
    """Strides of the first two dims of a 3-d tensor; those of dims of one element are of no account."""
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


# ------------------------------------------------------------------- norm --

def _norm(x, weight, eps, residual, out, scales, residual_out):
    dt = _act("x", x, 2)
    T, N = x.shape
    dev = x.device
    _vector("weight", weight, dt, N, dev)
    if residual is not None:
        _same("residual", residual, dt, (T, N), dev)
        if residual_out is None:
            residual_out = torch.empty((T, N), dtype=dt, device=dev)
        else:
            _same("residual_out", residual_out, dt, (T, N), dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    _check(lib().nvfp4_rms_norm(x.data_ptr(), _ld(x), _addr(residual), 0 if residual is None else _ld(residual),
                                weight.data_ptr(), eps, out.data_ptr(), _ld(out), _addr(scales), _addr(residual_out),
                                0 if residual is None else _ld(residual_out), T, N, dt == torch.float16,
                                _raw_stream(dev)))
    return residual_out


def rms_norm(x, weight, eps=1e-6, residual=None, out=None, residual_out=None):
    """y = RNE16(h * rsqrt(mean(h^2) + eps) * weight) of each row, h = RNE16(x + residual) or x.  x [T, N] bf16 or fp16.
    Returns y, or (y, h) with a residual; residual_out (where h goes) may be ``residual`` itself."""
    dt = _act("x", x, 2)
    if out is None:
        out = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        _same("out", out, dt, x.shape, x.device)
    h = _norm(x, weight, eps, residual, out, None, residual_out)
    return out if residual is None else (out, h)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, out=None, scales=None, residual_out=None):
    """The norm with an 8-bit output: (codes float8_e4m3fn [T, N], scales fp32 [T]), and h with a residual; a value is
    code * scale, each row's scale its largest absolute value / 448."""
    _act("x", x, 2)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _same("out", out, torch.float8_e4m3fn, x.shape, x.device)
    if scales is None:
        scales = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    else:
        _vector("scales", scales, torch.float32, x.shape[0], x.device)
    h = _norm(x, weight, eps, residual, out, scales, residual_out)
    return (out, scales) if residual is None else (out, scales, h)


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


def _pack_rope(positions, inv_freq, pair_axis, interleaved, T, device):
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-d fp32 tensor (one frequency per rotated pair)")
    half = inv_freq.shape[0]
    _vector("inv_freq", inv_freq, torch.float32, half, device)
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2) or positions.shape[-1] != T:
        raise ValueError(f"positions must be an int32 tensor [{T}] or [axes, {T}]")
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _same("positions", positions, torch.int32, positions.shape, device)
    if pair_axis is not None:
        _vector("pair_axis", pair_axis, torch.int32, half, device)
    elif axes > 1:
        raise ValueError("positions with several axes need pair_axis")
    ld = positions.stride(0) if axes > 1 else T
    return _ROPE_STRUCT.pack(inv_freq.data_ptr(), positions.data_ptr(), _addr(pair_axis) or 0, ld, axes, 2 * half,
                             bool(interleaved), 0)


def rope(x, positions, inv_freq, pair_axis=None, interleaved=False, out=None):
    """Rotary positions: x [T, H, D] bf16 or fp16, its first 2 * len(inv_freq) columns turned in pairs (i, i + R/2), or
    (2i, 2i+1) with interleaved; positions int32 [T] or [axes, T], inv_freq fp32 [R/2], pair_axis int32 [R/2] (the axis
    whose position turns a pair; ``rope_pair_axis``).  out may be x."""
    dt = _act("x", x, 3)
    T, H, D = x.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=dt, device=x.device)
    else:
        _same("out", out, dt, (T, H, D), x.device)
    desc = _pack_rope(positions, inv_freq, pair_axis, interleaved, T, x.device)
    _check(lib().nvfp4_rope_apply(desc, x.data_ptr(), *_steps(x), out.data_ptr(), *_steps(out), T, H, D,
                                  dt == torch.float16, _raw_stream(x.device)))
    return out


# ------------------------------------------------------------------ cache --

def kv_cache(pages, heads, page_size, head_dim, dtype, device="cuda"):
    """(k_cache, v_cache), zero-filled: dtype bf16 or fp16, float8_e4m3fn, or uint8 for NVFP4."""
    if dtype not in _KV_FORMATS:
        raise ValueError("cache dtype must be bf16, fp16, float8_e4m3fn or uint8 (NVFP4)")
    row = head_dim * 9 // 16 if dtype == torch.uint8 else head_dim
    return tuple(torch.zeros((pages, heads, page_size, row), dtype=dtype, device=device) for _ in range(2))


def _cache_strides(name, c, packed):
    if c.dim() != 4:
        raise ValueError(f"{name} must be [pages, heads, page_size, row]")
    if c.stride(3) != 1 or (packed and c.shape[2] > 1 and c.stride(2) != c.shape[3]):
        raise ValueError(f"{name} must have contiguous {'blocks' if packed else 'rows'}")
    n = c.element_size()
    return [c.stride(i) * n if c.shape[i] > 1 else 0 for i in range(3)]


def _pack_cache(k_cache, v_cache, k_scale, v_scale, act, device):
    """(descriptor, heads, head_dim, pages, page_size) of a cache used with activations of dtype `act`."""
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(c, torch.Tensor) or c.dtype not in _KV_FORMATS:
            raise ValueError(f"{name} must be a bf16, fp16, float8_e4m3fn or uint8 (NVFP4) tensor")
        if c.device != device:
            raise ValueError(f"{name} is on {c.device}, expected {device}")
    kind = k_cache.dtype
    if v_cache.dtype != kind or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one dtype and one shape")
    fmt = _KV_FORMATS[kind]
    if fmt == 0 and kind != act:
        raise ValueError(f"a {kind} cache takes {kind} activations, got {act}")
    strides = _cache_strides("k_cache", k_cache, fmt == 2) + _cache_strides("v_cache", v_cache, fmt == 2)
    pages, heads, page_size, row = k_cache.shape
    D = row
    if fmt == 2:
        D = row * 16 // 9
        if row % 9 or D % 32:
            raise ValueError(f"an NVFP4 cache row of {row} bytes is not 9/16 of a head_dim that is a multiple of 32")
    for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
        if s is not None:
            if fmt == 0:
                raise ValueError(f"a 16-bit cache takes no {name}")
            _vector(name, s, torch.float32, heads, device)
    desc = _KV_STRUCT.pack(k_cache.data_ptr(), v_cache.data_ptr(), _addr(k_scale) or 0, _addr(v_scale) or 0, *strides,
                           pages, page_size, heads, D, fmt)
    return desc, heads, D, pages, page_size


def _append(q, k, v, rope_desc, q_out, k_cache, v_cache, slots, k_scale, v_scale):
    dt = _act("k", k, 3)
    dev = k.device
    T = k.shape[0]
    desc, heads, D, _, _ = _pack_cache(k_cache, v_cache, k_scale, v_scale, dt, dev)
    _same("k", k, dt, (T, heads, D), dev)
    _same("v", v, dt, (T, heads, D), dev)
    _vector("slots", slots, torch.int32, T, dev)
    if q is None:
        qa, qs, oa, os, Hq = None, (0, 0), None, (0, 0), 0
    else:
        qa, qs, oa, os, Hq = q.data_ptr(), _steps(q), q_out.data_ptr(), _steps(q_out), q.shape[1]
    _check(lib().nvfp4_kv_append(desc, rope_desc, qa, *qs, oa, *os, Hq, k.data_ptr(), *_steps(k), v.data_ptr(),
                                 *_steps(v), slots.data_ptr(), T, dt == torch.float16, _raw_stream(dev)))


def kv_write(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None):
    """Quantises (by the caches' dtype) and writes k, v [T, heads, D] to rows slots int32 [T] of the cache, row s of the
    cache being token s % page_size of page s // page_size; tokens with a negative slot are skipped.  k_scale, v_scale:
    fp32 [heads], the values' scales in an 8- or 4-bit cache (None: 1)."""
    _append(None, k, v, None, None, k_cache, v_cache, slots, k_scale, v_scale)


def rope_kv_write(q, k, v, positions, inv_freq, k_cache, v_cache, slots, k_scale=None, v_scale=None, pair_axis=None,
                  interleaved=False, out=None):
    """One launch for a step's new tokens: q [T, Hq, D] and k rotated as ``rope`` does, k and v written as ``kv_write``
    does.  Returns the rotated queries (out may be q)."""
    dt = _act("q", q, 3)
    T, Hq, D = q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype != dt:
        raise ValueError(f"k must be a {dt} tensor [{T}, heads, {D}]")
    if k.device != q.device:
        raise ValueError(f"k is on {k.device}, expected {q.device}")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    else:
        _same("out", out, dt, (T, Hq, D), q.device)
    desc = _pack_rope(positions, inv_freq, pair_axis, interleaved, T, q.device)
    _append(q, k, v, desc, out, k_cache, v_cache, slots, k_scale, v_scale)
    return out


def kv_read(k_cache, v_cache, slots, dtype=None, k_scale=None, v_scale=None, out=None):
    """(k, v) [T, heads, D] of dtype (default: a 16-bit cache's own, bf16 otherwise): rows slots int32 [T] of the cache,
    zeros for a slot outside it.  out: an optional (k, v) pair to write to."""
    if not isinstance(k_cache, torch.Tensor) or not k_cache.is_cuda:
        raise ValueError("k_cache must be a tensor on the GPU")
    dt = dtype or (k_cache.dtype if k_cache.dtype in _ACT_DTYPES else torch.bfloat16)
    if dt not in _ACT_DTYPES:
        raise ValueError("dtype must be bf16 or fp16")
    dev = k_cache.device
    desc, heads, D, _, _ = _pack_cache(k_cache, v_cache, k_scale, v_scale, dt, dev)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-d int32 tensor")
    T = slots.shape[0]
    _vector("slots", slots, torch.int32, T, dev)
    if out is None:
        k = torch.empty((T, heads, D), dtype=dt, device=dev)
        v = torch.empty((T, heads, D), dtype=dt, device=dev)
    else:
        k, v = out
        _same("out[0]", k, dt, (T, heads, D), dev)
        _same("out[1]", v, dt, (T, heads, D), dev)
    _check(lib().nvfp4_kv_read(desc, slots.data_ptr(), k.data_ptr(), *_steps(k), v.data_ptr(), *_steps(v), T,
                               dt == torch.float16, _raw_stream(dev)))
    return k, v


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
    of any sizes on one stream; made per call if not given."""
    dt = _act("q", q, 3)
    B, Hq, D = q.shape
    dev = q.device
    desc, heads, Dc, _, page_size = _pack_cache(k_cache, v_cache, k_scale, v_scale, dt, dev)
    if D != Dc:
        raise ValueError(f"q has {D} columns a head, the cache {Dc}")
    if Hq % heads:
        raise ValueError(f"{Hq} query heads are not a multiple of the cache's {heads}")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be an int32 tensor [{B}, max_pages]")
    max_pages = page_table.shape[1]
    _same("page_table", page_table, torch.int32, (B, max_pages), dev)
    _vector("lengths", lengths, torch.int32, B, dev)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=dt, device=dev)
    else:
        _same("out", out, dt, (B, Hq, D), dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if return_lse else None
    if workspace_buf is None:
        workspace_buf = workspace(paged_attention_workspace_bytes(B, Hq, heads, D, max_pages * page_size), dev)
    _check(lib().nvfp4_paged_attention(desc, q.data_ptr(), *_steps(q), page_table.data_ptr(), _ld(page_table),
                                       max_pages, lengths.data_ptr(), B, Hq,
                                       1.0 / math.sqrt(D) if scale is None else scale, int(window), out.data_ptr(),
                                       *_steps(out), _addr(lse), workspace_buf.data_ptr(), workspace_buf.numel(),
                                       dt == torch.float16, _raw_stream(dev)))
    return (out, lse) if return_lse else out
