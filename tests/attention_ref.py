"""Plain 64-bit forms of the norm, the rotary positions, the cache formats and single-token attention, on the CPU, with
the error bounds their tests use.  Test-side only.

Bounds count roundings: one to a type t is off by at most u(t) = finfo(t).eps / 2 relative (and by half the least
subnormal), one fp32 operation by 2^-24."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def u(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the least subnormal of a type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


# ------------------------------------------------------------------- norm --

def norm(h, weight, eps):
    """h, weight float64 -> (y, relative bound of its fp32 evaluation).  The squares are summed in a tree whose longest
    path is below N / 64 + 16 additions; rsqrt, the mean, eps and three products take 8 more roundings."""
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight
    return y, (h.shape[1] / 64 + 32) * U32


# ----------------------------------------------------------------- rotary --

def rope(x, positions, inv_freq, pair_axis, interleaved):
    """x float64 [T, H, D] -> (rotated, the sum |x0| + |x1| each value was made of (0 where it passes))."""
    T, H, D = x.shape
    half = len(inv_freq)
    axis = np.zeros(half, dtype=np.int64) if pair_axis is None else np.asarray(pair_axis, dtype=np.int64)
    pos = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    angle = pos[axis].T * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y, size = x.copy(), np.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def rope_bound(y, size, dtype):
    """Cosine and sine are off by 2^-25 + 2^-40, then a product and a sum each round: below 4 fp32 roundings of |x0| +
    |x1|; then the rounding to dtype."""
    off = size * 4 * U32
    return off + (np.abs(y) + off) * u(dtype) + least(dtype)


# ------------------------------------------------------------------ cache --

def round_small(x, mantissa, least_exponent, largest):
    """float64 -> the nearest small float, ties to even, saturating; NaN stays."""
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(np.abs(x))
        step = np.exp2(np.maximum(np.where(np.isfinite(x), e, 1) - 1, least_exponent) - mantissa)
        return np.clip(np.round(x / step) * step, -largest, largest)


def e4m3(x):
    return round_small(x, 3, -6, 448.0)


def e2m1(x):
    return round_small(x, 1, 0, 6.0)


def f32(x):
    """float64 rounded to fp32, as float64 (the exact product or quotient of two fp32 values rounds the same)."""
    with np.errstate(over="ignore"):
        return np.asarray(x).astype(np.float32).astype(np.float64)


def stored(x, scale, kind):
    """x float64 [T, heads, D] of 16-bit values, scale fp32 [heads] or None -> (codes as numbers [T, heads, D], group
    scales [T, heads, D / 16] or None): what the cache holds."""
    if kind == "same":
        return x, None
    g = np.ones(x.shape[1]) if scale is None else np.asarray(scale, dtype=np.float64)
    r = f32(1.0 / g)[None, :, None]
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "fp8":
            return e4m3(f32(x * r)), None
        b = x.reshape(*x.shape[:2], -1, 16)
        top = np.abs(b).max(3)
        sixth = float(np.float32(1.0 / 6.0))
        S = e4m3(f32(f32(top * r) * sixth))
        by = np.where(S > 0, f32(r / np.where(S > 0, S, 1.0)), 0.0)[..., None]
        codes = np.where(by == 0, 0.0, e2m1(f32(b * by)))
    return codes.reshape(x.shape), S


def value(codes, S, scale):
    """The float64 values stored rows stand for."""
    v = codes if S is None else codes * np.repeat(S, 16, axis=-1)
    return v if scale is None else v * np.asarray(scale, dtype=np.float64)[:, None]


def e4m3_of_bytes(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def raw_rows(cache, kind, D):
    """A cache tensor -> (codes as numbers [pages, heads, page, D], group scales or None)."""
    c = cache.detach().cpu()
    if kind == "same":
        return f64(c), None
    if kind == "fp8":
        return f64(c), None
    pages, heads, page, _ = c.shape
    flat = c.numpy().reshape(pages, heads, -1)
    byte = flat[:, :, :page * D // 2].reshape(pages, heads, page, D // 2)
    code = np.stack((byte & 15, byte >> 4), -1).reshape(pages, heads, page, D)
    number = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    return number, e4m3_of_bytes(flat[:, :, page * D // 2:]).reshape(pages, heads, page, D // 16)


# -------------------------------------------------------------- attention --

def attention(q, k, v, scale, types):
    """One query head group over its tokens.  q [G, D], k, v [n, D] float64 (the values the cache stands for); types:
    (products, output) dtypes.  Returns out, lse and their bounds.

    Scores: D products summed in fp32 and three more roundings (scale, q's power of two): (D + 4) 2^-24 sum|q k|; with
    fp16 products of a quantised cache q's small columns lose 2^-25 of the largest.  A weight is off by exp(2 ds) - 1 and
    the exponential's 2^-22, its rounding by u(products) and half a subnormal; sums over n tokens by (n + 64) 2^-24."""
    n, D = k.shape
    G = q.shape[0]
    if n == 0:
        z = np.zeros((G, D))
        return z, np.full(G, -np.inf), z + 0.0, np.zeros(G)
    s = q @ k.T * scale
    size = np.abs(q) @ np.abs(k).T * abs(scale)
    ds = (size * (D + 6) * U32 + np.abs(s) * 2 * U32
          + 2.0 ** -24 * np.abs(q).max(1, keepdims=True) * np.abs(k).sum(1)[None] * abs(scale)).max(1)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    total = w.sum(1, keepdims=True)
    out = w @ v / total
    each = (w @ np.abs(v)) / total
    p, o = types
    few = least(p) * np.abs(v).sum(0)[None] / total
    rel = (u(p) + np.expm1(4 * ds) + 2.0 ** -21 + 2 * (n + 64) * U32)[:, None]
    off = each * rel + few
    bound = off + (np.abs(out) + off) * u(o) + least(o)
    lse = (m + np.log(total))[:, 0]
    return out, lse, bound, 2 * ds + (n + 64) * U32 + np.abs(lse) * 4 * U32 + 2.0 ** -21


def default_scale(D):
    return 1.0 / math.sqrt(D)
