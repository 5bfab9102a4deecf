"""Cases of the attention half of a decoder layer: normalisation, rotary positions, the paged key-value cache and
attention of one new token over it.

Every case names its operator in ``op``:

* ``norm``: root-mean-square norm of ``rows`` rows of ``cols`` values with the residual's addition, its output in 16
  bits or in E4M3 with one scale per row;
* ``rope``: rotary positions with ``axes`` axes on ``heads`` heads;
* ``append``: the new tokens of a step: queries and keys rotated, keys and values quantised into the paged cache, and
  the same rows read back in 16 bits;
* ``attend``: attention of one new token per sequence over the paged cache.

Caches are [pages, kv_heads, page_size, row]: 16-bit values, E4M3 values (row = head_dim), or bytes of the 4-bit
format, where a (page, head) block of page_size * 9 * head_dim / 16 bytes holds the codes of all its tokens (two E2M1
codes a byte, the even column in the low nibble), then their E4M3 scales (one per 16 columns).
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DEVICE = "cuda:0"
_EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the norm before a layer's projection, one user decoding: a launch and one row
        {"name": "norm-1x4096", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True, "fp8": False},
        # a ragged batch of prompts into an 8-bit projection
        {"name": "norm-fp8-777x5120", "op": "norm", "rows": 777, "cols": 5120, "dtype": "fp16", "residual": True,
         "fp8": True},
        # a long prompt's chunk, hidden size of the prefill workload
        {"name": "norm-8192x5120", "op": "norm", "rows": 8192, "cols": 5120, "dtype": "bf16", "residual": True,
         "fp8": False},
        # queries and keys of a decoding batch whose positions have three axes (time, height, width)
        {"name": "rope-16x36", "op": "rope", "tokens": 16, "heads": 36, "head_dim": 128, "rotary": 128, "axes": 3,
         "interleaved": False, "dtype": "bf16", "first": 900000},
        # an image tower: two axes (height, width), a head size that is no power of two
        {"name": "rope-image-5003x16", "op": "rope", "tokens": 5003, "heads": 16, "head_dim": 80, "rotary": 80,
         "axes": 2, "interleaved": False, "dtype": "fp16", "first": 0},
        # a decoding batch far into its texts, 4-bit cache
        {"name": "append-16-fp4", "op": "append", "tokens": 16, "q_heads": 32, "kv_heads": 4, "head_dim": 128,
         "rotary": 128, "axes": 1, "interleaved": False, "page": 16, "cache": "fp4", "dtype": "bf16",
         "first": 1000000, "padding": 1},
        # a prompt's chunk with images in it, 8-bit cache
        {"name": "append-4096-fp8", "op": "append", "tokens": 4096, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "rotary": 128, "axes": 3, "interleaved": False, "page": 64, "cache": "fp8", "dtype": "bf16", "first": 12000,
         "padding": 0},
        # short prompts batched, partly rotated neighbouring pairs, 16-bit cache, the batch padded
        {"name": "append-1003-16bit", "op": "append", "tokens": 1003, "q_heads": 24, "kv_heads": 24, "head_dim": 64,
         "rotary": 32, "axes": 1, "interleaved": True, "page": 32, "cache": "same", "dtype": "fp16", "first": 0,
         "padding": 21},
        # the first tokens of one conversation
        {"name": "attend-1x130", "op": "attend", "batch": 1, "length": 130, "ragged": False, "q_heads": 32,
         "kv_heads": 4, "head_dim": 128, "page": 16, "cache": "same", "dtype": "bf16", "window": 0},
        # one user with a book in the context, 8-bit cache
        {"name": "attend-1x131072-fp8", "op": "attend", "batch": 1, "length": 131072, "ragged": False, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "cache": "fp8", "dtype": "fp16", "window": 0},
        # a serving batch at all ages, 4-bit cache
        {"name": "attend-64x8191-fp4", "op": "attend", "batch": 64, "length": 8191, "ragged": True, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "cache": "fp4", "dtype": "bf16", "window": 0},
        # a full serving batch, 16-bit cache
        {"name": "attend-32x8192", "op": "attend", "batch": 32, "length": 8192, "ragged": False, "q_heads": 40,
         "kv_heads": 8, "head_dim": 128, "page": 32, "cache": "same", "dtype": "bf16", "window": 0},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "append", "attend"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "norm":
        cols = rng.choice((128, 1040, 2048, 4096, 5120, 7168, 8192, 14336, rng.randrange(64, 8192)))
        rows = _log_int(rng, 1, min(8192, 8192 * 5120 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7,
                "fp8": rng.random() < 0.4}
    if op == "rope":
        dim, rotary = rng.choice(((64, 64), (64, 32), (80, 80), (96, 96), (128, 128), (128, 64), (192, 64), (256, 256)))
        heads = rng.choice((8, 16, 20, 36, 40))
        return {"op": op, "tokens": _log_int(rng, 1, 8192 * 128 // dim * 16 // heads), "heads": heads, "head_dim": dim,
                "rotary": rotary, "axes": rng.choice((1, 2, 3)), "interleaved": rng.random() < 0.3, "dtype": dtype,
                "first": rng.choice((0, 5000, 1000000))}
    cache = rng.choice(("same", "fp8", "fp4"))
    page = rng.choice((16, 32, 64, 128))
    dim = rng.choice((64, 128, 128, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    q = kv * rng.choice((1, 3, 4, 5, 8, 16))
    if op == "append":
        tokens = _log_int(rng, 1, max(1, 4096 * 48 * 128 // ((q + 2 * kv) * dim) // 2))
        return {"op": op, "tokens": tokens, "q_heads": q, "kv_heads": kv, "head_dim": dim,
                "rotary": rng.choice((dim, dim // 2)), "axes": rng.choice((1, 1, 3)), "interleaved": rng.random() < 0.3,
                "page": page, "cache": cache, "dtype": dtype, "first": rng.choice((0, 5000, 1000000)),
                "padding": rng.choice((0, tokens // 16))}
    batch = _log_int(rng, 1, 128)
    most = min(131072, 32 * 8192 * 8 * 128 // (batch * kv * dim) // max(1, q // kv // 5))
    return {"op": op, "batch": batch, "length": _log_int(rng, 1, max(1, most)), "ragged": rng.random() < 0.6,
            "q_heads": q, "kv_heads": kv, "head_dim": dim, "page": page, "cache": cache, "dtype": dtype,
            "window": rng.choice((0, 0, 1024))}


def _lengths(case):
    """Cached tokens of each sequence: equal, or spread over a factor of 64 with one sequence that has none."""
    n, longest = case["batch"], case["length"]
    if not case["ragged"] or n == 1:
        return [longest] * n
    got = [max(1, int(longest * 2.0 ** (-6.0 * ((i * 7) % n) / n))) for i in range(n)]
    return [0 if i == n // 2 else x for i, x in enumerate(got)]


# ------------------------------------------------------------------ inputs --

def _normal(shape, gen, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen, device=_DEVICE) * sigma).to(dtype)


def _frequencies(rotary):
    i = torch.arange(rotary // 2, dtype=torch.float64)
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64), -2.0 * i / rotary).to(torch.float32).to(_DEVICE)


def _pair_axis(rotary, axes):
    """The axis of each rotated pair: the axes take the pairs in consecutive sections."""
    return ((torch.arange(rotary // 2) * axes) // (rotary // 2)).to(torch.int32).to(_DEVICE)


def _positions(tokens, axes, first, gen):
    """int32 [axes, tokens]: a text's positions, or those of a grid of patches after the text before it."""
    t = torch.arange(tokens, device=_DEVICE, dtype=torch.int64)
    start = int(torch.randint(0, 1000, (1,), generator=gen, device=_DEVICE)) + first
    if axes == 1:
        return (t + start).to(torch.int32)[None]
    side = max(1, int(math.sqrt(tokens)))
    grid = torch.stack((t // side, t % side, t // (4 * side))[:axes])
    return (grid + start).to(torch.int32)


def _cache(pages, case, gen, fill):
    """A cache and its per-head scales (None where values are kept in 16 bits).  fill: rows of normal values."""
    heads, dim, page, kind = case["kv_heads"], case["head_dim"], case["page"], case["cache"]
    dtype = _DTYPES[case["dtype"]]
    if kind == "same":
        shape, store, scale = (pages, heads, page, dim), dtype, None
    else:
        scale = 0.01 + 0.01 * torch.rand(heads, generator=gen, device=_DEVICE)
        shape, store = ((pages, heads, page, dim), torch.float8_e4m3fn) if kind == "fp8" else \
            ((pages, heads, page, dim * 9 // 16), torch.uint8)
    cache = torch.zeros(shape, dtype=store, device=_DEVICE)
    if fill:
        x = _normal((pages, heads, page, dim), gen, dtype)
        if kind == "same":
            cache = x
        elif kind == "fp8":
            cache = _to_e4m3(x.float(), scale.reciprocal()[:, None, None])
        else:
            codes, scales = _to_fp4(x.float(), scale.reciprocal()[:, None, None])
            c, s = _fp4_parts(cache, dim)
            c.copy_(codes)
            s.copy_(scales)
    return cache, scale


def prepare(case, seed):
    gen = torch.Generator(device=_DEVICE)
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    op = case["op"]
    state = {"case": case}
    if op == "norm":
        shape = (case["rows"], case["cols"])
        state["x"] = _normal(shape, gen, dtype)
        state["residual"] = _normal(shape, gen, dtype, 4.0) if case["residual"] else None
        state["weight"] = (1.0 + 0.2 * torch.randn(case["cols"], generator=gen, device=_DEVICE)).to(dtype)
        return state
    if op == "attend":
        lengths = _lengths(case)
        page = case["page"]
        width = -(-case["length"] // page)
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device=_DEVICE).to(torch.int32)
        index = np.zeros((case["batch"], width), dtype=np.int64)
        done = 0
        for b, n in enumerate(need):
            index[b, :n] = np.arange(done, done + n)
            done += n
        state["table"] = order[torch.from_numpy(index).to(_DEVICE)].contiguous()
        state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=_DEVICE)
        state["q"] = _normal((case["batch"], case["q_heads"], case["head_dim"]), gen, dtype, 1.5)
        state["k_cache"], state["k_scale"] = _cache(pages, case, gen, True)
        state["v_cache"], state["v_scale"] = _cache(pages, case, gen, True)
        state["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=_DEVICE)
        return state
    tokens, dim = case["tokens"], case["head_dim"]
    state["positions"] = _positions(tokens, case["axes"], case["first"], gen)
    state["inv_freq"] = _frequencies(case["rotary"])
    state["pair_axis"] = _pair_axis(case["rotary"], case["axes"]) if case["axes"] > 1 else None
    if op == "rope":
        state["x"] = _normal((tokens, case["heads"], dim), gen, dtype)
        return state
    # queries, keys and values are slices of one projection's output
    q, kv, page = case["q_heads"], case["kv_heads"], case["page"]
    qkv = _normal((tokens, q + 2 * kv, dim), gen, dtype)
    state["q"], state["k"], state["v"] = qkv[:, :q], qkv[:, q:q + kv], qkv[:, q + kv:]
    pages = -(-tokens // page) + 3
    order = torch.randperm(pages - 1, generator=gen, device=_DEVICE)   # the last page belongs to no sequence
    t = torch.arange(tokens, device=_DEVICE) + int(torch.randint(0, page, (1,), generator=gen, device=_DEVICE))
    slots = order[t // page] * page + t % page
    if case["padding"]:
        slots[tokens - case["padding"]:] = -1
    state["slots"] = slots.to(torch.int32)
    state["k_cache"], state["k_scale"] = _cache(pages, case, gen, False)
    state["v_cache"], state["v_scale"] = _cache(pages, case, gen, False)
    return state


# -------------------------------------------------------------- plain forms --

def _to_e4m3(x, r):
    return (x * r).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _from_e4m3(b):
    return b.view(torch.float8_e4m3fn).to(torch.float32)


def _to_fp4(x, r):
    """fp32 [..., D] and the reciprocal of its scale -> (codes uint8 [..., D/2], scale bytes [..., D/16])."""
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    r = r.unsqueeze(-1)
    largest = blocks.abs().amax(-1, keepdim=True)
    sixth = torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device)
    s8 = ((largest * r) * sixth).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(torch.float32)
    y = blocks * torch.where(s == 0, torch.zeros_like(s), r / s)
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).reshape(*x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8).squeeze(-1)


def _fp4_parts(cache, dim):
    """The codes [pages, heads, page, D/2] and scales [pages, heads, page, D/16] inside a 4-bit cache."""
    pages, heads, page, _ = cache.shape
    flat = cache.view(pages, heads, -1)
    return (flat[:, :, :page * dim // 2].unflatten(2, (page, dim // 2)),
            flat[:, :, page * dim // 2:].unflatten(2, (page, dim // 16)))


def _from_fp4(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    return table[both] * _from_e4m3(scales).repeat_interleave(16, -1)


def _rows(cache, kind, page, offset, dim):
    """fp32 rows [..., heads, D] of the cache at (page, offset), without the heads' scales."""
    if kind == "same":
        return cache[page, :, offset].to(torch.float32)
    if kind == "fp8":
        return _from_e4m3(cache.view(torch.uint8)[page, :, offset])
    codes, scales = _fp4_parts(cache, dim)
    return _from_fp4(codes[page, :, offset], scales[page, :, offset])


def _norm(state):
    x, residual, weight = state["x"], state["residual"], state["weight"]
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + _EPS) * weight.float()
    more = () if residual is None else (h,)
    if not state["case"]["fp8"]:
        return (y.to(x.dtype),) + more
    scale = (y.abs().amax(-1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
    return (_to_e4m3(y, scale.reciprocal()), scale.squeeze(-1)) + more


def _rotate(x, state):
    case, half = state["case"], state["case"]["rotary"] // 2
    positions = state["positions"].to(torch.float64)
    if state["pair_axis"] is None:
        angle = positions[0][:, None] * state["inv_freq"].to(torch.float64)
    else:
        angle = positions[state["pair_axis"].long()].T * state["inv_freq"].to(torch.float64)
    c, s = torch.cos(angle).to(torch.float32)[:, None], torch.sin(angle).to(torch.float32)[:, None]
    f = x.to(torch.float32)
    if case["interleaved"]:
        a, b = f[..., 0:2 * half:2], f[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, f[..., 2 * half:]), -1).to(x.dtype)


def _store(x, cache, scale, slots, case):
    """Rows of x into the cache at their slots, and back."""
    pages, page, dim, kind = cache.shape[0], case["page"], case["head_dim"], case["cache"]
    there = slots >= 0
    row = torch.where(there, slots, pages * page - 1).long()   # a padded token's row goes where nothing is kept
    at, offset = row // page, row % page
    if kind == "same":
        cache[at, :, offset] = x
    elif kind == "fp8":
        cache.view(torch.uint8)[at, :, offset] = _to_e4m3(x.float(), scale.reciprocal()[:, None]).view(torch.uint8)
    else:
        codes, scales = _fp4_parts(cache, dim)
        codes[at, :, offset], scales[at, :, offset] = _to_fp4(x.float(), scale.reciprocal()[:, None])
    back = _rows(cache, kind, at, offset, dim)
    back = back if scale is None else back * scale[:, None]
    return torch.where(there[:, None, None], back, torch.zeros_like(back)).to(x.dtype)


def _attend(state):
    case, q = state["case"], state["q"]
    dim, page, group = case["head_dim"], case["page"], case["q_heads"] // case["kv_heads"]
    longest = case["length"]
    t = torch.arange(longest, device=q.device)
    at, offset = state["table"][:, t // page].long(), (t % page)[None].expand(case["batch"], -1)
    k = _rows(state["k_cache"], case["cache"], at, offset, dim).transpose(1, 2)
    v = _rows(state["v_cache"], case["cache"], at, offset, dim).transpose(1, 2)
    n = state["lengths"][:, None].long()
    seen = t[None] < n
    if case["window"]:
        seen = seen & (t[None] >= n - case["window"])
    seen = seen[:, None, None]
    f = q.float().unflatten(1, (case["kv_heads"], group)) * (1.0 / math.sqrt(dim))
    if state["k_scale"] is not None:
        f = f * state["k_scale"][:, None, None]
    s = torch.matmul(f, k.transpose(2, 3).contiguous()).masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(seen.squeeze(2)[..., None], v, torch.zeros_like(v)))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    if state["v_scale"] is not None:
        o = o * state["v_scale"][:, None, None]
    lse = (m + torch.log(total)).squeeze(-1).flatten(1)
    return o.flatten(1, 2).to(q.dtype), lse


# ---------------------------------------------------------------------- run --

def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _norm(state)
    if op == "rope":
        return _rotate(state["x"], state)
    if op == "append":
        case = state["case"]
        q, k = _rotate(state["q"], state), _rotate(state["k"], state)
        return (q, _store(k, state["k_cache"], state["k_scale"], state["slots"], case),
                _store(state["v"], state["v_cache"], state["v_scale"], state["slots"], case))
    return _attend(state)


def _run_own(state):
    import weight_only_fp4_amd as nv
    case = state["case"]
    if case["op"] == "norm":
        f = nv.rms_norm_fp8 if case["fp8"] else nv.rms_norm
        return f(state["x"], state["weight"], _EPS, residual=state["residual"])
    if case["op"] == "rope":
        return nv.rope(state["x"], state["positions"], state["inv_freq"], pair_axis=state["pair_axis"],
                       interleaved=case["interleaved"])
    if case["op"] == "append":
        q = nv.rope_kv_write(state["q"], state["k"], state["v"], state["positions"], state["inv_freq"],
                             state["k_cache"], state["v_cache"], state["slots"], k_scale=state["k_scale"],
                             v_scale=state["v_scale"], pair_axis=state["pair_axis"], interleaved=case["interleaved"])
        k, v = nv.kv_read(state["k_cache"], state["v_cache"], state["slots"], state["q"].dtype,
                          k_scale=state["k_scale"], v_scale=state["v_scale"])
        return q, k, v
    return nv.paged_attention(state["q"], state["k_cache"], state["v_cache"], state["table"], state["lengths"],
                              scale=1.0 / math.sqrt(case["head_dim"]), k_scale=state["k_scale"],
                              v_scale=state["v_scale"], window=case["window"], return_lse=True,
                              workspace_buf=state["workspace"])


def _row_bytes(kind, dim):
    return {"same": 2.0 * dim, "fp8": 1.0 * dim, "fp4": dim * 9 / 16}[kind]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        each = 2 + (1 if case["fp8"] else 2) + (4 if case["residual"] else 0)
        return {"bytes": n * each + 2.0 * case["cols"] + (4.0 * case["rows"] if case["fp8"] else 0), "flops": 5.0 * n}
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["head_dim"]
        return {"bytes": 4.0 * n + 4.0 * case["tokens"] * case["axes"] + 2.0 * case["rotary"], "flops": 3.0 * n}
    if case["op"] == "append":
        dim, kv = case["head_dim"], case["kv_heads"]
        n = case["tokens"] * dim
        # queries in and out; keys and values in, into the cache, out of it and back in 16 bits
        each = case["tokens"] * 2 * kv * (4.0 * dim + 2 * _row_bytes(case["cache"], dim))
        return {"bytes": 4.0 * n * case["q_heads"] + each + 4.0 * case["tokens"] * (case["axes"] + 1),
                "flops": 3.0 * n * (case["q_heads"] + kv)}
    seen = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
    dim, page = case["head_dim"], case["page"]
    return {"bytes": 2.0 * sum(seen) * case["kv_heads"] * _row_bytes(case["cache"], dim)
            + case["batch"] * case["q_heads"] * (4.0 * dim + 4) + 4.0 * sum(-(-n // page) for n in seen),
            "flops": 4.0 * sum(seen) * case["q_heads"] * dim}


# -------------------------------------------------------------------- exact --

def _small_float(x, mantissa, least, largest):
    """float64 values rounded to a small float (ties to even), saturated: `mantissa` stored bits, the least normal
    exponent, the largest value."""
    _, e = torch.frexp(x.abs())
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=least) - mantissa)
    return (torch.round(x / step) * step).clamp(-largest, largest)


def _exact_stored(x, g, kind):
    """What 16-bit rows x (float64) read back as; g: the heads' scales as float32 [heads]."""
    if kind == "same":
        return x
    inverse = (1.0 / g.double()).float()
    if kind == "fp8":
        return _small_float((x * inverse.double()[:, None]).float().double(), 3, -6, 448.0) * g.double()[:, None]
    t, h, d = x.shape
    b = x.view(t, h, d // 16, 16)
    r = inverse[None, :, None, None]
    top = (b.abs().amax(3, keepdim=True) * r.double()).float()
    s = _small_float((top.double() * float(np.float32(1.0 / 6.0))).float().double(), 3, -6, 448.0)
    by = torch.where(s > 0, (r.double() / s.clamp(min=2.0 ** -12)).float().double(), torch.zeros_like(s))
    return (_small_float((b * by).float().double(), 1, 0, 6.0) * s).view(t, h, d) * g.double()[:, None]


def _exact_rotated(x, state):
    case = state["case"]
    half = case["rotary"] // 2
    axis = state["pair_axis"].long() if case["axes"] > 1 else torch.zeros(half, dtype=torch.int64, device=x.device)
    angle = state["positions"].double()[axis, :].t() * state["inv_freq"].double()[None]
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.double().clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else \
        (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    state = prepare(case, seed)
    op, dtype = case["op"], _DTYPES[case["dtype"]]
    if op == "norm":
        x = state["x"].double()
        more = ()
        if case["residual"]:
            total = x + state["residual"].double()
            more, x = (total,), total.to(dtype).double()   # the norm is of the residual as it is kept
        y = state["weight"].double() * x / torch.sqrt((x * x).sum(1, keepdim=True) / case["cols"] + _EPS)
        if case["fp8"]:
            s = y.abs().max(1).values / 448.0
            return (y / s[:, None], s) + more
        return (y,) + more
    if op == "rope":
        return _exact_rotated(state["x"], state)
    if op == "append":
        keep = (state["slots"] >= 0)[:, None, None].double()
        k = _exact_rotated(state["k"], state)
        if case["cache"] != "same":
            k = k.to(torch.float32).to(dtype).double()   # keys are rounded to 16 bits before they are quantised
        return (_exact_rotated(state["q"], state), _exact_stored(k, state["k_scale"], case["cache"]) * keep,
                _exact_stored(state["v"].double(), state["v_scale"], case["cache"]) * keep)
    dim, page, heads = case["head_dim"], case["page"], case["kv_heads"]
    out = torch.zeros(case["batch"], case["q_heads"], dim, dtype=torch.float64, device=_DEVICE)
    lse = torch.full((case["batch"], case["q_heads"]), -math.inf, dtype=torch.float64, device=_DEVICE)

    def tokens(cache, scale, b, first, last):
        own_pages = state["table"][b, : -(-last // page)].long()
        x = cache[own_pages]   # [pages, heads, page, row]
        if case["cache"] == "fp4":
            x = x.reshape(x.shape[0], heads, -1)
            values = torch.tensor(_E2M1, dtype=torch.float64, device=_DEVICE)
            byte = x[:, :, :page * dim // 2].reshape(-1, heads, page, dim // 2).long()
            pair = torch.stack((byte % 16, byte // 16), 4).reshape(-1, heads, page, dim)
            sign = 1.0 - 2.0 * (pair // 8).double()
            per = x[:, :, page * dim // 2:].reshape(-1, heads, page, dim // 16).long()
            e, f = (per // 8) % 16, (per % 8).double()
            per = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f * 2.0 ** -9)
            x = (sign * values[pair % 8]).view(-1, heads, page, dim // 16, 16) * per[..., None]
            x = x.reshape(-1, heads, page, dim)
        x = x.float().double() if case["cache"] == "fp8" else x.double()
        x = x.permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, first:last]
        return x if scale is None else x * scale.double()[:, None, None]

    for b, n in enumerate(_lengths(case)):
        if not n:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        k, v = tokens(state["k_cache"], state["k_scale"], b, first, n), tokens(state["v_cache"], state["v_scale"], b, first, n)
        q = state["q"][b].double().view(heads, -1, dim)
        s = (q @ k.mT.contiguous()) / math.sqrt(dim)
        out[b] = (torch.softmax(s, 2) @ v).view(-1, dim)
        lse[b] = torch.logsumexp(s, 2).view(-1)
    return out, lse
