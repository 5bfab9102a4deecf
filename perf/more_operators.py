"""Cases of what a decode step runs around and between a layer's linears: page tables and slots from request lengths,
low-rank adapters beside a shared projection, a mixture-of-experts layer for a few tokens, and the choice of the next
token.

Every case names its operator in ``op``:

* ``plan``: page tables, slots and positions of a step's new tokens from the requests' lengths;
* ``lora``: low-rank adapters of several requests at once, added to a shared projection's output;
* ``moe``: a whole mixture-of-experts layer (two FP4 products, the gated activation between them, the weighted sum) for
  a few tokens;
* ``sample``: one token a row from its logits, with temperature, top-k, top-p and min-p, from given random numbers.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DEVICE = "cuda:0"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a small decoding batch: one new token a request
        {"name": "plan-16x1", "op": "plan", "requests": 16, "longest": 8192, "new": 1, "page": 16, "tokens": 16},
        # decoding requests and chunks of prompts in one step, the batch padded
        {"name": "plan-mixed-257", "op": "plan", "requests": 257, "longest": 16384, "new": 64, "page": 32,
         "tokens": 16384},
        # an offline run's prompts, a whole step of them
        {"name": "plan-prompts-131072", "op": "plan", "requests": 600, "longest": 0, "new": 250, "page": 16,
         "tokens": 131072},
        # a decoding batch in which everyone has an adapter of their own
        {"name": "lora-16x4096-r16", "op": "lora", "tokens": 16, "k": 4096, "n": 4096, "rank": 16, "adapters": 32,
         "run": 1, "none": 0.0, "dtype": "bf16"},
        # a larger decoding batch with a few popular adapters and requests without one, up projection
        {"name": "lora-133x4096-r64", "op": "lora", "tokens": 133, "k": 4096, "n": 14336, "rank": 64, "adapters": 12,
         "run": 1, "none": 0.25, "dtype": "fp16"},
        # prompts of several requests: their tokens come in runs
        {"name": "lora-prompts-4099-r32", "op": "lora", "tokens": 4099, "k": 5120, "n": 5120, "rank": 32, "adapters": 6,
         "run": 700, "none": 0.1, "dtype": "bf16"},
        # one user decoding, many narrow experts
        {"name": "moe-1-e128", "op": "moe", "tokens": 1, "experts": 128, "topk": 8, "hidden": 2048, "inter": 768,
         "mx": False, "dtype": "bf16"},
        # a small decoding batch, many narrow experts, the other weight format
        {"name": "moe-16-e128-mx", "op": "moe", "tokens": 16, "experts": 128, "topk": 8, "hidden": 2048, "inter": 768,
         "mx": True, "dtype": "fp16"},
        # a few users, few wide experts
        {"name": "moe-5-e8-wide", "op": "moe", "tokens": 5, "experts": 8, "topk": 2, "hidden": 4096, "inter": 14336,
         "mx": False, "dtype": "bf16"},
        # one user, the whole vocabulary, settings of a chat
        {"name": "sample-1x131072", "op": "sample", "rows": 1, "vocab": 131072, "k": 50, "p": 0.9, "min_p": 0.0,
         "masked": 0.0, "dtype": "bf16"},
        # a batch whose rows mask what a grammar forbids; rows have settings of their own, some are greedy
        {"name": "sample-23x32003-min-p", "op": "sample", "rows": 23, "vocab": 32003, "k": 0, "p": 1.0, "min_p": 0.05,
         "masked": 0.5, "dtype": "fp32"},
        # a full serving batch, nucleus over the whole vocabulary
        {"name": "sample-64x131072-top-p", "op": "sample", "rows": 64, "vocab": 131072, "k": 0, "p": 0.95, "min_p": 0.0,
         "masked": 0.0, "dtype": "bf16"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("plan", "lora", "moe", "sample"))
    if op == "plan":
        requests = _log_int(rng, 1, 4096)
        new = rng.choice((1, 1, _log_int(rng, 1, max(1, 131072 // requests))))
        tokens = min(131072, requests * new + rng.choice((0, 7, 64)))
        return {"op": op, "requests": requests, "longest": rng.choice((0, _log_int(rng, 1, 16384))), "new": new,
                "page": rng.choice((1, 16, 32, 48, 64, 128)), "tokens": tokens}
    if op == "lora":
        k, n = (rng.choice((1024, 2048, 4096, 5120, 8 * rng.randrange(64, 640))) for _ in range(2))
        rank = rng.choice((8, 16, 32, 64, 128))
        tokens = _log_int(rng, 1, max(1, 4096 * 10240 // (k + n) * 32 // max(32, rank)))
        return {"op": op, "tokens": tokens, "k": k, "n": rng.choice((n, n + rng.randrange(16))), "rank": rank,
                "adapters": _log_int(rng, 1, 64), "run": 1 if tokens < 256 else rng.choice((50, 700)),
                "none": rng.choice((0.0, 0.2)), "dtype": rng.choice(("bf16", "fp16"))}
    if op == "moe":
        experts, topk = rng.choice(((4, 1), (8, 2), (16, 4), (32, 4), (60, 4), (64, 6), (128, 8)))
        hidden = rng.choice((512, 1056, 2048, 2880, 4096))
        inter = rng.choice((128, 352, 768, 1408, 2048))
        return {"op": op, "tokens": _log_int(rng, 1, 64), "experts": experts, "topk": topk, "hidden": hidden,
                "inter": inter, "mx": rng.random() < 0.4, "dtype": rng.choice(("bf16", "fp16"))}
    vocab = rng.choice((131072, 128000, _log_int(rng, 50, 131072)))
    return {"op": op, "rows": _log_int(rng, 1, 64), "vocab": vocab, "k": rng.choice((0, 1, 20, 50, 1000)),
            "p": rng.choice((1.0, 0.5, 0.9, 0.99)), "min_p": rng.choice((0.0, 0.0, 0.02, 0.1)),
            "masked": rng.choice((0.0, 0.0, 0.7)), "dtype": rng.choice(("bf16", "fp16", "fp32"))}


# ------------------------------------------------------------------ inputs --

def _normal(shape, gen, dtype=torch.float32, sigma=1.0):
    return (torch.randn(shape, generator=gen, device=_DEVICE) * sigma).to(dtype)


def _uniform(shape, gen):
    return torch.rand(shape, generator=gen, device=_DEVICE)


def _whole(low, high, shape, gen, dtype=torch.int32):
    return torch.randint(low, high, shape, generator=gen, device=_DEVICE, dtype=dtype)


def _prepare_plan(case, gen):
    b, page = case["requests"], case["page"]
    cached = (_uniform(b, gen) ** 2 * case["longest"]).to(torch.int32)
    new = torch.ones(b, dtype=torch.int32, device=_DEVICE)
    if case["new"] > 1:
        # some requests decode, the others bring a part of a prompt, whose mean makes the step's size
        some = (_uniform(b, gen) * 2 * case["new"]).to(torch.int32)
        new = torch.where(_uniform(b, gen) < 0.2, new, some)
    over = (torch.cumsum(new, 0) > case["tokens"])
    new = torch.where(over, 0, new).to(torch.int32)   # what does not fit the step waits for the next
    width = -(-(case["longest"] + 2 * case["new"] + 1) // page)
    held = (cached + page - 1) // page
    pages = int(held.sum())
    need = int(((cached + new + page - 1) // page - held).sum())
    order = torch.randperm(pages + need + 8, generator=gen, device=_DEVICE).to(torch.int32)
    at = torch.arange(width, device=_DEVICE)
    first = torch.cumsum(held, 0) - held
    inside = at[None] < held[:, None]
    table = torch.where(inside, order[torch.where(inside, first[:, None] + at, 0)], 0).to(torch.int32).contiguous()
    return {"cached": cached, "new": new, "table": table, "free": order[pages:].contiguous(),
            "head": torch.full((1,), int(_whole(0, 8, (1,), gen)), dtype=torch.int32, device=_DEVICE)}


def _prepare_lora(case, gen):
    t, k, n, r, adapters = (case[x] for x in ("tokens", "k", "n", "rank", "adapters"))
    dtype = _DTYPES[case["dtype"]]
    runs = -(-t // case["run"])
    of_run = _whole(0, adapters, (runs,), gen)
    if case["run"] == 1 and adapters >= t:
        of_run = torch.randperm(adapters, generator=gen, device=_DEVICE)[:t].to(torch.int32)
    of_run = torch.where(_uniform(runs, gen) < case["none"], -1, of_run)
    return {"x": _normal((t, k), gen, dtype), "y": _normal((t, n), gen, dtype),
            "a": _normal((adapters, r, k), gen, dtype, 1.0 / math.sqrt(k)),
            "b": _normal((adapters, n, r), gen, dtype, 1.0 / math.sqrt(r)),
            "adapter": of_run.repeat_interleave(case["run"])[:t].to(torch.int32).contiguous(),
            "scale": 0.25 + 0.5 * _uniform(adapters, gen), "out": torch.empty((t, n), dtype=dtype, device=_DEVICE)}


def _in_turn(rows, inter):
    """Units of 16 gate rows and 16 up rows in turn, of rows [experts, 2 * inter, n]."""
    return rows.view(rows.shape[0], 2, inter // 16, 16, -1).transpose(1, 2).reshape(rows.shape)


def _laid_out(codes, scales):
    """Packed codes [e, n, k / 2] and scale bytes in the kernels' layout: blocks of 16 rows by 128 columns, in which
    each of 64 lanes has 32 columns of a row; the codes of all blocks, then their scales, two bytes a lane."""
    parts = []
    if scales.shape[2] * 8 != codes.shape[2]:   # one scale for 32 columns: the same byte twice
        scales = scales.repeat_interleave(2, 2)
    for x, each in ((codes, 16), (scales, 2)):
        e, n, k = x.shape
        x = torch.nn.functional.pad(x, (0, -k % (4 * each), 0, -n % 16))
        x = x.view(e, x.shape[1] // 16, 16, x.shape[2] // (4 * each), 4, each)
        parts.append(x.permute(0, 1, 3, 4, 2, 5).reshape(-1))
    return torch.cat(parts)


def _prepare_moe(case, gen):
    t, e, k, h, i = (case[x] for x in ("tokens", "experts", "topk", "hidden", "inter"))
    group = 32 if case["mx"] else 16
    state = {"x": _normal((t, h), gen, _DTYPES[case["dtype"]])}
    # tokens choose their experts by a skewed preference, as trained routers do
    logits = _normal((t, e), gen) + _normal((e,), gen, sigma=0.7)
    top, ids = torch.topk(torch.softmax(logits, 1), k, dim=1)
    state["ids"] = ids.to(torch.int32).contiguous()
    state["weights"] = (top / top.sum(1, keepdim=True)).contiguous()
    for name, rows, cols in (("1", 2 * i, h), ("2", h, i)):
        state["c" + name] = _whole(0, 256, (e, rows, cols // 2), gen, torch.uint8)
        low, high = (122, 126) if case["mx"] else (0x30, 0x40)
        state["s" + name] = _whole(low, high, (e, rows, cols // group), gen, torch.uint8)
        # products of about unit size: codes have a root mean square of 2.9
        state["g" + name] = None if case["mx"] else (0.31 / math.sqrt(cols)) * (0.7 + 0.6 * _uniform(e, gen))
    if case["mx"]:   # no global scale: the groups' powers of two bring the products to that size
        for name, cols in (("1", h), ("2", i)):
            state["s" + name] -= int(round(math.log2(math.sqrt(cols)))) - 1
    # the same weights as a program keeps them: laid out once, the first product's gate and up rows in turn
    state["w1"] = _laid_out(*(_in_turn(state[n], i) for n in ("c1", "s1")))
    state["w2"] = _laid_out(state["c2"], state["s2"])
    return state


def _prepare_sample(case, gen):
    b, v = case["rows"], case["vocab"]
    logits = _normal((b, v), gen, sigma=2.5)
    peaks = _whole(0, v, (b, 12), gen, torch.int64)
    logits.scatter_add_(1, peaks, 4.0 + 5.0 * _uniform((b, 12), gen))
    if case["masked"]:
        logits = logits.masked_fill(_uniform((b, v), gen) < case["masked"], -math.inf)
    state = {"logits": logits.to(_DTYPES[case["dtype"]]), "u": _uniform(b, gen)}
    temperature = 0.6 + 0.8 * _uniform(b, gen)
    state["temperature"] = torch.where(_uniform(b, gen) < 0.1, 0.0, temperature) if b > 8 else temperature
    state["k"] = torch.full((b,), case["k"], dtype=torch.int32, device=_DEVICE) if case["k"] else None
    state["p"] = torch.full((b,), case["p"], device=_DEVICE) if case["p"] < 1 else None
    state["min_p"] = torch.full((b,), case["min_p"], device=_DEVICE) if case["min_p"] else None
    return state


def prepare(case, seed):
    gen = torch.Generator(device=_DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    makers = {"plan": _prepare_plan, "lora": _prepare_lora, "moe": _prepare_moe, "sample": _prepare_sample}
    state = makers[op](case, gen)
    state["case"] = case
    state["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=_DEVICE)
    return state


# -------------------------------------------------------------- plain forms --

def _plan(state):
    page, tokens = state["case"]["page"], state["case"]["tokens"]
    cached, new, table, free = (state[x] for x in ("cached", "new", "table", "free"))
    cached, new, head = cached.long(), new.long(), state["head"].long()
    width, total = table.shape[1], cached + new
    ends = torch.cumsum(new.clamp(min=0), 0)
    held, want = (cached + page - 1) // page, (total + page - 1) // page
    fits = (cached >= 0) & (new >= 0) & (want <= width) & (ends <= tokens)
    need = torch.where(fits, want - held, 0)
    upto = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (head + upto <= free.shape[0]))
    row = torch.arange(tokens, device=table.device)
    r = torch.searchsorted(ends, row, right=True).clamp(max=cached.shape[0] - 1)
    there = (row < ends[-1]) & granted[r]
    position = torch.where(there, cached[r] + row - (ends[r] - new[r]), 0)
    entry = position // page
    fresh = entry >= held[r]
    at = torch.where(there & fresh, head + upto[r] - need[r] + entry - held[r], 0)
    number = torch.where(fresh, free[at], table[r, torch.where(there & ~fresh, entry, 0)]).long()
    slots = torch.where(there, number * page + position % page, -1)
    # the entries of new pages; rows that begin none write what is there
    begins = there & (position % page == 0)
    i, j = torch.where(begins, r, 0), torch.where(begins, entry, 0)
    spare = torch.cat((table.flatten(), table.new_zeros(1)))
    spare[torch.where(begins, i * width + j, table.numel())] = number.to(torch.int32)
    table.copy_(spare[:-1].view_as(table))
    offsets = torch.cat((ends.new_zeros(1), ends)).clamp(max=tokens)
    lengths = torch.where(granted, total, cached.clamp(min=0))
    head = head + torch.where(granted, need, 0).sum()
    requests = torch.where(there, r, -1)
    return tuple(x.to(torch.int32) for x in (slots, position, requests, lengths, offsets, head)) + (table,)


def _lora(state):
    x, y, a, b, adapter = (state[n] for n in ("x", "y", "a", "b", "adapter"))
    adapters, r, k = a.shape
    mine = adapter.long()[:, None] == torch.arange(adapters, device=x.device)
    h = torch.matmul(x.float(), a.float().view(adapters * r, k).t()).view(-1, adapters, r)
    h = h * (mine * state["scale"])[..., None]
    delta = torch.matmul(h.flatten(1), b.float().transpose(1, 2).reshape(adapters * r, -1))
    return (y.float() + delta).to(y.dtype)


def _weights(codes, scales, mx):
    """fp32 [.., rows, cols] of packed codes and their groups' scales."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float32, device=codes.device)
    values = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    if mx:
        s = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    return (values.unflatten(-1, (s.shape[-1], -1)) * s[..., None]).flatten(-2)


def _moe(state):
    x, ids, inter, mx = state["x"].float(), state["ids"].long(), state["case"]["inter"], state["case"]["mx"]
    t, k = ids.shape
    pairs, e = ids.flatten(), state["case"]["experts"]
    few = pairs.numel() <= e   # the pairs' experts one by one, or all experts
    which = pairs if few else torch.arange(e, device=x.device)
    w = _weights(state["c1"][which], state["s1"][which], mx)
    if few:
        h = torch.matmul(w, x.repeat_interleave(k, 0)[..., None]).squeeze(-1)
    else:
        h = torch.matmul(x, w.transpose(1, 2).contiguous())[pairs, torch.arange(t * k, device=x.device) // k]
    if not mx:
        h = h * state["g1"][pairs][:, None]
    gate, up = h[:, :inter], h[:, inter:]
    a = gate / (1 + torch.exp(-gate)) * up
    del w
    w = _weights(state["c2"][which], state["s2"][which], mx)
    if few:
        y = torch.matmul(w, a[..., None]).squeeze(-1)
    else:
        mine = pairs[None] == which[:, None]
        y = torch.matmul(torch.where(mine[..., None], a, 0), w.transpose(1, 2).contiguous()).sum(0)
    if not mx:
        y = y * state["g2"][pairs][:, None]
    return (y.view(t, k, -1) * state["weights"][..., None]).sum(1).to(state["x"].dtype)


def _sample(state):
    x = state["logits"].double() + 0.0   # no negative zeros
    x = torch.where(torch.isnan(x), -math.inf, x)
    b, v = x.shape
    t = state["temperature"].double()[:, None]
    ordered, index = torch.sort(x, dim=1, descending=True, stable=True)
    top = ordered[:, :1]
    w = torch.exp((ordered - top) / torch.where(t > 0, t, 1.0))
    w = torch.where(ordered == top, 1.0, torch.where(ordered == -math.inf, 0.0, w))
    rank = torch.arange(v, device=x.device)[None]
    keep = torch.ones((b, v), dtype=torch.bool, device=x.device)
    if state["k"] is not None:
        k = state["k"][:, None]
        keep = (k <= 0) | (rank < k)
    if state["p"] is not None:
        p = state["p"].double()[:, None]
        mass = torch.where(keep, w, 0.0)
        before = torch.cumsum(mass, 1) - mass
        keep = keep & ((p >= 1) | (rank == 0) | (before < p * mass.sum(1, keepdim=True)))
    if state["min_p"] is not None:
        keep = keep & (w >= state["min_p"].double()[:, None])
    keep = keep & torch.where(t > 0, True, rank == 0)
    kept = torch.zeros_like(w).scatter_(1, index, torch.where(keep, w, 0.0))
    c = torch.cumsum(kept, 1)
    total = c[:, -1:]
    token = (c <= state["u"].double()[:, None] * total).sum(1, keepdim=True)
    last = torch.where(kept > 0, rank, -1).amax(1, keepdim=True)
    token = torch.minimum(token, last)
    logprob = torch.log(kept.gather(1, token.clamp(min=0)) / total)
    empty = top == -math.inf
    token, logprob = torch.where(empty, -1, token), torch.where(empty, -math.inf, logprob)
    return token.squeeze(1).to(torch.int32), logprob.squeeze(1).float()


# ---------------------------------------------------------------------- run --

def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan, "lora": _lora, "moe": _moe, "sample": _sample}[state["case"]["op"]](state)


def _run_own(state):
    import weight_only_fp4_amd as nv
    case = state["case"]
    if case["op"] == "plan":
        p = nv.kv_plan(state["cached"], state["new"], state["table"], state["free"], state["head"], case["page"],
                       case["tokens"])
        return p.slots, p.positions, p.requests, p.lengths, p.offsets, p.head, state["table"]
    if case["op"] == "lora":
        return nv.lora_add(state["y"], state["x"], state["a"], state["b"], state["adapter"], scale=state["scale"],
                           out=state["out"], workspace_buf=state["workspace"])
    if case["op"] == "moe":
        return nv.moe_layer(state["x"], state["ids"], state["weights"], state["w1"], state["w2"], case["experts"],
                            case["inter"], state["g1"], state["g2"], mxfp4=case["mx"], workspace_buf=state["workspace"])
    return nv.sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["k"], top_p=state["p"],
                     min_p=state["min_p"], return_logprobs=True, workspace_buf=state["workspace"])


def _active(case):
    """Experts that the tokens of a step choose, on average over an even choice."""
    e, k, t = case["experts"], case["topk"], case["tokens"]
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    if case["op"] == "plan":
        b, t = case["requests"], case["tokens"]
        pages = b * case["new"] / case["page"]
        return {"bytes": 12.0 * t + 16.0 * b + 8.0 * pages, "flops": 4.0 * t}
    if case["op"] == "lora":
        t, k, n, r = case["tokens"], case["k"], case["n"], case["rank"]
        mine = t * (1.0 - case["none"])
        runs = mine / case["run"]
        used = case["adapters"] * (1.0 - (1.0 - 1.0 / case["adapters"]) ** runs)
        if case["run"] == 1 and case["adapters"] >= t:
            used = mine
        return {"bytes": 2.0 * used * r * (k + n) + 2.0 * mine * k + 4.0 * t * n, "flops": 2.0 * mine * r * (k + n)}
    if case["op"] == "moe":
        h, i, p = case["hidden"], case["inter"], case["tokens"] * case["topk"]
        each = 0.53125 if case["mx"] else 0.5625
        return {"bytes": _active(case) * 3.0 * i * h * each + 4.0 * case["tokens"] * h + 8.0 * p,
                "flops": 6.0 * p * i * h}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4.0 if case["dtype"] == "fp32" else 2.0) + 28.0 * case["rows"], "flops": 4.0 * n}


# -------------------------------------------------------------------- exact --

def _exact_lora(state):
    y = state["y"].double()
    for a in range(state["case"]["adapters"]):
        at = (state["adapter"] == a).nonzero().flatten()
        h = state["x"][at].double() @ state["a"][a].double().t()
        y[at] += float(state["scale"][a]) * (h @ state["b"][a].double().t())
    return y


def _exact_weight(codes, scales, mx):
    byte = codes.long()
    code = torch.stack((byte % 16, byte // 16), 2).reshape(byte.shape[0], -1)
    value = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)[code % 8] * (1.0 - 2.0 * (code // 8))
    s = scales.long()
    if mx:
        s = torch.exp2((s - 127).double())
    else:
        e, f = (s // 8) % 16, (s % 8).double()
        s = torch.where(e > 0, (1 + f / 8) * torch.exp2((e - 7).double()), f * 2.0 ** -9)
    return value * s.repeat_interleave(32 if mx else 16, 1)


def _exact_moe(state):
    x, ids, inter = state["x"].double(), state["ids"], state["case"]["inter"]
    out = torch.zeros_like(x)
    for e in ids.unique().tolist():
        token, slot = (ids == e).nonzero(as_tuple=True)
        g1, g2 = (1.0, 1.0) if state["case"]["mx"] else (float(state["g1"][e]), float(state["g2"][e]))
        h = g1 * (x[token] @ _exact_weight(state["c1"][e], state["s1"][e], state["case"]["mx"]).t())
        a = torch.nn.functional.silu(h[:, :inter]) * h[:, inter:]
        y = g2 * (a @ _exact_weight(state["c2"][e], state["s2"][e], state["case"]["mx"]).t())
        out.index_add_(0, token, y * state["weights"][token, slot].double()[:, None])
    return out


def _exact_sample(state):
    rows = state["logits"].double().cpu().numpy()
    settings = ("u", "temperature", "k", "p", "min_p")
    host = {n: None if state[n] is None else state[n].double().cpu().numpy() for n in settings}
    tokens, logprobs = [], []
    for i, row in enumerate(rows):
        order = np.lexsort((np.arange(row.size), -row))
        if host["temperature"][i] <= 0:
            tokens.append(int(order[0]))
            logprobs.append(0.0)
            continue
        if host["k"] is not None and host["k"][i] > 0:
            order = order[:int(host["k"][i])]
        w = np.exp(((row[order] - row[order[0]]) / host["temperature"][i]).astype(np.longdouble))
        if host["p"] is not None and host["p"][i] < 1:
            upto = np.cumsum(w)
            n = 1 + int(np.sum(upto[:-1] < host["p"][i] * upto[-1]))
            order, w = order[:n], w[:n]
        if host["min_p"] is not None:
            n = int(np.sum(w >= host["min_p"][i]))
            order, w = order[:n], w[:n]
        by_index = np.argsort(order)
        share = np.cumsum(w[by_index]) / w.sum()
        j = by_index[min(int(np.sum(share <= host["u"][i])), share.size - 1)]
        tokens.append(int(order[j]))
        logprobs.append(float(np.log(w[j] / w.sum())))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=torch.float64)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "lora":
        return _exact_lora(state)
    if case["op"] == "moe":
        return _exact_moe(state)
    if case["op"] == "sample":
        return _exact_sample(state)
    return None   # whole numbers
