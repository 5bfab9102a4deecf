"""Plain forms of what a decode step runs around its layers, in 64 bits or whole numbers, for the tests to compare with.
They share no code with the library."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def plan(cached, new, table, free, head, page, tokens):
    """One request after another: (slots, positions, requests, lengths, offsets, head, table)."""
    B, width = len(cached), table.shape[1]
    table = table.copy()
    slots, positions, requests = np.full(tokens, -1), np.zeros(tokens, np.int64), np.full(tokens, -1)
    lengths, offsets = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    at, head = 0, max(0, int(head))
    next_page = head   # counts the pages of refused requests too, once the list has ended
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        begin, at = at, at + max(0, n)
        offsets[b + 1] = min(at, tokens)
        lengths[b] = max(0, c)
        if c < 0 or n < 0 or -(-(c + n) // page) > width or at > tokens:
            continue
        held, want = -(-c // page), -(-(c + n) // page)
        first, next_page = next_page, next_page + want - held
        if want > held and next_page > len(free):
            continue
        lengths[b] = c + n
        head += want - held
        table[b, held:want] = free[first:first + want - held]
        for i in range(n):
            pos = c + i
            number = int(table[b, pos // page])
            if 0 <= number < 2 ** 31 // page:
                slots[begin + i] = number * page + pos % page
            positions[begin + i], requests[begin + i] = pos, b
    return slots, positions, requests, lengths, offsets, np.array([head]), table


def lora(y, x, a, b, adapter, scale):
    """(out, bound): 64-bit values and how far off 16-bit outputs may be.  u: half a step of the type; h = x A^T has
    16 bits in bf16 (two parts of 8) and 22 of its row's largest in fp16, a K-term fp32 sum is off by K 2^-24 of its terms'
    absolute sum, an R-term one by R 2^-24 (twice each for the split and the waves' order)."""
    bf = y.dtype == torch.bfloat16
    y, x, a, b = (t.double().cpu() for t in (y, x, a, b))
    out, slack = y.clone(), torch.zeros_like(y)
    for t, i in enumerate(adapter.tolist()):
        if not 0 <= i < a.shape[0]:
            continue
        s = 1.0 if scale is None else float(scale[i])
        h, habs = a[i] @ x[t], a[i].abs() @ x[t].abs()
        out[t] = y[t] + s * (b[i] @ h)
        kept = h.abs() * 2.0 ** -16 if bf else torch.full_like(h, float(h.abs().max()) * 2.0 ** -21)
        off = kept + habs * (2 * x.shape[1] * 2.0 ** -24)
        slack[t] = abs(s) * (b[i].abs() @ (off + h.abs() * (4 * a.shape[1] * 2.0 ** -24)))
    u = 2.0 ** -8 if bf else 2.0 ** -11
    return out, u * (out.abs() + slack) + slack + y.abs() * 2.0 ** -23 + (0 if bf else 2.0 ** -25)


def weights(codes, scales, mx):
    """float64 [rows, cols] of packed E2M1 codes and their E4M3 (or E8M0) scale bytes."""
    codes, s = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64)
    code = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    value = E2M1[code & 7] * np.where(code >> 3, -1.0, 1.0)
    if mx:
        s = 2.0 ** (s - 127.0)
    else:
        e, m, sign = (s >> 3) & 15, s & 7, np.where(s >> 7, -1.0, 1.0)
        s = sign * np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    return value * np.repeat(s, 32 if mx else 16, axis=1)


def moe(x, ids, topk_weights, w1, w2, g1, g2, inter, gated=True, mx=False, pre1=None, pre2=None):
    """(out, bound) as float64 numpy; w1, w2 (codes, scales) per expert.  Roundings: X' (if scaled) and the output, half a
    step each; a to two parts of its type (half a step of half a step; in fp16 not below half its least step); sums in
    fp32, n 2^-24 of the terms' absolute sum each (twice n in the second, for the two parts)."""
    dt = x.dtype
    u = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -11
    tiny = 0.0 if dt == torch.bfloat16 else 2.0 ** -25
    T, H = x.shape
    xs = x if pre1 is None else (x.float() * pre1.float()).to(dt)
    xs = xs.double().cpu().numpy()
    p2 = np.ones(inter) if pre2 is None else pre2.double().cpu().numpy()
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    E, cache = w1[0].shape[0], {}
    for t in range(T):
        for e, w in zip(ids[t].tolist(), topk_weights[t].tolist()):
            if not 0 <= e < E:
                continue
            if e not in cache:
                cache[e] = weights(w1[0][e], w1[1][e], mx), weights(w2[0][e], w2[1][e], mx)
            m1, m2 = cache[e]
            s1, s2 = (1.0, 1.0) if mx else (float(g1[e]), float(g2[e]))
            h = s1 * (m1 @ xs[t])
            dh = abs(s1) * (np.abs(m1) @ np.abs(xs[t])) * (H * 2.0 ** -24) + np.abs(h) * 2.0 ** -23
            if gated:
                gate, up = h[:inter], h[inter:]
                sig = 1 / (1 + np.exp(-gate))
                a = gate * sig * up
                slope = np.abs(sig * (1 + gate * (1 - sig)))
                da = (slope + 0.25 * dh[:inter]) * dh[:inter] * (np.abs(up) + dh[inter:]) + np.abs(gate * sig) * dh[inter:] \
                    + np.abs(a) * 2.0 ** -21
            else:
                a = np.maximum(h, 0) ** 2
                da = (2 * np.maximum(h, 0) + dh) * dh + a * 2.0 ** -22
            ap, dap = a * p2, da * np.abs(p2) + np.abs(a * p2) * 2.0 ** -24
            dap = dap + u * u * (np.abs(ap) + dap) + tiny
            y = m2 @ ap
            dy = np.abs(m2) @ (dap + (2 * inter + 64) * 2.0 ** -24 * np.abs(ap))
            out[t] += w * s2 * y
            slack[t] += abs(w * s2) * (dy + np.abs(y) * 2.0 ** -21)
    return out, slack + u * (np.abs(out) + slack) + tiny


def sample_row(l, u, t=1.0, k=0, p=1.0, min_p=0.0):
    """(token, logprob) of one row, l float64 [V]."""
    l = np.where(np.isnan(l), -np.inf, l) + 0.0
    order = np.lexsort((np.arange(l.size), -l))
    top = l[order[0]]
    if top == -np.inf:
        return -1, -np.inf
    if not t > 0:
        return int(order[0]), 0.0
    if k > 0:
        order = order[:k]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(l[order] == top, 1.0, np.where(np.isneginf(l[order]) | np.isposinf(top), 0.0,
                                                    np.exp((l[order] - top) / t)))
    if p < 1:
        c = np.cumsum(w)
        n = 1 + int(np.sum(c[:-1] < p * c[-1]))
        order, w = order[:n], w[:n]
    keep = (w >= min_p) | (w == 1.0) if min_p == min_p else np.ones(w.size, bool)
    order, w = order[keep], w[keep]
    by = np.argsort(order)
    c = np.cumsum(w[by])
    x = u if u > 0 else 0.0
    j = int(np.sum(c <= x * c[-1]))
    j = min(j, int(np.nonzero(w[by] > 0)[0][-1]))
    return int(order[by[j]]), float(np.log(w[by[j]] / c[-1]))
