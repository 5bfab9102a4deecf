"""How many bits single-token attention keeps on its way: sums that cancel and weights far apart, against 64-bit plain
forms on the CPU.  The bounds count roundings as attention_ref.py does."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import weight_only_fp4_amd as nv
from test_gpu_attention import BF, DEV, HF, make_cache, say

pytestmark = pytest.mark.gpu


def attend(q, k, v, kind, dt, scale=1.0):
    """q [B, Hq, D], k, v [B, n, Hk, D] through a cache without head scales -> (out, lse, the keys and values the cache
    stands for), float64."""
    B, n, Hk, D = k.shape
    page = 16
    width = -(-n // page)
    kc, vc = make_cache(kind, dt, B * width, Hk, page, D)
    table = torch.arange(B * width, dtype=torch.int32).view(B, width)
    t = torch.arange(n)
    slots = (table[:, t // page] * page + t % page).reshape(-1).to(torch.int32)
    rows = [x.to(dt).reshape(B * n, Hk, D) for x in (k, v)]
    nv.kv_write(rows[0].to(DEV), rows[1].to(DEV), kc, vc, slots.to(DEV))
    out, lse = nv.paged_attention(q.to(dt).to(DEV), kc, vc, table.to(DEV), torch.full((B,), n, dtype=torch.int32, device=DEV),
                                  scale=scale, return_lse=True)
    held = [ref.value(*ref.stored(ref.f64(x), None, kind), None).reshape(B, n, Hk, D) for x in rows]
    return ref.f64(out), ref.f64(lse), *held


@pytest.mark.parametrize("kind,dt", [("same", BF), ("same", HF), ("fp8", BF), ("fp8", HF)])
def test_weights_keep_more_bits_than_the_type_of_the_products(kind, dt):
    """One token's value is cancelled by three whose values add up to its weight as the products' type would round it,
    so the result is what that rounding would lose.  A weight in two parts is off by u^2 of itself, by the exponential's
    and the subtraction's 2^-20 and by the score's four roundings; the sum of four tokens by eight fp32 roundings."""
    say(f"weights {kind} {dt}")
    D, heads = 64, torch.tensor([1.0, 0.75, 1.25, 1.5])
    products = HF if kind != "same" or dt == HF else BF
    keys = torch.arange(8, 16, dtype=torch.float64)[:, None] * 2.0 ** torch.arange(-7, -2)
    keys = -keys.flatten()                                     # 4 significant bits, -1/16 .. -15/8: exact in every cache
    B, G = len(keys), len(heads)
    q = torch.zeros((B * G, 1, D), dtype=torch.float64)
    k, v = (torch.zeros((B * G, 4, 1, D), dtype=torch.float64) for _ in range(2))
    q[:, 0, 0] = heads.double().repeat(B)
    k[:, 3, 0, 0] = keys.repeat_interleave(G)
    p = torch.exp(q[:, 0, 0] * k[:, 3, 0, 0])
    left = 64 * p.to(products).double()
    v[:, 3] = 64
    for i in range(3):   # in steps of four significant bits, towards zero
        step = 2.0 ** (torch.floor(torch.log2(left.clamp(min=2.0 ** -6))) - 3)
        part = torch.floor(left / step) * step
        v[:, i] = -part[:, None, None]
        left = left - part
    out, lse, kk, vv = attend(q, k, v, kind, dt)
    s = (q.numpy() * kk[:, :, 0]).sum(2)                       # [B G, 4]
    w = np.exp(s)
    total = w.sum(1, keepdims=True)
    want = (w[..., None] * vv[:, :, 0]).sum(1) / total
    size = (w[..., None] * np.abs(vv[:, :, 0])).sum(1) / total
    rel = ref.u(products) ** 2 + 2.0 ** -20 + 4 * ref.U32 * np.abs(s).max() + 8 * ref.U32
    off = size * rel
    assert np.median(np.abs(want) / size) > 4 * rel            # the rounding of the weights would show
    assert np.all(np.abs(out[:, 0] - want) <= off + (np.abs(want) + off) * ref.u(dt) + ref.least(dt))
    assert np.all(np.abs(lse[:, 0] - np.log(total[:, 0])) <= 2.0 ** -20)


@pytest.mark.parametrize("kind,dt", [("same", BF), ("same", HF), ("fp8", BF), ("fp8", HF), ("fp4", BF), ("fp4", HF)])
def test_many_small_weights_add_up(kind, dt):
    """One token of 32 is far above the others, which each weigh e^-18 of it (below fp16's least value), and the others'
    values make the result.  A weight is off by the exponential's 2^-20 of itself, the score's four roundings and its
    own, and with products in fp16 by half its least value on a scale of 2^7."""
    say(f"small weights {kind} {dt}")
    D, n = 64, 4096
    q = torch.zeros((1, 1, D), dtype=torch.float64)
    k, v = torch.zeros((1, n, 1, D), dtype=torch.float64), torch.full((1, n, 1, D), 6.0, dtype=torch.float64)
    q[..., 0] = 1
    k[..., 0] = -18
    k[:, ::32], v[:, ::32] = 0, 0
    out, lse, kk, vv = attend(q, k, v, kind, dt)
    assert np.all(kk[0, 1:32, 0, 0] == -18) and np.all(vv[0, 1:32] == 6)
    w = 31 * np.exp(-18.0)
    want = 6 * w / (1 + w)
    u = 2.0 ** -8 if kind == "same" and dt == BF else 2.0 ** -11
    off = want * (u + 2.0 ** -20 + 4 * 18 * ref.U32 + 2 * (n + 64) * ref.U32) + 6 * 31 * 2.0 ** -32
    assert np.all(np.abs(out - want) <= off + (want + off) * ref.u(dt) + ref.least(dt))
    assert np.all(np.abs(lse - np.log(n // 32) - np.log1p(w)) <= 2 * (n + 64) * ref.U32 + 2.0 ** -20)


@pytest.mark.parametrize("kind,dt", [("same", BF), ("same", HF), ("fp8", BF), ("fp8", HF), ("fp4", BF), ("fp4", HF)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_every_size(kind, dt, sign):
    """Four equal scores from 2^-6 to 2^60, whose last place passes everything the running maximum is kept apart by, and
    a fifth below them by a quarter: the mean of four, or of five where the fifth is near."""
    D, n = 64, 5
    size = 2.0 ** torch.arange(-6, 61)[:, None]
    k, v = torch.zeros((1, n, 1, D), dtype=torch.float64), torch.zeros((1, n, 1, D), dtype=torch.float64)
    k[..., 0] = sign * 4.0
    k[:, 4, :, 0] = 3.0 if sign > 0 else -6.0
    v[:] = torch.tensor([1.0, 2.0, 3.0, 6.0, 1.5]).double()[None, :, None, None]
    q = torch.zeros((1, 1, D), dtype=torch.float64)
    q[..., 0] = 1
    for scale in size.flatten().tolist():
        say(f"scale {scale} {kind} {dt}")
        out, lse, kk, vv = attend(q, k, v, kind, dt, scale=scale)
        s = scale * kk[0, :, 0, 0]
        w = np.exp(s - s.max())
        want = (w[:, None] * vv[0, :, 0]).sum(0) / w.sum()
        # the fifth score is off by four roundings of itself, which is what its weight is off by
        rel = 2.0 ** -8 + min(1.0, np.expm1(min(8 * ref.U32 * np.abs(s).max(), 1.0))) * w[4] * 2
        assert np.all(np.abs(out[0, 0] - want) <= np.abs(want) * (rel + 2 * ref.u(dt)) + ref.least(dt))
        assert np.all(np.abs(lse - (s.max() + np.log(w.sum()))) <= 8 * ref.U32 * np.abs(s).max() + 2.0 ** -20)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("dt,far,size", [(BF, 2.0 ** 26, 1.0), (HF, 2.0 ** 15, 2.0 ** -8)])
def test_columns_far_below_the_largest_of_a_query_count(kind, dt, far, size):
    """Queries whose largest column meets keys of zero: the scores are made of columns 2^-23 to 2^-26 of it.  With a
    quantised cache a column is held as fp16 on a scale where the largest is 2^14 or more, so it is off by 2^-39 of
    that; the rest as in attention_ref.attention."""
    say(f"far columns {kind} {dt}")
    g = torch.Generator()
    g.manual_seed(7)
    D, n, G = 128, 200, 3
    q, k, v = (torch.randn(s, generator=g).to(dt).double() for s in ((1, G, D), (1, n, 1, D), (1, n, 1, D)))
    q = (q * size).to(dt).double()
    q[..., 5] = far
    k[..., 5] = 0
    scale = 0.125 / size
    out, lse, kk, vv = attend(q, k, v, kind, dt, scale=scale)
    q, kk, vv = q[0].numpy(), kk[0, :, 0], vv[0, :, 0]
    want, want_lse, _, _ = ref.attention(q, kk, vv, scale, (HF, dt))
    s = q @ kk.T * scale
    ds = (np.abs(q) @ np.abs(kk).T * scale * (D + 6) * ref.U32 + np.abs(s) * 2 * ref.U32
          + 2.0 ** -39 * far * np.abs(kk).sum(1)[None] * scale).max(1, keepdims=True)
    w = np.exp(s - s.max(1, keepdims=True))
    each = w @ np.abs(vv) / w.sum(1, keepdims=True)
    off = each * (ref.u(HF) + np.expm1(4 * ds) + 2.0 ** -20 + 2 * (n + 64) * ref.U32) + 2.0 ** -32 * np.abs(vv).sum(0)
    assert np.all(off < 0.02 * np.abs(vv).max())
    assert np.all(np.abs(out[0] - want) <= off + (np.abs(want) + off) * ref.u(dt) + ref.least(dt))
    assert np.all(np.abs(lse[0] - want_lse) <= 2 * ds[:, 0] + (n + 64) * ref.U32 + 2.0 ** -20)
