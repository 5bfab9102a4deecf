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
