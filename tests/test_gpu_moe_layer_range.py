"""The expert layer of a few tokens where the activation between its products is far from one: what goes from the first
product to the second has the range of fp32 and 24 bits in both types, so that only the output is rounded."""
import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv
from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def check(layer, got, x, ids, w):
    """Against 64 bits.  A result is off by its sums' fp32 roundings (n terms: n 2^-24 of their absolute sum), the
    activation's (2^-20 of it, and what h's error makes of it) and half a step of the output's type: nothing else is
    rounded, whatever the size of a.  The root mean square of half steps is 1 / sqrt(3) of their largest."""
    T, H = x.shape
    out, slack = np.zeros((T, H)), np.zeros((T, H))
    xs, inter, cache = x.double().cpu().numpy(), layer.I, {}
    for t in range(T):
        for e, c in zip(ids[t].tolist(), w[t].tolist()):
            if e not in cache:
                cache[e] = [ref.weights(m[0][e], m[1][e], False) for m in (layer.w1, layer.w2)]
            m1, m2 = cache[e]
            g1, g2 = float(layer.g1[e]), float(layer.g2[e])
            h = g1 * (m1 @ xs[t])
            dh = abs(g1) * (np.abs(m1) @ np.abs(xs[t])) * (H * 2.0 ** -24) + np.abs(h) * 2.0 ** -23
            if layer.gated:
                gate, up = h[:inter], h[inter:]
                sig = 1 / (1 + np.exp(-np.maximum(gate, -700)))
                a = gate * sig * up
                slope = np.abs(sig * (1 + gate * (1 - sig)))   # of silu; its second derivative is at most 1/2
                da = (slope + 0.25 * dh[:inter]) * dh[:inter] * (np.abs(up) + dh[inter:]) + np.abs(gate * sig) * dh[inter:] \
                    + np.abs(a) * 2.0 ** -20
            else:
                a = np.maximum(h, 0) ** 2
                da = (2 * np.maximum(h, 0) + dh) * dh + a * 2.0 ** -22
            y = m2 @ a
            # a's own 24 bits, sums of I terms in two parts, and the waves' and workgroups' sums
            dy = np.abs(m2) @ (da + (2 * inter + 66) * 2.0 ** -24 * np.abs(a))
            out[t] += c * g2 * y
            slack[t] += abs(c * g2) * (dy + np.abs(y) * 2.0 ** -21)
    u, tiny = (2.0 ** -8, 0.0) if layer.dtype == BF else (2.0 ** -11, 2.0 ** -25)
    off = np.abs(got.double().cpu().numpy() - out)
    bound = slack + u * (np.abs(out) + slack) + tiny
    assert (off <= bound).all(), float((off / bound).max())
    assert np.linalg.norm(off) < 0.6 * u * np.linalg.norm(out)
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 2), (3, 2), (2, 3), (9, 2), (16, 1), (40, 3)])
@pytest.mark.parametrize("size", [2.0 ** -30, 5e-5, 4e-6, 200.0, 3e5, 2.0 ** 60])
def test_small_and_large_activations(size, T, k, gated, dtype):
    """a of root mean square about `size`, outputs of about one."""
    layer = Layer(4, 256, 192, dtype, gated, seed=int(T + 10 * k))
    x, ids, w = layer.tokens(T, k)
    layer.g1 *= size ** 0.5
    layer.g2 /= size
    out = check(layer, layer.run(x, ids, w), x, ids, w)
    assert 0.02 < np.sqrt(np.mean(out ** 2)) < 50


def test_rows_of_very_different_activations():
    """Experts whose activations lie up to 2^80 apart."""
    for dtype in (BF, FP):
        layer = Layer(6, 128, 320, dtype, False, seed=4)
        factor = torch.tensor([2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** -10, 2.0 ** 10, 1.0], device=DEV)
        layer.g1 *= factor
        layer.g2 /= factor ** 2
        x, ids, w = layer.tokens(12, 4)
        check(layer, layer.run(x, ids, w), x, ids, w)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (2, 1, 1), (3, 1, 1), (4, 1, 1), (5, 1, 1), (6, 2, 4)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_what_cancels_keeps_its_bits(T, k, E, dtype):
    """Pairs of columns of a that are made alike up to their pre-quant scales, and whose terms cancel but for one part in
    7028: with fewer than 24 bits of a next to nothing of the difference is right."""
    H, I = 64, 256
    layer = Layer(E, H, I, dtype, False, seed=9)
    c1, s1 = layer.w1
    first = torch.arange(I, device=DEV).view(-1, 2, 16)[:, 0].flatten()   # and its partner 16 further, in the next group
    c1[:, first + 16], s1[:, first + 16] = c1[:, first], s1[:, first]
    # 7029 and 7028 parts of 2048: 3/2 11/8 213/128 and 2/2 14/8 251/128
    c2, s2 = layer.w2
    c2[:] = 0
    s2[:, :, ::2], s2[:, :, 1::2] = 0x38 + 11 - 8, 0x38 + 14 - 8
    rows = torch.arange(H, device=DEV)
    col = first[rows]
    shift = (col % 2 * 4).to(torch.uint8)
    c2[:, rows, col // 2] = torch.full_like(shift, 3) << shift
    c2[:, rows, col // 2 + 8] = torch.full_like(shift, 8 | 2) << shift
    layer.pre2 = torch.where(torch.arange(I, device=DEV) % 32 < 16, 213 / 128, 251 / 128).to(dtype)
    layer.b1, layer.b2 = nv.repack(*layer.w1), nv.repack(*layer.w2)
    x, ids, w = layer.tokens(T, k)
    got = layer.run(x, ids, w).double().cpu().numpy()
    want, slack = np.zeros((T, H)), np.zeros((T, H))
    xs, at = x.double().cpu().numpy(), col.cpu().numpy()
    for t in range(T):
        for e, c in zip(ids[t].tolist(), w[t].tolist()):
            m1, g1 = ref.weights(c1[e], s1[e], False)[at], float(layer.g1[e])
            h = np.maximum(g1 * (m1 @ xs[t]), 0)
            dh = abs(g1) * (np.abs(m1) @ np.abs(xs[t])) * (H * 2.0 ** -24) + h * 2.0 ** -23
            scale = c * float(layer.g2[e])
            want[t] += scale * h ** 2 / 2048
            # a's error, the same in both columns, counts with the difference; each column rounds for itself in the product
            # with pre2, as it is split (2^-24 of it or, for a small one, 2^-38 of its 16 neighbours' largest) and where
            # its parts' products are added up: half a step of 2^-24 each
            most = np.maximum(g1 * (ref.weights(c1[e], s1[e], False) @ xs[t]), 0).max() ** 2
            slack[t] += abs(scale) * (((2 * h + dh) * dh + h ** 2 * 2.0 ** -21) / 2048
                                      + 7029 / 2048 * 2 * (3 * 2.0 ** -24 * h ** 2 + 2.0 ** -37 * most))
    u, tiny = (2.0 ** -8, 0.0) if dtype == BF else (2.0 ** -11, 2.0 ** -25)
    off = np.abs(got - want)
    bound = slack + u * (np.abs(want) + slack) + tiny
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinite_and_nan_activations(dtype):
    """Beyond fp32's range a is an infinity; a NaN stays in its token."""
    layer = Layer(2, 128, 64, dtype, True, seed=2)
    x, ids, w = layer.tokens(4, 1)
    ids[:] = 0
    layer.g1[0] = 2.0 ** 70
    assert not torch.isfinite(layer.run(x, ids, w)).any()
    layer.g1[0] = 2.0 ** 50
    layer.g2[0] = 2.0 ** -104
    x[2, 5] = float("nan")
    got = layer.run(x, ids, w)
    rows = torch.tensor([0, 1, 3], device=DEV)
    assert torch.isnan(got[2]).all() and torch.isfinite(got[rows]).all()
    check(layer, got[rows], x[rows], ids[rows], w[rows])


@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 16, 16), (3, 2, 4, 64, 16), (5, 1, 2, 48, 144), (9, 3, 4, 1040, 272),
                                       (64, 8, 9, 32, 112)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_that_end_inside_a_chunk(T, k, E, H, I, dtype):
    """What lies behind a row of a in the workspace counts for nothing: it was NaN, and is what other calls left."""
    layer = Layer(E, H, I, dtype, seed=T)
    x, ids, w = layer.tokens(T, k)
    ws = torch.full((nv.moe_layer_workspace_bytes(64, 8, E, H, 512),), 255, dtype=torch.uint8, device=DEV)
    ws[:4096] = 0
    want = layer.run(x, ids, w, workspace_buf=ws)
    check(layer, want, x, ids, w)
    big = Layer(E, H, 512, dtype, seed=1)
    bx, bids, bw = big.tokens(64, min(8, k + 1))
    bx[:] = float("inf")
    big.run(bx, bids, bw, workspace_buf=ws)
    assert torch.equal(layer.run(x, ids, w, workspace_buf=ws), want)
