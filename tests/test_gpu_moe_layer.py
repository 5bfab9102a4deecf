"""The expert layer of a few tokens in one call, against 64-bit sums and the framework's separate calls."""
import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


class Layer:
    def __init__(self, E, H, I, dtype, gated=True, mx=False, seed=0, pre=False):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.gen, self.E, self.H, self.I, self.gated, self.mx, self.dtype = g, E, H, I, gated, mx, dtype
        F, group = (2 if gated else 1) * I, 32 if mx else 16
        byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV, dtype=torch.uint8)  # noqa: E731
        low, high = (118, 122) if mx else (0x30, 0x40)
        self.w1 = byte(0, 256, E, F, H // 2), byte(low, high, E, F, H // group)
        self.w2 = byte(0, 256, E, H, I // 2), byte(low, high, E, H, I // group)
        if mx:
            self.b1 = nv.repack_gated(*self.w1, mxfp4=True) if gated else nv.repack_mxfp4(*self.w1)
            self.b2 = nv.repack_mxfp4(*self.w2)
            self.g1 = self.g2 = None
        else:
            self.b1 = nv.repack_gated(*self.w1) if gated else nv.repack(*self.w1)
            self.b2 = nv.repack(*self.w2)
            self.g1 = 0.3 / H ** 0.5 * (0.5 + torch.rand(E, generator=g, device=DEV))
            self.g2 = 0.3 / I ** 0.5 * (0.5 + torch.rand(E, generator=g, device=DEV))
        self.pre1 = (0.5 + torch.rand(H, generator=g, device=DEV)).to(dtype) if pre else None
        self.pre2 = (0.5 + torch.rand(I, generator=g, device=DEV)).to(dtype) if pre else None

    def tokens(self, T, k, repeat=False):
        x = torch.randn((T, self.H), generator=self.gen, device=DEV).to(self.dtype)
        if repeat or k > self.E:
            ids = torch.randint(0, self.E, (T, k), generator=self.gen, device=DEV)
        else:
            ids = torch.rand((T, self.E), generator=self.gen, device=DEV).argsort(1)[:, :k]
        w = torch.rand((T, k), generator=self.gen, device=DEV)
        return x, ids.to(torch.int32).contiguous(), w / k

    def run(self, x, ids, w, **kw):
        return nv.moe_layer(x, ids, w, self.b1, self.b2, self.E, self.I, self.g1, self.g2, mxfp4=self.mx,
                            activation=nv.MOE_SILU_GLU if self.gated else nv.MOE_RELU2, pre_scale1=self.pre1,
                            pre_scale2=self.pre2, **kw)

    def check(self, got, x, ids, w):
        want, bound = ref.moe(x, ids, w, self.w1, self.w2, self.g1, self.g2, self.I, self.gated, self.mx, self.pre1, self.pre2)
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= bound).all(), (off / bound).max()
        # the output's rounding: uniform errors of at most half a step, whose root mean square is its 1 / sqrt(3)
        u = 2.0 ** -8 if self.dtype == BF else 2.0 ** -11
        n = np.linalg.norm(want)
        assert want.size < 2000 or n == 0 or np.linalg.norm(off) / n < u * 0.6


@pytest.mark.parametrize("T,k,E,H,I,dtype", [
    (1, 1, 1, 32, 32, BF), (1, 8, 128, 256, 128, BF), (2, 2, 8, 512, 96, FP), (5, 2, 8, 1056, 352, BF),
    (16, 8, 128, 256, 160, FP), (16, 8, 16, 512, 256, BF), (33, 4, 8, 288, 128, BF), (64, 8, 32, 256, 64, FP),
    (64, 1, 1, 128, 256, BF), (3, 6, 60, 2048, 1408, BF), (64, 2, 4, 160, 2048, FP), (7, 70, 128, 64, 64, BF),
    (1, 512, 600, 64, 32, BF), (4, 4, 4, 18432, 64, BF),
])
@pytest.mark.parametrize("gated,mx", [(True, False), (True, True), (False, False)])
def test_moe_layer(T, k, E, H, I, dtype, gated, mx):
    layer = Layer(E, H, I, dtype, gated, mx, seed=T + E)
    args = layer.tokens(T, k)
    layer.check(layer.run(*args), *args)


@pytest.mark.parametrize("dtype,gated,mx", [(BF, True, False), (FP, True, True), (FP, False, False), (BF, False, True)])
@pytest.mark.parametrize("T", [1, 9, 40])
def test_pre_scales(T, dtype, gated, mx):
    layer = Layer(8, 320, 96, dtype, gated, mx, seed=T, pre=True)
    args = layer.tokens(T, 3)
    layer.check(layer.run(*args), *args)


@pytest.mark.parametrize("T,k,E", [(5, 4, 8), (64, 8, 6), (30, 2, 2)])
def test_ids_outside_and_twice(T, k, E):
    layer = Layer(E, 256, 128, BF, seed=3)
    x, ids, w = layer.tokens(T, k, repeat=True)
    ids[0] = -1            # a token without an expert
    ids[1:, 0][::3] = E    # pairs of no expert
    ids[-1] = ids[-1, 0].clamp(0, E - 1)
    got = layer.run(x, ids, w)
    layer.check(got, x, ids, w)
    assert (got[0] == 0).all()
    ids[:] = E + 5
    assert (layer.run(x, ids, w) == 0).all()


def test_weights_and_divisors():
    layer = Layer(8, 256, 128, BF, seed=4)
    x, ids, w = layer.tokens(6, 4)
    w[0], w[1, 2], w[2] = 0, -0.5, 3
    layer.check(layer.run(x, ids, w), x, ids, w)
    inv = [1 / g for g in (layer.g1, layer.g2)]
    got = nv.moe_layer(x, ids, w, layer.b1, layer.b2, 8, 128, *inv, divisor=True)
    layer.g1, layer.g2 = (1 / g for g in inv)
    layer.check(got, x, ids, w)


def test_strided_rows_given_output_and_the_rows_next_to_it():
    layer = Layer(8, 256, 128, FP, seed=6)
    x, ids, w = layer.tokens(9, 2)
    bx, bo = torch.zeros((9, 264), dtype=FP, device=DEV), torch.full((11, 301), 5.0, dtype=FP, device=DEV)
    bx[:, 8:].copy_(x)
    out = bo[1:10, 3:259]
    got = layer.run(bx[:, 8:], ids, w, out=out)
    assert got.data_ptr() == out.data_ptr()
    layer.check(got, x, ids, w)
    assert (bo[0] == 5).all() and (bo[10] == 5).all() and (bo[:, :3] == 5).all() and (bo[:, 259:] == 5).all()


def test_output_over_the_input_and_on_another_stream():
    layer = Layer(8, 256, 128, BF, seed=6)
    x, ids, w = layer.tokens(9, 2)
    want = layer.run(x, ids, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x.clone()
        got = layer.run(y, ids, w, out=y)
    side.synchronize()
    assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)


def test_a_token_does_not_depend_on_the_others_values():
    layer = Layer(8, 256, 128, BF, seed=7)
    x, ids, w = layer.tokens(12, 3)
    x2 = x.clone()
    x2[5], x2[8] = float("nan"), float("inf")
    a, b = layer.run(x, ids, w), layer.run(x2, ids, w)
    rows = [t for t in range(12) if t not in (5, 8)]
    assert torch.equal(a[rows], b[rows]) and torch.isnan(b[5]).all()


def test_as_the_separate_calls():
    """Within the roundings the separate calls make more: h and each expert's output."""
    layer = Layer(128, 512, 256, BF, seed=8)
    x, ids, w = layer.tokens(16, 8)
    got = layer.run(x, ids, w)
    off, row_token, token_row = nv.moe_route(ids, 128)
    a = nv.moe_fc1(x, row_token, off, layer.b1, 128, 256, 512, layer.g1)
    y = nv.moe_combine(nv.grouped_gemm(a, off, layer.b2, 128, 512, 256, layer.g2), token_row, w)
    # gate and up, a, the experts' outputs and the sum, on each side at most
    assert float((got.double() - y.double()).norm() / y.double().norm()) < 2.0 ** -8 * (7 / 3) ** 0.5


def test_one_workspace_for_calls_of_many_sizes_and_graphs():
    layers = [Layer(16, 512, 256, BF, seed=1), Layer(8, 1056, 352, BF, seed=2)]
    calls = [(layers[0], layers[0].tokens(4, 4)), (layers[1], layers[1].tokens(64, 2)), (layers[0], layers[0].tokens(1, 2))]
    need = max(nv.moe_layer_workspace_bytes(a[0].shape[0], a[1].shape[1], l.E, l.H, l.I) for l, a in calls)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    ws[:4096] = 0
    want = [l.run(*a) for l, a in calls]
    graphs = []
    for (l, a), first in zip(calls, want):
        out = torch.empty_like(first)
        assert torch.equal(l.run(*a, out=out, workspace_buf=ws), first)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.run(*a, out=out, workspace_buf=ws)
        graphs.append((g, out))
    for _ in range(4):
        for (g, out), first in zip(graphs, want):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
    assert (ws[:4096] == 0).all()
