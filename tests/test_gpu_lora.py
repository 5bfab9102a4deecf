"""Low-rank adapters on the GPU, against 64-bit sums."""
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def make(T, K, N, R, L, dtype, seed=0, sigma=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=DEV) * scale).to(dtype)  # noqa: E731
    adapter = torch.randint(-1, L + 1, (T,), generator=g, device=DEV, dtype=torch.int32)   # none: -1 and L
    return (r(T, N), r(T, K, scale=sigma), r(L, R, K, scale=K ** -0.5), r(L, N, R, scale=R ** -0.5), adapter,
            torch.rand(L, generator=g, device=DEV) * 3 - 1)


def check(got, y, x, a, b, adapter, scale):
    want, bound = ref.lora(y, x, a, b, adapter, scale)
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    none = ~((adapter >= 0) & (adapter < a.shape[0])).cpu()
    assert torch.equal(got.cpu()[none], y.cpu()[none])


@pytest.mark.parametrize("T,K,N,R,L,dtype", [
    (1, 8, 1, 8, 1, BF), (1, 128, 64, 16, 1, FP), (3, 136, 33, 8, 2, BF), (16, 1024, 512, 16, 20, BF),
    (17, 4096, 257, 64, 5, FP), (33, 520, 1000, 24, 3, BF), (40, 2048, 72, 128, 9, FP), (64, 5120, 640, 32, 64, BF),
    (255, 256, 48, 40, 4, FP), (256, 264, 130, 48, 300, BF), (257, 256, 66, 72, 6, BF), (600, 640, 320, 16, 2, FP),
    (1003, 1152, 31, 104, 1, BF), (16, 16384, 16, 16, 16, BF), (300, 8200, 24, 8, 5, FP),
    (384, 256, 150, 16, 30, BF), (385, 256, 150, 16, 30, BF), (385, 512, 150, 64, 3, FP), (1100, 136, 264, 128, 77, BF),
    (2048, 128, 2048, 8, 40, BF),
])
def test_lora(T, K, N, R, L, dtype):
    args = make(T, K, N, R, L, dtype, seed=T + K)
    check(nv.lora_add(*args[:5], scale=args[5]), *args)
    check(nv.lora_add(*args[:5]), *args[:5], None)


@pytest.mark.parametrize("T", [48, 700])
@pytest.mark.parametrize("kind", ["all one", "none", "runs"])
def test_adapters_of_prompts(T, kind):
    args = list(make(T, 512, 200, 32, 4, BF, seed=T))
    if kind == "all one":
        args[4] = torch.full((T,), 2, dtype=torch.int32, device=DEV)
    elif kind == "none":
        args[4] = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    else:
        args[4] = (torch.arange(T, device=DEV) // 37 % 5 - 1).to(torch.int32)
    check(nv.lora_add(*args[:5], scale=args[5]), *args)


def test_no_adapters_and_no_rows():
    y, x = torch.randn((5, 64), device=DEV).to(BF), torch.randn((5, 128), device=DEV).to(BF)
    a, b = torch.empty((0, 16, 128), dtype=BF, device=DEV), torch.empty((0, 64, 16), dtype=BF, device=DEV)
    ids = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert torch.equal(nv.lora_add(y, x, a, b, ids), y)
    assert nv.lora_add(y[:0], x[:0], a, b, ids[:0]).shape == (0, 64)


@pytest.mark.parametrize("T", [9, 400])
def test_in_place_strided_and_misaligned(T):
    K, N, R, L = 256, 90, 16, 3
    y, x, a, b, adapter, scale = make(T, K, N, R, L, FP, seed=5)
    bx, by = torch.zeros((T, K + 40), dtype=FP, device=DEV), torch.full((T, N + 11), 7.0, dtype=FP, device=DEV)
    ba, bb = torch.zeros((L, R + 1, K + 8), dtype=FP, device=DEV), torch.zeros((L, N, R + 24), dtype=FP, device=DEV)
    xv, yv, av, bv = bx[:, 8:8 + K], by[:, 3:3 + N], ba[:, :R, 8:], bb[:, :, 16:16 + R]
    for v, t in ((xv, x), (yv, y), (av, a), (bv, b)):
        v.copy_(t)
    got = nv.lora_add(yv, xv, av, bv, adapter, scale=scale, out=yv)
    assert got.data_ptr() == yv.data_ptr()
    check(got, y, x, a, b, adapter, scale)
    assert (by[:, :3] == 7).all() and (by[:, 3 + N:] == 7).all()


def test_two_calls_at_once_on_two_streams():
    calls = [make(60, 1024, 500, 32, 7, BF, seed=s) for s in (1, 2)]
    want = [nv.lora_add(*c[:5], scale=c[5]) for c in calls]
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for c, st in zip(calls, streams):
            with torch.cuda.stream(st):
                got.append(nv.lora_add(*c[:5], scale=c[5]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


def test_large_and_small_values_in_fp16():
    """x A^T beyond fp16's range, and far below it."""
    for sigma in (60000.0, 2.0 ** -22):
        y, x, a, b, adapter, _ = make(20, 512, 64, 16, 3, FP, seed=9)
        x = (x * (200.0 if sigma > 1 else sigma)).to(FP)
        a = (a * (2000.0 if sigma > 1 else 1.0)).to(FP)
        scale = torch.full((3,), 1e-6 if sigma > 1 else 1e6, device=DEV)
        check(nv.lora_add(y, x, a, b, adapter, scale=scale), y, x, a, b, adapter, scale)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinities_and_nan_stay_in_their_rows(dtype):
    y, x, a, b, adapter, scale = make(20, 256, 64, 16, 3, dtype, seed=2)
    adapter = torch.arange(20, device=DEV, dtype=torch.int32) % 3
    x2 = x.clone()
    x2[4, 7], x2[11, 100] = float("inf"), float("nan")
    p, q = nv.lora_add(y, x, a, b, adapter, scale), nv.lora_add(y, x2, a, b, adapter, scale)
    rows = [t for t in range(20) if t not in (4, 11)]
    assert torch.equal(p[rows], q[rows])
    assert not torch.isfinite(q[4]).any() and torch.isnan(q[11]).all()


def test_two_graphs_share_a_workspace_and_rows_do_not_depend_on_the_batch():
    args = make(30, 1024, 300, 16, 6, BF, seed=4)
    ws = nv.workspace(max(nv.lora_workspace_bytes(30, 1024, 300, 16), 64), DEV)
    want = nv.lora_add(*args[:5], scale=args[5])
    one = torch.cat([nv.lora_add(*(t[i:i + 1] for t in args[:2]), args[2], args[3], args[4][i:i + 1], scale=args[5])
                     for i in range(30)])
    check(one, *args)
    graphs, outs = [], []
    for part in (slice(0, 30), slice(7, 25)):
        out = torch.empty_like(args[0][part])
        ins = (args[0][part], args[1][part], args[2], args[3], args[4][part])
        nv.lora_add(*ins, scale=args[5], out=out, workspace_buf=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.lora_add(*ins, scale=args[5], out=out, workspace_buf=ws)
        graphs.append(g)
        outs.append((out, out.clone()))
    assert torch.equal(outs[0][1], want)
    for _ in range(3):
        for g, (out, first) in zip(graphs, outs):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
