"""The next token from logits on the GPU, against 64-bit sorting and sums."""
import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f32(v):
    return None if v is None else torch.tensor(v, dtype=torch.float32, device=DEV)


def check(logits, u, t=None, k=None, p=None, min_p=None, **kw):
    B = logits.shape[0]
    kd = None if k is None else torch.tensor(k, dtype=torch.int32, device=DEV)
    tokens, logprobs = nv.sample(logits, f32(u), f32(t), kd, f32(p), f32(min_p), return_logprobs=True, **kw)
    rows = logits.double().cpu().numpy()
    as32 = lambda v, d: [d] * B if v is None else np.float32(v).astype(np.float64)  # noqa: E731
    us, ts, ps, ms = as32(u, 0), as32(t, 1.0), as32(p, 1.0), as32(min_p, 0.0)
    ks = [0] * B if k is None else k
    for b in range(B):
        token, lp = ref.sample_row(rows[b], us[b], ts[b], ks[b], ps[b], ms[b])
        assert int(tokens[b]) == token, (b, int(tokens[b]), token, us[b], ts[b], ks[b], ps[b], ms[b])
        got = float(logprobs[b])
        # computed in 64 bits from weights to 2^-38 or better of the total and rounded once
        assert got == lp or abs(got - lp) <= abs(lp) * 2.0 ** -24 + 2.0 ** -26, (b, got, lp)
    return tokens


def logits_of(B, V, dtype, seed, sigma=2.5, masked=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((B, V), generator=g, device=DEV) * sigma
    if masked:
        x = x.masked_fill(torch.rand((B, V), generator=g, device=DEV) < masked, -float("inf"))
    return x.to(TYPES[dtype])


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 63), (4, 1000), (7, 4097), (3, 32003), (2, 131072), (2, 200001)])
def test_settings(dtype, B, V):
    rng = np.random.default_rng(V)
    x = logits_of(B, V, dtype, V)
    u = lambda: rng.random(B).astype(np.float32)  # noqa: E731
    check(x, u())
    check(x, u(), t=rng.uniform(0.3, 3, B))
    check(x, u(), k=rng.integers(1, 60, B).tolist())
    check(x, u(), p=rng.uniform(0.05, 0.99, B))
    check(x, u(), min_p=rng.uniform(0.001, 0.3, B))
    check(x, u(), t=rng.uniform(0.3, 3, B), k=rng.integers(1, max(2, V), B).tolist(), p=rng.uniform(0.3, 1.1, B),
          min_p=rng.uniform(0, 0.05, B))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_each_row_has_its_settings(dtype):
    B, V = 64, 5003
    rng = np.random.default_rng(1)
    pick = lambda *v: [v[i] for i in rng.integers(0, len(v), B)]  # noqa: E731
    check(logits_of(B, V, dtype, 2, masked=0.4), rng.random(B), t=pick(0.0, -1.0, 0.5, 1.0, 1e-6, 1e4, float("nan")),
          k=pick(0, -3, 1, 2, 50, 5003, 1 << 30), p=pick(0.0, -1.0, 0.1, 0.9, 1.0, 2.0, float("nan")),
          min_p=pick(0.0, -0.5, 0.1, 1.0, 2.0, float("nan")))


@pytest.mark.parametrize("V", [9, 4099, 70000])
@pytest.mark.parametrize("kind", ["equal", "two values", "steps", "flat", "peak", "half masked", "one left", "wide"])
def test_ties_and_masks(kind, V):
    B = 6
    rng = np.random.default_rng(V + len(kind))
    i = torch.arange(V, device=DEV)
    x = torch.zeros((B, V), device=DEV)
    if kind == "two values":
        x[:, i % 3 == 1] = 1.0
    elif kind == "steps":
        x += (i * 7919 % 13).float()
    elif kind == "flat":
        x += torch.randn((B, V), device=DEV) * 0.01
    elif kind == "peak":
        x[:, V // 2] = 50.0
    elif kind == "half masked":
        x[:, i % 2 == 0] = -float("inf")
    elif kind == "one left":
        x[:] = -float("inf")
        x[:, V - 2] = -3.0
    elif kind == "wide":
        x += torch.randn((B, V), device=DEV) * 1e5
    for dtype in TYPES.values():
        y = x.to(dtype)
        check(y, rng.random(B), k=rng.integers(1, V + 1, B).tolist())
        check(y, rng.random(B), p=rng.uniform(0.05, 0.95, B))
        check(y, rng.random(B), t=rng.uniform(0.5, 2, B), k=rng.integers(1, V + 1, B).tolist(), p=rng.uniform(0.2, 1, B),
              min_p=[0.5] * B)
        check(y, rng.random(B))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_infinities_nan_zeros_and_empty_rows(dtype):
    V, inf, nan = 300, float("inf"), float("nan")
    x = torch.randn((8, V), device=DEV)
    x[0] = -inf
    x[1] = nan
    x[2, 7], x[2, 200] = inf, inf
    x[3, ::2] = nan
    x[4] = -0.0
    x[4, 5:9] = 0.0
    x[5] = torch.finfo(TYPES[dtype]).min
    x[6] = torch.finfo(TYPES[dtype]).min
    x[6, 77] = 1.0
    x[7, 3] = inf
    x[7, 9] = nan
    y = x.to(TYPES[dtype])
    for u in (0.0, 0.3, 0.999):
        assert check(y, [u] * 8)[:2].tolist() == [-1, -1]
        check(y, [u] * 8, k=[3] * 8, p=[0.6] * 8)
        check(y, [u] * 8, t=[0.0] * 8)
        check(y, [u] * 8, t=[inf] * 8, min_p=[0.2] * 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_slices_of_several_reads_and_very_long_rows(dtype):
    """So many rows that a slice is more than a workgroup holds, and rows of the most slices."""
    rng = np.random.default_rng(7)
    B = 300
    x = logits_of(B, 40001, dtype, 8)
    k = [int(v) for v in rng.choice([0, 1, 40, 700], B)]
    check(x, rng.random(B), t=rng.choice([0.0, 0.7, 1.3], B), k=k, p=rng.choice([0.5, 0.9, 1.0], B),
          min_p=rng.choice([0.0, 0.05], B))
    x = logits_of(1, 1200007, dtype, 9)
    for kw in (dict(), dict(k=[300]), dict(p=[0.8]), dict(min_p=[0.03]), dict(t=[0.0])):
        check(x, rng.random(1), **kw)


def test_long_lists():
    """More candidates than a slice or a row lists: the row itself is read again."""
    rng = np.random.default_rng(8)
    x = logits_of(4, 60000, "fp32", 10)
    check(x, rng.random(4), k=[5000, 9000, 2500, 59999], p=[1.0, 0.9, 0.7, 0.99])
    check(x * 0.02, rng.random(4), p=[0.1, 0.5, 0.9, 0.999])
    check(x * 0.02, rng.random(4), min_p=[0.9, 0.99, 0.95, 0.5], p=[1.0, 0.9, 1.0, 0.9])


@pytest.mark.parametrize("large", [3e5, 1e6, 1e8, 1e30])
def test_logits_far_from_zero(large):
    """Grids whose bins are finer than the logits' own steps."""
    rng = np.random.default_rng(9)
    x = logits_of(5, 9000, "fp32", 11)
    for y in (x + large, x - large, x * large):
        for kw in (dict(), dict(k=[30] * 5), dict(p=[0.7] * 5), dict(min_p=[0.2] * 5), dict(min_p=[0.2] * 5, p=[0.9] * 5)):
            check(y, rng.random(5), t=rng.uniform(0.3, 3, 5), **kw)


def test_random_numbers_at_their_ends():
    x = logits_of(7, 999, "fp32", 3)
    check(x, [0.0, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan"), 2.0 ** -24])


def test_draws_follow_the_weights():
    """With evenly spread random numbers every kept token comes as often as its weight says, within one."""
    n = 4096
    x = torch.tensor([0.0, 1.0, 2.0, -1.0, 1.0], device=DEV).expand(n, 5)
    u = (torch.arange(n, device=DEV) + 0.5) / n
    got = torch.bincount(nv.sample(x, u).long(), minlength=5).double().cpu()
    want = torch.softmax(x[0].double().cpu(), 0) * n
    assert (got - want).abs().max() <= 1


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_rows_of_any_alignment_and_stride(dtype):
    rng = np.random.default_rng(4)
    big = logits_of(6, 2100, dtype, 5)
    for first, V in ((0, 2000), (1, 2000), (3, 1999), (7, 1), (5, 17)):
        check(big[:, first:first + V], rng.random(6), k=[40] * 6, p=[0.9] * 6)
    check(big[::2, 1:1000], rng.random(3))
    check(big[:1, :].expand(4, 2100), rng.random(4), p=[0.5] * 4)


def test_the_same_bits_each_time_and_as_a_graph():
    x = logits_of(9, 40000, "bf16", 6)
    B = 9
    u, t, p = torch.rand(B, device=DEV), torch.full((B,), 0.8, device=DEV), torch.full((B,), 0.9, device=DEV)
    k = torch.full((B,), 2000, dtype=torch.int32, device=DEV)
    ws = nv.workspace(max(nv.sample_workspace_bytes(B, 40000), 16), DEV)
    out = torch.zeros(B, dtype=torch.int32, device=DEV)
    first = nv.sample(x, u, t, k, p, return_logprobs=True)
    assert torch.equal(nv.sample(x, u, t, k, p, out=out, workspace_buf=ws), first[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.sample(x, u, t, k, p, out=out, workspace_buf=ws)
    for _ in range(3):
        u.copy_(torch.rand(B, device=DEV))
        want = nv.sample(x, u, t, k, p)
        out.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        again = nv.sample(x, u, t, k, p, return_logprobs=True)
        assert torch.equal(again[0], want)
