"""Page tables and slots from request lengths on the GPU, against a plain loop over the requests."""
import numpy as np
import pytest
import torch

import step_ref as ref
import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def make(rng, B, page, longest, most, width=None, spare=5):
    cached = rng.integers(0, longest + 1, B)
    new = rng.integers(0, most + 1, B)
    width = -(-(longest + most) // page) + 1 if width is None else width
    held = -(-cached // page)
    need = -(-(cached + new) // page) - held
    order = rng.permutation(int(held.sum() + need.sum()) + spare)
    table, at = np.full((B, width), -7), 0
    for b in range(B):
        n = min(width, held[b])
        table[b, :n] = order[at:at + n]
        at += held[b]
    return cached, new, table, order[at:], rng.integers(0, spare + 1)


def check(cached, new, table, free, head, page, tokens, table_dev=None, **kw):
    want = ref.plan(cached, new, table, free, head, page, tokens)
    t = dev(table) if table_dev is None else table_dev
    got = nv.kv_plan(dev(cached), dev(new), t, dev(free), dev([head]), page, tokens, **kw)
    for name, g, w in zip(("slots", "positions", "requests", "lengths", "offsets", "head", "table"), (*got, t), want):
        assert np.array_equal(g.cpu().numpy(), w), name
    return got


@pytest.mark.parametrize("B,page,longest,most,extra", [
    (1, 16, 0, 1, 0), (1, 16, 40, 1, 3), (16, 16, 8192, 1, 0), (7, 1, 5, 3, 2), (33, 48, 500, 100, 0), (64, 128, 0, 60, 9),
    (1023, 16, 300, 1, 0), (1025, 7, 100, 2, 1), (4096, 16, 50, 1, 0), (4097, 16, 50, 1, 0), (5000, 32, 70, 0, 0),
    (20, 16, 1000, 1000, 100), (600, 16, 0, 400, 5), (9000, 16, 20, 8, 0), (2, 16, 0, 70000, 0),
])
def test_plan(B, page, longest, most, extra):
    rng = np.random.default_rng(B * 31 + page)
    case = make(rng, B, page, longest, most)
    check(*case, page, int(case[1].sum()) + extra)


@pytest.mark.parametrize("B", [3, 900, 4500])
@pytest.mark.parametrize("fault", ["list", "table", "rows", "negative", "empty list", "late head"])
def test_refused_requests(B, fault):
    rng = np.random.default_rng(B + len(fault))
    page, longest, most = 16, 60, 40
    cached, new, table, free, head = make(rng, B, page, longest, most)
    tokens = int(new.sum())
    if fault == "list":
        free = free[:len(free) // 2]
    elif fault == "table":
        table = table[:, :3].copy()
    elif fault == "rows":
        tokens //= 2
    elif fault == "negative":
        cached[::3] = -1
        new[1::5] = -4
    elif fault == "empty list":
        free = free[:0]
    else:
        head = len(free) + 3
    check(cached, new, table, free, head, page, tokens)


def test_pages_without_a_slot():
    """Entries of the table or the list outside the slots' range give -1 and nothing else."""
    free = np.array([5, -3, 2 ** 31 // 16, 2 ** 31 // 16 - 1, 9])
    check(np.array([0, 17]), np.array([70, 20]), np.array([[0] * 6, [-1, 2 ** 31 - 1] + [0] * 4]), free, 0, 16, 90)


@pytest.mark.parametrize("B", [5, 300, 5000])
def test_lengths_beyond_all_limits(B):
    """Sums of lengths past 32 bits, and lengths whose own sum is: those requests are refused, the ones before them not."""
    cached, new = np.full(B, 20), np.full(B, 3)
    new[1::2] = 2 ** 31 - 1
    cached[2::4] = 2 ** 31 - 1
    check(cached, new, np.zeros((B, 4)), np.arange(4 * B), 0, 16, 50)
    new[:] = 2 ** 30
    check(cached, new, np.zeros((B, 4)), np.arange(4 * B), 0, 16, 50)


@pytest.mark.parametrize("tokens", [0, 5, 5000])
def test_no_requests_and_no_rows(tokens):
    got = check(np.zeros(0), np.zeros(0), np.zeros((0, 4)), np.arange(3), 1, 16, tokens)
    assert got.offsets.tolist() == [0] and got.head.tolist() == [1]
    check(np.array([3]), np.array([0]), np.array([[1]]), np.arange(3), 1, 16, tokens)
    check(np.array([0]), np.array([0]), np.zeros((1, 0)), np.zeros(0), 0, 16, tokens)


def test_strided_table_and_given_outputs():
    rng = np.random.default_rng(8)
    cached, new, table, free, head = make(rng, 40, 16, 200, 30)
    big = torch.full((40, table.shape[1] + 9), 77, dtype=torch.int32, device=DEV)
    view = big[:, 4:4 + table.shape[1]]
    view.copy_(dev(table))
    tokens = int(new.sum())
    out = nv.KvPlan(*(torch.full((n,), 99, dtype=torch.int32, device=DEV) for n in (tokens, tokens, tokens, 40, 41, 1)))
    got = check(cached, new, table, free, head, 16, tokens, table_dev=view, out=out)
    assert all(g.data_ptr() == o.data_ptr() for g, o in zip(got, out))
    assert (big[:, :4] == 77).all() and (big[:, 4 + table.shape[1]:] == 77).all()


@pytest.mark.parametrize("B,most", [(5, 4), (5, 3000), (32, 32), (41, 25), (65, 3)])
def test_steps_that_advance_in_place_and_as_a_graph(B, most):
    """lengths over cached and head over free_head: each step goes on where the last ended, also replayed."""
    rng = np.random.default_rng(most)
    page, steps = 16, 5
    news = [rng.integers(0, most + 1, B) for _ in range(steps)]
    width = -(-steps * most // page) + 1
    free = rng.permutation(B * width)
    tokens = B * most

    def buffers():
        return (torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV),
                torch.zeros((B, width), dtype=torch.int32, device=DEV), dev(free), torch.zeros(1, dtype=torch.int32, device=DEV))

    def outputs(cached, head):
        rows = [torch.empty(tokens, dtype=torch.int32, device=DEV) for _ in range(3)]
        return (*rows, cached, torch.empty(B + 1, dtype=torch.int32, device=DEV), head)

    cached, new, table, fr, head = buffers()
    out = outputs(cached, head)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.kv_plan(cached, new, table, fr, head, page, tokens, out=out)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        nv.kv_plan(cached, new, table, fr, head, page, tokens, out=out)
    c, t, h = np.zeros(B), np.zeros((B, width)), 0
    for n in news:
        want = ref.plan(c, n, t, free, h, page, tokens)
        new.copy_(dev(n))
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip((*out, table), want):
            assert np.array_equal(g.cpu().numpy(), w)
        c, h, t = want[3], int(want[5][0]), want[6]
    assert h > 0


def test_another_stream():
    rng = np.random.default_rng(3)
    cached, new, table, free, head = make(rng, 300, 16, 100, 50)
    args = [dev(x) for x in (cached, new, table, free, [head])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = nv.kv_plan(*args, 16, int(new.sum()))
    side.synchronize()
    assert np.array_equal(got.slots.cpu().numpy(), ref.plan(cached, new, table, free, head, 16, int(new.sum()))[0])
