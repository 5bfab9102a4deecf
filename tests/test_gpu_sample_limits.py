"""The next token where the bins of a row's logits end: largest logits about 2^18 temperatures from zero, up to which a
slice's bins are exact.  Such a row's slices lie on both sides of that limit."""
import numpy as np
import pytest
import torch

import weight_only_fp4_amd as nv
from test_gpu_sample import check, logits_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LIMIT = 2.0 ** 18


def at_the_limit(B, V, largest, t, seed):
    """Normal logits (in units of t), each row's largest `largest` t."""
    x = logits_of(B, V, "fp32", seed).double()
    return ((x - x.amax(1, keepdim=True) + largest) * t).float()


@pytest.mark.parametrize("V", [9001, 131072])
@pytest.mark.parametrize("t", [1.0, 0.0625])
@pytest.mark.parametrize("inside", [-0.5, 0.5, 4.0, 20.0, 33.0, 70.0])
@pytest.mark.parametrize("side", [-1, 1])
def test_slices_on_both_sides(V, t, inside, side):
    rng = np.random.default_rng(V + int(8 * inside))
    B = 3
    x = at_the_limit(B, V, side * LIMIT - side * inside, t, seed=V)
    u = lambda: rng.random(B).astype(np.float32)  # noqa: E731
    for kw in (dict(), dict(p=[0.9] * B), dict(p=[0.5] * B, min_p=[0.01] * B), dict(min_p=[0.05] * B), dict(k=[50] * B)):
        check(x, u(), t=[t] * B, **kw)


@pytest.mark.parametrize("t", [0.37, 1.9])
def test_a_slice_far_below_the_row(t):
    """One slice has the row's largest, the others lie up to the bins' whole reach below it, past the limit."""
    V = 70000
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = -torch.rand((4, V), generator=g, device=DEV).double() * 14
    x[:, 60000:60040] = 3
    for inside in (0.01, 1.0, 16.0):
        y = ((x - 3 - LIMIT + inside) * t).float()
        check(y, [0.05, 0.3, 0.6, 0.97], t=[t] * 4)
        check(y, [0.05, 0.3, 0.6, 0.97], t=[t] * 4, p=[0.97, 0.9, 0.6, 0.2])


def test_the_limit_does_not_move_a_distribution():
    """Every token as often as its weight says, across a slice that lies past the limit."""
    n, V = 512, 20000
    x = torch.full((V,), -LIMIT - 8.0, device=DEV)
    x[100], x[19000] = -LIMIT + 0.5, -LIMIT - 0.5   # in two slices, one on each side
    u = (torch.arange(n, device=DEV) + 0.5) / n
    got = torch.bincount(nv.sample(x.expand(n, V), u).long(), minlength=V).double().cpu()
    want = torch.softmax(x.double().cpu(), 0) * n
    assert abs(float(got[100] - want[100])) <= 1 and abs(float(got[19000] - want[19000])) <= 1
