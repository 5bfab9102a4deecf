"""What a row of lora_add depends on: its own values and adapter, and the call's sizes, not where it stands or who its
neighbours are."""
import pytest
import torch

import weight_only_fp4_amd as nv
from test_gpu_lora import BF, DEV, FP, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,R,L,dtype", [
    (30, 1024, 300, 16, 6, BF), (30, 1024, 300, 16, 64, FP), (200, 4096, 130, 64, 3, BF), (256, 640, 72, 128, 9, FP),
    (257, 640, 72, 128, 9, BF), (700, 2048, 200, 32, 5, FP), (700, 2048, 200, 32, 900, BF),
])
def test_rows_in_another_order_have_the_same_bits(T, K, N, R, L, dtype):
    y, x, a, b, adapter, scale = make(T, K, N, R, L, dtype, seed=T)
    want = nv.lora_add(y, x, a, b, adapter, scale)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for order in (torch.randperm(T, generator=g, device=DEV), adapter.argsort(), torch.arange(T - 1, -1, -1, device=DEV)):
        got = nv.lora_add(y[order], x[order], a, b, adapter[order].contiguous(), scale)
        assert torch.equal(got, want[order])


@pytest.mark.parametrize("T", [30, 300])
def test_other_rows_values_and_adapters_do_not_count(T):
    y, x, a, b, adapter, scale = make(T, 1024, 300, 16, 6, BF, seed=4)
    want = nv.lora_add(y, x, a, b, adapter, scale)
    keep = torch.arange(T, device=DEV) % 3 == 0
    others = torch.randint(-1, 7, (T,), device=DEV, dtype=torch.int32)
    got = nv.lora_add(torch.where(keep[:, None], y, y * 2), torch.where(keep[:, None], x, -x), a, b,
                      torch.where(keep, adapter, others), scale)
    assert torch.equal(got[keep], want[keep])
