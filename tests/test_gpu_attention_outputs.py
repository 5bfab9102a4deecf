"""Outputs the attention half's calls refuse: rows that share memory would be written by several workgroups at once."""
import pytest
import torch

import weight_only_fp4_amd as nv

pytestmark = pytest.mark.gpu
DEV, BF = "cuda:0", torch.bfloat16


def test_outputs_whose_rows_share_memory_are_refused():
    x, w = torch.ones((4, 64), dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    one = torch.zeros((1, 64), dtype=BF, device=DEV).expand(4, 64)
    h = torch.ones((4, 2, 64), dtype=BF, device=DEV)
    rows, heads = torch.zeros((1, 2, 64), dtype=BF, device=DEV).expand(4, 2, 64), h[:, :1].clone().expand(4, 2, 64)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    inv = torch.ones(32, device=DEV)
    kc, vc = nv.kv_cache(3, 2, 16, 64, BF, DEV)
    shared = kc[:, :1].clone().expand(3, 2, 16, 64)
    table, n = torch.zeros((4, 1), dtype=torch.int32, device=DEV), torch.ones(4, dtype=torch.int32, device=DEV)
    for call in (
        lambda: nv.rms_norm(x, w, out=one), lambda: nv.rms_norm(x, w, residual=x, residual_out=one),
        lambda: nv.rms_norm_fp8(x, w, out=one.to(torch.float8_e4m3fn)[:1].expand(4, 64)),
        lambda: nv.rms_norm_fp8(x, w, scales=torch.zeros(1, device=DEV).expand(4)),
        lambda: nv.rope(h, pos, inv, out=rows), lambda: nv.rope(h, pos, inv, out=heads),
        lambda: nv.rope_kv_write(h, h, h, pos, inv, kc, vc, pos, out=heads),
        lambda: nv.kv_write(h, h, shared, vc, pos), lambda: nv.kv_write(h, h, kc, shared, pos),
        lambda: nv.kv_read(kc, vc, pos, out=(rows, h)), lambda: nv.kv_read(kc, vc, pos, out=(h, heads)),
        lambda: nv.paged_attention(h, kc, vc, table, n, out=rows),
    ):
        with pytest.raises(ValueError, match="share memory|unit stride"):
            call()
    # read, they are fine; so is an output row by row inside a larger one
    out = torch.zeros((4, 3, 2, 64), dtype=BF, device=DEV)[:, 1]
    assert torch.equal(nv.rope(rows + 1, pos, inv, out=out), rows + 1)
    assert torch.equal(nv.paged_attention(heads, shared, shared, table, n), nv.paged_attention(
        heads, shared.contiguous(), shared.contiguous(), table, n))
