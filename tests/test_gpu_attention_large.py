"""The attention half on the GPU at sizes no other test has: blocks of more than 2 GB, segments of many tiles, uneven
batches of more sequences than are counted."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import weight_only_fp4_amd as nv
from test_gpu_attention import BF, DEV, HF, gen, normal, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page", [(256, (1 << 24) + 67), (128, (1 << 25) + 62), (64, (1 << 26) + 60)])
def test_nvfp4_blocks_past_two_gigabytes(D, page):
    """A page whose codes pass 2 GB: rows on both sides of the 2^31st byte and at the end are written where the layout
    has them, read back, and attended to (a window over the last)."""
    say(f"NVFP4 page of {page} tokens, D={D}")
    page += -page % (256 // D)                       # whole 16-byte steps
    turn = (1 << 31) // (D // 2)                     # the first token past 2^31 bytes of codes
    assert turn < page - 40
    kc, vc = nv.kv_cache(1, 1, page, D, torch.uint8, DEV)
    at = sorted({0, 1, turn - 1, turn, turn + 1} | set(range(page - 40, page)))
    g = gen(D)
    k, v, q = (normal(s, g, BF) for s in ((len(at), 1, D), (len(at), 1, D), (1, 4, D)))
    slots = torch.tensor(at, dtype=torch.int32, device=DEV)
    nv.kv_write(k.to(DEV), v.to(DEV), kc, vc, slots)
    held = []
    for cache, x in ((kc, k), (vc, v)):
        codes, S = ref.stored(ref.f64(x), None, "fp4")
        flat = cache.view(-1)
        for i, t in enumerate(at):
            b = flat[t * (D // 2):(t + 1) * (D // 2)].cpu().numpy()
            code = np.stack((b & 15, b >> 4), -1).reshape(D)
            np.testing.assert_array_equal(np.where(code >= 8, -1.0, 1.0) * ref.E2M1[code & 7], codes[i, 0])
            first = page * (D // 2) + t * (D // 16)
            np.testing.assert_array_equal(ref.e4m3_of_bytes(flat[first:first + D // 16].cpu().numpy()), S[i, 0])
        held.append(ref.value(codes, S, None))
    for got, want in zip(nv.kv_read(kc, vc, slots, HF), held):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(HF))
    out, lse = nv.paged_attention(q.to(DEV), kc, vc, torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                                  torch.tensor([page], dtype=torch.int32, device=DEV), window=40, return_lse=True)
    o, l, bo, bl = ref.attention(ref.f64(q[0]), held[0][-40:, 0], held[1][-40:, 0], ref.default_scale(D), (HF, BF))
    assert np.all(np.abs(ref.f64(out[0]) - o) <= bo) and np.all(np.abs(ref.f64(lse[0]) - l) <= bl)
