"""The attention half on the GPU at sizes no other test has: blocks of more than 2 GB, segments of many tiles, uneven
batches of more sequences than are counted."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import weight_only_fp4_amd as nv
from test_gpu_attention import BF, DEV, HF, Paged, gen, normal, say

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


@pytest.mark.parametrize("kind", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [3968, 4095, 4096, 4097, 4224, 8192, 8300])
def test_segments_of_more_tiles_than_are_looked_up_at_once(n, D, kind):
    """More sequences than are counted: each is one segment, whose waves look their pages up 32 tiles (4096 tokens) at a
    time.  One and two lookups, filled and begun; a window that starts inside the first; pages outside the cache behind
    it."""
    say(f"segment of {n} tokens, D={D}, {kind}")
    lengths = [0] * 2049
    lengths[1027] = n
    p = Paged(lengths, 3, 1, D, 16, kind, BF if D != 128 else HF, seed=n)
    p.check(p.run())
    for window in (n - 75, 4097):
        if window < n:
            p.check(p.run(window=window), window=window)
    table = p.table.clone()
    out = [70, 253, 254, 257, 300, 513]
    for page in out:
        if page < table.shape[1]:
            table[1027, page] = -1 if page % 2 else p.kc.shape[0]
    keep = [np.ones(m, dtype=bool) for m in lengths]
    keep[1027] = ~np.isin(np.arange(n) // 16, out)
    p.check(p.run(table=table), keep=keep)
