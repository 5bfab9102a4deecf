"""The benchmark's source digest, by which recorded HBM traffic counts as current: it covers the sources of the kernels that
the benchmark times, and no others."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "weight_only_fp4_amd", "csrc")
TIMED = ["nvfp4_w4a16.hip", "nvfp4_mfma.hip", "gemm_small.hip", "gemm_tile.hip", "gemm_xres.hip", "gemm_mfma.hip"]


def included(name, seen):
    if "/" in name or name in seen or not os.path.exists(os.path.join(CSRC, name)):
        return seen
    seen.add(name)
    with open(os.path.join(CSRC, name)) as f:
        for other in re.findall(r'#include "([^"]+)"', f.read()):
            included(other, seen)
    return seen


def test_the_digest_covers_the_timed_kernels_sources():
    covered = set(os.listdir(CSRC)) - bench.NOT_TIMED
    needed = set().union(*(included(name, set()) for name in TIMED))
    assert covered == needed
