"""Sizes at the edge of what the attention half's calls take, on the CPU: refusals come before any launch."""
import ctypes

import pytest

import weight_only_fp4_amd as nv

OK, INVALID = 0, 1
A = 1 << 20   # a fake, aligned address; never dereferenced


@pytest.mark.parametrize("N,status", [(2 ** 31 - 256, OK), (2 ** 31 - 255, INVALID), (2 ** 31 - 1, INVALID), (2 ** 31, INVALID)])
def test_norm_rows_whose_column_counter_would_wrap_are_refused(N, status):
    """No rows, so that an accepted call launches nothing."""
    P, I64 = ctypes.c_void_p, ctypes.c_int64
    f = ctypes.CFUNCTYPE(ctypes.c_int, P, I64, P, I64, P, ctypes.c_float, P, I64, P, P, I64, I64, I64, ctypes.c_int,
                         P)(("nvfp4_rms_norm", nv.lib()))
    assert f(A, N, None, 0, A, 1e-6, A, N, None, None, 0, 0, N, 0, None) == status
