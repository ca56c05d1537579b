"""CPU check: fp8_block_gemm refuses an output over its codes."""
import ctypes

import pytest

import sparse_moe_transformer_fwd_b200 as moe
from sparse_moe_transformer_fwd_b200 import _native as N

A = 0x7F0000000000  # never dereferenced on the host


@pytest.mark.parametrize("T,K,n,f32,offset", [(4, 256, 128, 0, 0), (4, 256, 128, 0, 1008), (4, 256, 128, 0, -1008),
                                              (4, 256, 128, 1, -1024), (300, 128, 4096, 0, 16)])
def test_out_over_the_codes(T, K, n, f32, offset):
    s = moe.make_linear_shape(T, K, n)
    s.out_f32 = f32
    need = moe.moe_linear_workspace_size(s)
    p = lambda v: ctypes.c_void_p(v)
    far = p(A + (1 << 30))
    rc = moe.lib().fp8_block_gemm(ctypes.byref(s), p(A), far, far, far, None, p(A + offset), far, need, None)
    assert rc == N.MOE_ERR_INVALID_ARG and "overlaps" in moe.moe_last_error()
