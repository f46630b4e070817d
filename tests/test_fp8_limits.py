"""Sizes at the edge of what the row and 8-bit calls take, on the host."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    from fine_grained_mixture_top_b200 import build
    build.build()
    from fine_grained_mixture_top_b200 import moe as m
    return m


def test_a_gradient_of_no_tokens_has_the_same_limits(moe):
    """Without a routing there is one product, so one output: several would be
    written past it."""
    dw = lambda M=64, N=72, E=1, rt=None, ldc=72: moe.lib().moe_fp8_gemm_dw(   # noqa: E731
        M, N, 0, E, rt, None, 0, None, 0, None, 0, None, 0, 4096, ldc, None)
    assert dw(E=2) == 2 and dw(E=1025) == 2
    assert dw(M=1 << 31) == 2 and dw(N=1 << 31, ldc=1 << 31) == 2
    st = moe.MoeRouting(**{k: 4096 for k in moe._ROUTING_PTRS}, P_max=8, R_max=0)
    assert dw(E=1025, rt=ctypes.byref(st)) == 2


def test_sizes_whose_product_leaves_64_bits(moe):
    """2^62 tokens of 4 choices, or rows of 4 blocks, come to 0 in 64 bits."""
    P, R, ws = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
    L = moe.lib()
    assert L.moe_sort_sizes(1 << 62, 8, 4, ctypes.byref(P), ctypes.byref(R), ctypes.byref(ws)) == 2
    st = moe.MoeRouting(**{k: 4096 for k in moe._ROUTING_PTRS}, P_max=8, R_max=1024)
    assert L.moe_sort_pairs(1 << 62, 8, 4, ctypes.byref(st), None, 0, None) == 2
    assert L.moe_fp8_quantize_rows(0, 4096, 512, 8, 1 << 62, 512, None, None, 0, 4096, 512, 4096, 1 << 62, None, 0,
                                   None) == 2
