"""What the 8-bit quantizer and products refuse, on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    from fine_grained_mixture_top_b200 import build
    build.build()
    from fine_grained_mixture_top_b200 import moe as m
    return m


def test_c_entries_refuse(moe):
    L = moe.lib()
    rows = lambda type=0, x=4096, ldx=256, r=8, c=200, swiglu=0, q=4096, ldq=208, s=4096, lds=8: (   # noqa: E731
        L.moe_fp8_quantize_rows(type, x, ldx, max(r, 0), r, c, None, None, swiglu, q, ldq, s, lds, None, 0, None))
    assert rows(type=3) == 1 and rows(type=9) == 1           # codes are not quantized again
    assert rows(r=-1) == 1 and rows(c=0) == 1 and rows(swiglu=2) == 1
    assert rows(x=None) == 1 and rows(q=None) == 1 and rows(s=None) == 1
    assert rows(x=4097) == 1 and rows(q=4104) == 1 and rows(s=4098) == 1
    assert rows(ldx=199) == 1 and rows(swiglu=1, ldx=399) == 1
    assert rows(ldq=200) == 1 and rows(ldq=192) == 1         # not a multiple of 16; shorter than a row
    assert rows(lds=7) == 1
    assert rows(c=(1 << 20) + 1, ldx=1 << 21, ldq=1 << 21) == 2 and rows(r=1 << 31, lds=1 << 31) == 2
    assert rows(r=0, x=None) == 0
    cols = lambda x=4096, ldx=200, r=300, c=200, q=4096, ldq=304, lds=200: L.moe_fp8_quantize_cols(   # noqa: E731
        0, x, ldx, r, r, c, None, None, q, ldq, 4096, lds, None)
    assert cols(ldq=288) == 1 and cols(lds=199) == 1 and cols(ldx=100) == 1 and cols(r=65536 * 128, ldq=1 << 24) == 2
    blocks = lambda E=2, K=100, N=64, tr=0, q=4096, ldq=112: L.moe_fp8_quantize_blocks(   # noqa: E731
        0, 4096, E, K, N, tr, q, ldq, 4096, None)
    assert blocks(E=-1) == 1 and blocks(K=0) == 1 and blocks(tr=2) == 1 and blocks(q=None) == 1
    assert blocks(ldq=48) == 1 and blocks(tr=1, ldq=96) == 1 and blocks(E=70000) == 2
    gemm = lambda M=64, N=72, K=100, E=1, rt=None, a=4096, lda=112, sa=4096, ldsa=64, b=4096, ldb=112, sb=4096, c=4096, ldc=72: (   # noqa: E731,E501
        L.moe_fp8_gemm(M, N, K, E, rt, a, lda, sa, ldsa, b, ldb, sb, c, ldc, None))
    assert gemm(M=-1) == 1 and gemm(N=0) == 1 and gemm(K=0) == 1 and gemm(E=0) == 1
    for name in ("a", "sa", "b", "sb", "c"):
        assert gemm(**{name: None}) == 1 and gemm(**{name: 4098}) == 1, name
    assert gemm(lda=96) == 1 and gemm(lda=100) == 1 and gemm(ldb=104) == 1 and gemm(ldc=71) == 1 and gemm(ldc=76) == 1
    assert gemm(ldsa=63) == 1
    assert gemm(E=3) == 2                                    # several experts need a routing
    st = moe.MoeRouting(**{k: 4096 for k in moe._ROUTING_PTRS}, P_max=8, R_max=1024)
    assert gemm(rt=ctypes.byref(st), E=3, M=100, ldsa=128) == 1   # rows in whole tiles
    assert gemm(rt=ctypes.byref(st), E=2000, M=128, ldsa=128) == 2
    st.offsets = None
    assert gemm(rt=ctypes.byref(st), E=3, M=128, ldsa=128) == 1
    assert gemm(M=0, a=None, c=None) == 0
    dw = lambda M=64, N=72, K=256, E=1, rt=None, lda=256, ldsa=64, ldsb=72, ldc=72, c=4096: L.moe_fp8_gemm_dw(   # noqa: E731,E501
        M, N, K, E, rt, 4096, lda, 4096, ldsa, 4096, 256, 4096, ldsb, c, ldc, None)
    assert dw(M=0) == 1 and dw(ldsa=63) == 1 and dw(ldsb=71) == 1 and dw(ldc=64) == 1 and dw(E=2) == 2
    assert dw(K=0, c=None) == 1
    assert moe.last_error() == ""


def test_binding_refuses(moe):
    x = torch.zeros(8, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.fp8_quantize_rows(x)
    with pytest.raises(TypeError):
        moe.fp8_quantize_rows(x.double())
    with pytest.raises(ValueError, match="halves"):
        moe.fp8_quantize_rows(torch.zeros(8, 63), swiglu=True)
    with pytest.raises(TypeError, match="row_src"):
        moe.fp8_quantize_rows(x, row_src=torch.zeros(4))
    with pytest.raises(ValueError, match="contiguous"):
        moe.fp8_quantize_blocks(torch.zeros(2, 64, 8).transpose(1, 2), transpose=True)
    a, sa = torch.zeros(16, 64).to(E4M3), torch.zeros(1, 16)
    b, sb = torch.zeros(24, 64).to(E4M3), torch.zeros(1, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.fp8_gemm(a, sa, b, sb)
    with pytest.raises(TypeError, match="a"):
        moe.fp8_gemm(torch.zeros(16, 64), sa, b, sb)
    with pytest.raises(ValueError, match="16-byte"):
        moe.fp8_gemm(torch.zeros(16, 60).to(E4M3), sa, torch.zeros(24, 60).to(E4M3), sb)
    with pytest.raises(ValueError, match="b: shape"):
        moe.fp8_gemm(a, sa, torch.zeros(24, 128).to(E4M3), sb)
    with pytest.raises(ValueError, match="sa"):
        moe.fp8_gemm(a, torch.zeros(1, 15), b, sb)
    with pytest.raises(ValueError, match="sb"):
        moe.fp8_gemm(a, sa, b, torch.zeros(1, 2))
    with pytest.raises(ValueError, match="sb"):
        moe.fp8_gemm_dw(a, sa, b, torch.zeros(1, 23))
