"""Gathers of the 8-bit quantizers at their edges."""
import pytest

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [16, 129, 512])
def test_a_gather_from_no_rows(cols, dtype):
    """Every row is outside an input without rows: zeros, and the scale of zeros."""
    from fine_grained_mixture_top_b200 import moe
    src = torch.tensor([-1, 0, 5, -1, 2 ** 31 - 1] * 30, dtype=torch.int32, device="cuda")
    for swiglu in (False, True):
        x = torch.empty(0, cols * (2 if swiglu else 1), dtype=dtype, device="cuda")
        q, s = moe.fp8_quantize_rows(x, row_src=src, swiglu=swiglu)
        assert q.shape == (150, cols) and torch.all(q.float() == 0)
        assert torch.all(s == torch.tensor(2.0 ** -110) / 448.0)
    q, s = moe.fp8_quantize_cols(torch.empty(0, cols, dtype=dtype, device="cuda"), row_src=src)
    assert q.shape == (cols, 150) and torch.all(q.float() == 0)
    assert torch.all(s == torch.tensor(2.0 ** -110) / 448.0)
    assert moe.moe_get_status() == (0, 0)
