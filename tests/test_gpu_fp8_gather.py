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


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,R,swiglu,dtype", [(3, 7168, 2600, False, torch.bfloat16),
                                                (2000, 1024, 16512, True, torch.bfloat16),
                                                (700, 4001, 4300, False, torch.float16),
                                                (50, 520, 32640, False, torch.float32)])
def test_rows_that_repeat_often(T, C, R, swiglu, dtype):
    """A gather of at least six times the input's rows and more than 2^24 codes
    quantizes each row once and copies its codes: the same bits as pieces of it
    that are too small for that, here and on a stream given by name."""
    from fine_grained_mixture_top_b200 import moe
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, C * (2 if swiglu else 1), generator=g, device="cuda").to(dtype)
    src = torch.randint(-1, T + 1, (R,), generator=g, dtype=torch.int32, device="cuda")
    n = R - R // 5
    used = torch.tensor([n], dtype=torch.int32, device="cuda")
    ld = -(-C // 16) * 16 + 16

    def gather(stream=None):
        store = torch.full((R, ld), 1.5, device="cuda").to(E4M3)
        scales = torch.full((-(-C // 128), R + 3), 9.0, device="cuda")[:, :R]
        torch.cuda.synchronize()
        moe.fp8_quantize_rows(x, row_src=src, rows_used=used, swiglu=swiglu, codes=store[:, :C], scales=scales,
                              stream=stream)
        torch.cuda.synchronize()
        return store, scales
    moe.moe_profile_enable(True)
    store, scales = gather()
    names = [r[0] for r in moe.moe_profile_records()]
    moe.moe_profile_enable(False)
    assert names == ["fp8_quantize_rows", "fp8_gather_codes"]
    step = min(6 * T - 1, (1 << 24) // C)
    parts = [moe.fp8_quantize_rows(x, row_src=src[r:min(n, r + step)].contiguous(), swiglu=swiglu)
             for r in range(0, n, step)]
    codes = torch.cat([p[0].contiguous().view(torch.uint8) for p in parts])
    assert torch.equal(store[:n, :C].contiguous().view(torch.uint8), codes)
    assert torch.equal(scales[:, :n], torch.cat([p[1] for p in parts], 1))
    assert torch.all(store[n:].float() == 1.5) and torch.all(store[:, C:].float() == 1.5)
    assert torch.all(scales[:, n:] == 9.0)
    side = torch.cuda.Stream()
    store2, scales2 = gather(side)
    assert torch.equal(store2.view(torch.uint8), store.view(torch.uint8)) and torch.equal(scales2, scales)
