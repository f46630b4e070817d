"""E4M3 quantization per block of 128 and the products of such codes.

Quantization is compared bit for bit with the same fp32 arithmetic on the CPU
(one division per block, one product and one rounding per value).

Products: C is rounded once to bf16, off by at most 2^-8 |C|.  Before that, a
block of 128 products is summed by the tensor core, 32 at a time, aligned to
the largest term with at least 13 bits below its leading one; each of the 33
addends of a step loses less than 2^-13 of the largest, and on random codes the
largest of 32 terms is under a quarter of the sum of their magnitudes, so a
step loses less than 33 / 4 * 2^-13 < 2^-9 of that sum.  The fp32 sums over the
blocks add at most 2^-24 per block, negligible here.  Scales differ from block
to block by factors of two and more, so a misplaced one is far outside."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -110


def up(x, m):
    return -(-x // m) * m


def ref_blocks(x, br, bc):
    """Codes (uint8) and scales of x [R, C] (fp32, CPU) in br x bc blocks."""
    R, C = x.shape
    t = torch.zeros(up(R, br), up(C, bc))
    t[:R, :C] = x
    t = t.view(t.shape[0] // br, br, t.shape[1] // bc, bc)
    amax = torch.nan_to_num(t.abs(), nan=0.0, posinf=float("inf")).amax((1, 3), keepdim=True).clamp_min(FLOOR)
    # one division: `448.0 / tensor` is a reciprocal and a product, rounded twice
    q = (t * (torch.full_like(amax, 448.0) / amax)).to(E4M3).view(torch.uint8)
    return q.reshape(up(R, br), up(C, bc))[:R, :C].contiguous(), (amax / torch.full_like(amax, 448.0))[:, 0, :, 0]


def same(got, want):
    np.testing.assert_array_equal(got.contiguous().view(torch.uint8).cpu().numpy(), want.numpy())


def data(R, C, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-6, 7, (R, 1), generator=g).float())
    if R > 2 and C > 3:
        x[1] = 0.0
        x[0, 1] = -0.0
        x[2, 3] = 1e-30 if dt != torch.float16 else 1e-7
    return x.to(dt)


SHAPES = [(1, 1), (1, 128), (3, 127), (7, 129), (128, 64), (130, 200), (257, 1000), (300, 2048), (5, 7168), (64, 333)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,C", SHAPES)
def test_quantize_rows_and_cols(R, C, dtype):
    from fine_grained_mixture_top_b200 import moe
    x = data(R, C, DTYPES[dtype], R + C)
    q, s = moe.fp8_quantize_rows(x.cuda())
    cq, cs = ref_blocks(x.float(), 1, 128)
    assert q.shape == (R, C) and s.shape == (-(-C // 128), R)
    same(q, cq)
    assert torch.equal(s.cpu(), cs.t())
    q, s = moe.fp8_quantize_cols(x.cuda())
    cq, cs = ref_blocks(x.float(), 128, 1)
    assert q.shape == (C, R) and s.shape == (-(-R // 128), C)
    same(q, cq.t())
    assert torch.equal(s.cpu(), cs)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (3, 128, 128), (2, 130, 257), (5, 64, 1000), (2, 300, 72)])
def test_quantize_blocks(E, K, N, dtype):
    from fine_grained_mixture_top_b200 import moe
    w = torch.stack([data(K, N, DTYPES[dtype], e) for e in range(E)])
    for tr in (False, True):
        q, s = moe.fp8_quantize_blocks(w.cuda(), transpose=tr)
        for e in range(E):
            cq, cs = ref_blocks(w[e].float(), 128, 128)
            same(q[e], cq.t() if tr else cq)
            assert torch.equal(s[e].cpu(), cs.t() if tr else cs)
    q2, s2 = moe.fp8_quantize_blocks(w[0].cuda(), transpose=True)      # a single weight
    q3, s3 = moe.fp8_quantize_blocks(w[:1].cuda(), transpose=True)
    assert torch.equal(q2.view(torch.uint8), q3[0].view(torch.uint8)) and torch.equal(s2, s3[0])


@pytest.mark.gpu
def test_gathered_rows_strides_and_what_is_left_alone():
    from fine_grained_mixture_top_b200 import moe
    T, C, R = 50, 200, 384
    for dt, off in ((torch.bfloat16, 0), (torch.bfloat16, 3), (torch.float32, 1)):
        base = data(T, C + 8, dt, 3).cuda()
        x = base[:, off:off + C]
        src = torch.randint(-1, T, (R,), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
        used = torch.tensor([256], dtype=torch.int32, device="cuda")
        want = torch.where((src >= 0)[:, None], x.cpu().float()[src.clamp_min(0).long()], torch.zeros(()))[:256]
        store = torch.full((R, up(C, 16) + 16), 1.5, device="cuda").to(E4M3)
        codes, scales = store[:, :C], torch.full((2, R + 5), 9.0, device="cuda")[:, :R]
        moe.fp8_quantize_rows(x, row_src=src.cuda(), rows_used=used, codes=codes, scales=scales)
        cq, cs = ref_blocks(want, 1, 128)
        same(codes[:256], cq)
        assert torch.equal(scales[:, :256].cpu(), cs.t())
        assert torch.all(store[256:].float() == 1.5) and torch.all(store[:, C:].float() == 1.5)
        assert torch.all(scales[:, 256:] == 9.0)
        store = torch.full((C, R), 1.5, device="cuda").to(E4M3)
        scales = torch.full((3, C), 9.0, device="cuda")
        moe.fp8_quantize_cols(x, row_src=src.cuda(), rows_used=used, codes=store, scales=scales)
        cq, cs = ref_blocks(want, 128, 1)
        same(store[:, :256], cq.t())
        assert torch.equal(scales[:2].cpu(), cs)
        assert torch.all(store[:, 256:].float() == 1.5) and torch.all(scales[2] == 9.0)


@pytest.mark.gpu
def test_a_source_row_that_is_none_gives_zeros():
    from fine_grained_mixture_top_b200 import moe
    x = torch.randn(5, 160, device="cuda")
    src = torch.tensor([4, 5, -1, 2 ** 31 - 1, -2 ** 31, 0, 1000000], dtype=torch.int32)
    want = torch.where(((src >= 0) & (src < 5))[:, None], x.cpu()[src.clamp(0, 4).long()], torch.zeros(()))
    q, s = moe.fp8_quantize_rows(x, row_src=src.cuda())
    cq, cs = ref_blocks(want, 1, 128)
    same(q, cq)
    assert torch.equal(s.cpu(), cs.t())
    q, s = moe.fp8_quantize_cols(x, row_src=src.cuda())
    cq, cs = ref_blocks(want, 128, 1)
    same(q, cq.t())
    assert torch.equal(s.cpu(), cs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,R,swiglu", [(1, 16, 7, False), (9, 130, 300, False), (50, 1000, 384, True),
                                          (33, 4100, 129, False), (20, 8192, 200, False)])
def test_repeated_rows_are_the_same_either_way(T, C, R, swiglu):
    """A gather that repeats rows quantizes each once and copies the codes: the
    same bits as row by row (a gather of fewer rows than twice the input's)."""
    from fine_grained_mixture_top_b200 import moe
    x = data(T, C * (2 if swiglu else 1), torch.bfloat16, T).clamp_(-30, 30).cuda()
    src = torch.randint(-1, T, (R,), dtype=torch.int32, generator=torch.Generator().manual_seed(T)).cuda()
    used = torch.tensor([R - R // 4], dtype=torch.int32, device="cuda")
    store = torch.full((R, up(C, 16) + 16), 1.5, device="cuda").to(E4M3)
    scales = torch.full((-(-C // 128), R), 9.0, device="cuda")
    moe.fp8_quantize_rows(x, row_src=src, rows_used=used, swiglu=swiglu, codes=store[:, :C], scales=scales)
    n = int(used)
    one, parts = max(1, 2 * T - 1), []
    for r in range(0, n, one):
        parts.append(moe.fp8_quantize_rows(x, row_src=src[r:min(n, r + one)].contiguous(), swiglu=swiglu))
    assert torch.equal(store[:n, :C].contiguous().view(torch.uint8), torch.cat([p[0].contiguous().view(torch.uint8) for p in parts]))
    assert torch.equal(scales[:, :n], torch.cat([p[1] for p in parts], 1))
    assert torch.all(store[n:].float() == 1.5) and torch.all(store[:, C:].float() == 1.5)
    assert torch.all(scales[:, n:] == 9.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,R,swiglu", [(1, 16, 7, False), (9, 130, 300, False), (50, 1000, 384, True), (7, 33, 7, False),
                                          (33, 4100, 129, False), (20, 8192, 200, False), (3, 7168, 2600, False)])
def test_repeated_rows_with_a_workspace(T, C, R, swiglu):
    """The workspace makes a gather quantize each row once: the same bits as without."""
    from fine_grained_mixture_top_b200 import moe
    x = data(T, C * (2 if swiglu else 1), torch.bfloat16, T).clamp_(-30, 30).cuda()
    src = torch.randint(-1, T + 1, (R,), dtype=torch.int32, generator=torch.Generator().manual_seed(T)).cuda()
    used = torch.tensor([R - R // 4], dtype=torch.int32, device="cuda")
    need = moe.lib().moe_fp8_gather_ws(T, C)
    got = []
    for n in (0, need):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        codes = torch.full((R, up(C, 16) + 16), 1.5, device="cuda").to(E4M3)
        scales = torch.full((-(-C // 128), R), 9.0, device="cuda")
        moe._check(moe.lib().moe_fp8_quantize_rows(
            0, moe._ptr(x), x.shape[1], T, R, C, moe._ptr(src), moe._ptr(used), 1 if swiglu else 0, moe._ptr(codes),
            codes.shape[1], moe._ptr(scales), R, moe._ptr(ws) if n else None, n, moe._current(x.device)), "rows")
        got.append((codes.view(torch.uint8), scales))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.gpu
def test_rows_past_32_bits_of_elements():
    """Row tensors of more than 2^31 elements: the first, some in between and the
    last rows of the gather, the quantizer, a product and the weighted sum."""
    from fine_grained_mixture_top_b200 import moe
    T, E, K, d = 42000, 3, 1, 64
    W = 52224                     # 42000 x 52224 > 2^31 elements
    idx = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda")
    rt = moe.sort_pairs(idx, torch.ones(T, K, device="cuda"), E)
    R = rt.struct.R_max
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    x[:, ::1000] = torch.randn(T, 1, device="cuda").bfloat16()
    x[:, -1] = 3.0
    rows = moe.permute(rt, x)
    tok = rt["row_tok"].long()
    real = (tok >= 0).nonzero()[:, 0]
    pick = real[torch.linspace(0, real.numel() - 1, 9).long().cuda()]
    assert torch.equal(rows[pick], x[tok[pick]])
    out = moe.unpermute(rt, rows)
    assert torch.equal(out[-5:], x[-5:]) and torch.equal(out[:5], x[:5])
    del out
    q, s = moe.fp8_quantize_rows(x, row_src=rt["row_tok"], rows_used=rt["offsets"][-1:])
    cq, cs = ref_blocks(x[tok[pick]].float().cpu(), 1, 128)
    same(q[pick], cq)
    assert torch.equal(s[:, pick].cpu(), cs.t())
    del x, rows
    b, sb = rand_codes((E, 72, W), 3), rand_scales((E, 1, W // 128), 4)
    y = moe.fp8_gemm(q, s, b, sb, routing=rt)
    del q
    e = int(rt["tile_expert"][int(pick[-1]) // 128])
    a = cq.cuda().view(E4M3)[-1:]
    check(y[pick[-1:]], *block_sum(a, cs.t()[:, -1:].cuda(), b[e], by_col(sb[e], 72)))
    a, sa = rand_codes((R, d), 5), rand_scales((1, R), 6)
    b, sb = rand_codes((E, W - 3, d), 7), rand_scales((E, W // 128, 1), 8)
    y = moe.fp8_gemm(a, sa, b, sb, routing=rt)      # more than 2^31 elements of C, ragged columns
    assert y.shape[0] * y.stride(0) > 2 ** 31
    for r in (int(pick[0]), int(pick[-1])):
        e = int(rt["tile_expert"][r // 128])
        check(y[r:r + 1], *block_sum(a[r:r + 1], sa[:, r:r + 1], b[e], by_col(sb[e], W - 3)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("R,C", [(3, 128), (70, 200), (33, 77), (129, 1024)])
def test_swiglu_then_quantize(R, C, dtype):
    """silu(g) u in fp32 is within 2^-18 of the value (exp 2^-21 relative at
    these arguments, a quotient and two products), so each code is one of the
    two E4M3 values around x / scale, or the nearest one up to that error."""
    from fine_grained_mixture_top_b200 import moe
    h = data(R, 2 * C, DTYPES[dtype], R).clamp_(-30, 30)
    q, s = moe.fp8_quantize_rows(h.cuda(), swiglu=True)
    g, u = h[:, :C].double(), h[:, C:].double()
    x = g / (1 + torch.exp(-g)) * u
    pad = torch.zeros(R, up(C, 128), dtype=torch.float64)
    pad[:, :C] = x
    amax = pad.view(R, -1, 128).abs().amax(2).clamp_min(FLOOR)
    sc = s.double().cpu().t()
    assert torch.all((sc - amax / 448).abs() <= 2.0 ** -18 * amax / 448)
    y = x / sc.repeat_interleave(128, 1)[:, :C]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
    assert torch.all((q.float().double().cpu() - y).abs() <= step / 2 + 2.0 ** -17 * y.abs())


@pytest.mark.gpu
def test_nan_and_infinity():
    from fine_grained_mixture_top_b200 import moe
    x = torch.randn(4, 256, device="cuda")
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    q, s = moe.fp8_quantize_rows(x)
    v = q.float()
    assert torch.isnan(v[1, 5]) and int(torch.isnan(v).sum()) == 2     # the infinity's own code: inf * 0
    assert torch.isinf(s[1, 2]) and torch.isfinite(s).sum() == 7
    clean, cs = moe.fp8_quantize_rows(torch.nan_to_num(x, nan=0.0, posinf=0.0))
    same(q[0], clean[0].view(torch.uint8).cpu())
    same(q[3], clean[3].view(torch.uint8).cpu())
    b, sb = moe.fp8_quantize_blocks(torch.randn(256, 32, device="cuda"), transpose=True)
    out = moe.fp8_gemm(q, s, b, sb)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all() and torch.isfinite(out[[0, 3]]).all()


# ----------------------------------------------------------------- products
def rand_codes(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape[-2:]
    store = torch.zeros(*shape[:-1], up(cols, 16), dtype=E4M3, device="cuda")
    store[..., :cols] = (torch.randn(shape, generator=g, device="cuda") * 60).clamp_(-448, 448).to(E4M3)
    return store[..., :cols]


def rand_scales(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp2(torch.randint(-3, 4, shape, generator=g, device="cuda").float()) * (
        1 + torch.rand(shape, generator=g, device="cuda"))


def block_sum(a, sa, b, sb):
    """In 64 bits: the product and the sum of its terms' magnitudes; sb [blocks, N]."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for i in range(-(-a.shape[1] // 128)):
        k = slice(128 * i, 128 * i + 128)
        f = sa[i].double()[:, None] * sb[i].double()[None, :]
        x, y = a[:, k].float().double(), b[:, k].float().double()
        out += (x @ y.t()) * f
        mag += (x.abs() @ y.abs().t()) * f
    return out, mag


def check(got, ref, mag, what=""):
    err = (got.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -9 * mag
    assert torch.isfinite(got.float()).all(), what
    assert torch.all(err <= tol), (what, float((err - tol).max()), float((err / mag.clamp_min(1e-300)).max()))


def by_col(sb, N):
    return sb.t().repeat_interleave(128, 1)[:, :N]


DENSE = [(1, 1, 1), (1, 8, 16), (2, 136, 128), (128, 128, 128), (129, 130, 131), (16, 512, 7168), (300, 1000, 257),
         (1, 4096, 2000), (64, 72, 4096), (1000, 264, 640), (40, 2100, 1100), (2500, 520, 384), (33, 129, 8192),
         (700, 700, 700), (257, 257, 129), (4100, 2056, 256),
         # either side of a tile of 128 x 128 per SM
         (16, 16392, 300), (128, 18944, 128), (600, 3700, 129), (600, 3850, 129), (1280, 2040, 131), (257, 8200, 640)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_product(M, N, K):
    from fine_grained_mixture_top_b200 import moe
    a, b = rand_codes((M, K), M), rand_codes((N, K), N + 1)
    kb = -(-K // 128)
    sa, sb = rand_scales((kb, M), 3), rand_scales((-(-N // 128), kb), 4)
    out = moe.fp8_gemm(a, sa, b, sb)
    ref, mag = block_sum(a, sa, b, by_col(sb, N))
    check(out, ref, mag)
    wide = torch.full((M + 2, up(N, 8) + 16), 7.0, dtype=torch.bfloat16, device="cuda")   # into a larger tensor
    sa_wide = torch.full((kb, M + 3), float("nan"), device="cuda")
    sa_wide[:, :M] = sa
    moe.fp8_gemm(a, sa_wide[:, :M], b, sb, out=wide[:M, :N])
    assert torch.equal(wide[:M, :N].view(torch.int16), out.view(torch.int16))
    assert torch.all(wide[M:] == 7) and torch.all(wide[:, N:] == 7)
    assert moe.moe_get_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 40, 1), (40, 70, 129), (300, 600, 250), (5000, 1000, 131), (2500, 2500, 7)])
def test_bytes_between_rows_count_for_nothing(M, N, K):
    """Row strides are multiples of 16: what lies between a row's end and the next
    row (here the NaN code) is not part of the product."""
    from fine_grained_mixture_top_b200 import moe

    def padded(rows, seed):
        t = torch.full((rows, up(K, 16) + 16), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)[:, :K]
        t.copy_(rand_codes((rows, K), seed))
        return t
    a, b = padded(M, 1), padded(N, 2)
    kb = -(-K // 128)
    sa, sb = rand_scales((kb, M), 3), rand_scales((-(-N // 128), kb), 4)
    check(moe.fp8_gemm(a, sa, b, sb), *block_sum(a, sa, b, by_col(sb, N)))
    sa, sb = rand_scales((kb, M), 5), rand_scales((kb, N), 6)
    check(moe.fp8_gemm_dw(a, sa, b, sb), *block_sum(a, sa, b, sb))
    x = torch.randn(M, K, device="cuda")
    q, s = moe.fp8_quantize_rows(x)      # the quantizer's own padding is left as it was allocated
    y = moe.fp8_gemm(q, s, b, sb := rand_scales((-(-N // 128), kb), 7))
    check(y, *block_sum(q, s, b, by_col(sb, N)))


GROUPED = [  # T, E, K, N, width, drop
    (1, 4, 1, 8, 16, 0.0), (5, 64, 4, 136, 128, 0.0), (300, 7, 3, 520, 640, 0.3), (2000, 5, 2, 264, 1000, 0.0),
    (130, 3, 2, 1000, 129, 0.9), (700, 16, 6, 384, 256, 0.1), (60, 9, 2, 72, 300, 1.0), (3000, 2, 1, 1544, 520, 0.0),
]


def routing(T, E, K, drop, seed):
    from fine_grained_mixture_top_b200 import moe
    rs = np.random.RandomState(seed)
    idx = np.argsort(rs.rand(T, E) - 0.5 * (np.arange(E) < 2), axis=1)[:, :K].astype(np.int32)
    idx[rs.rand(T, K) < drop] = -1
    return moe.sort_pairs(torch.from_numpy(idx).cuda(), torch.from_numpy(rs.rand(T, K).astype(np.float32)).cuda(), E)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,N,width,drop", GROUPED)
def test_grouped_product(T, E, K, N, width, drop):
    from fine_grained_mixture_top_b200 import moe
    rt = routing(T, E, K, drop, T)
    R, off = rt.struct.R_max, rt["offsets"].cpu().tolist()
    a, b = rand_codes((R, width), 5), rand_codes((E, N, width), 6)
    kb = -(-width // 128)
    sa, sb = rand_scales((kb, R), 7), rand_scales((E, -(-N // 128), kb), 8)
    out = torch.full((R, up(N, 8)), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.fp8_gemm(a, sa, b, sb, routing=rt, out=out[:, :N])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            check(out[lo:hi, :N], *block_sum(a[lo:hi], sa[:, lo:hi], b[e], by_col(sb[e], N)), e)
    assert torch.all(out[off[-1]:] == 7) and torch.all(out[:, N:] == 7)
    assert moe.moe_get_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,N,width,drop", GROUPED)
def test_weight_gradient_product(T, E, K, N, width, drop):
    from fine_grained_mixture_top_b200 import moe
    rt = routing(T, E, K, drop, T + 1)
    R, off = rt.struct.R_max, rt["offsets"].cpu().tolist()
    a, b = rand_codes((width, R), 9), rand_codes((N, R), 10)
    sa, sb = rand_scales((R // 128, width), 11), rand_scales((R // 128, N), 12)
    out = torch.full((E, width, up(N, 8)), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.fp8_gemm_dw(a, sa, b, sb, routing=rt, out=out[:, :, :N])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        t = slice(lo // 128, hi // 128)
        check(out[e, :, :N], *block_sum(a[:, lo:hi], sa[t], b[:, lo:hi], sb[t]), e)
        if lo == hi:
            assert torch.all(out[e, :, :N] == 0)
    assert torch.all(out[:, :, N:] == 7)
    assert moe.moe_get_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(8, 8, 1), (130, 136, 257), (512, 264, 1000)])
def test_dense_weight_gradient(M, N, K):
    from fine_grained_mixture_top_b200 import moe
    a, b = rand_codes((M, K), 1), rand_codes((N, K), 2)
    kb = -(-K // 128)
    sa, sb = rand_scales((kb, M), 3), rand_scales((kb, N), 4)
    check(moe.fp8_gemm_dw(a, sa, b, sb), *block_sum(a, sa, b, sb))


@pytest.mark.gpu
def test_no_tokens():
    from fine_grained_mixture_top_b200 import moe
    rt = routing(0, 3, 2, 0.0, 0)
    b, sb = rand_codes((3, 40, 64), 1), rand_scales((3, 1, 1), 2)
    a, sa = moe.fp8_quantize_rows(torch.zeros(0, 64, device="cuda"))
    assert moe.fp8_gemm(a, sa, b, sb, routing=rt).shape == (0, 40)
    assert moe.fp8_gemm(a, sa, b[0], sb[0]).shape == (0, 40)
    at, sat = moe.fp8_quantize_cols(torch.zeros(0, 64, device="cuda"))
    bt, sbt = moe.fp8_quantize_cols(torch.zeros(0, 40, device="cuda"))
    out = torch.full((3, 64, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.fp8_gemm_dw(at, sat, bt, sbt, routing=rt, out=out[:, :, :40])
    assert torch.all(out[:, :, :40] == 0) and torch.all(out[:, :, 40:] == 7)


@pytest.mark.gpu
def test_the_three_products_of_a_linear_layer():
    """y = x w, dx = dy w^T, dw = x^T dy from quantized operands against the
    unquantized product in 64 bits and against differences.  Each operand is
    within 2^-4 relative of its value (normal codes) or 2^-10 of its block's
    largest, errors of both signs: sums of hundreds of products are within
    2^-4 of the norm."""
    from fine_grained_mixture_top_b200 import moe
    M, K, N = 384, 256, 320
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda") for s in ((M, K), (K, N), (M, N)))
    y = moe.fp8_gemm(*moe.fp8_quantize_rows(x), *moe.fp8_quantize_blocks(w, transpose=True))
    dx = moe.fp8_gemm(*moe.fp8_quantize_rows(dy), *moe.fp8_quantize_blocks(w, transpose=False))
    dw = moe.fp8_gemm_dw(*moe.fp8_quantize_cols(x), *moe.fp8_quantize_cols(dy))
    x, w, dy = x.double(), w.double(), dy.double()
    for got, ref in ((y, x @ w), (dx, dy @ w.t()), (dw, x.t() @ dy)):
        assert got.shape == ref.shape
        assert float((got.double() - ref).norm() / ref.norm()) < 2.0 ** -4
    # directional differences of L = <x w, dy>, which is bilinear
    u, v = torch.randn(M, K, generator=g, device="cuda").double(), torch.randn(K, N, generator=g, device="cuda").double()
    h = 1e-3
    num = ((((x + h * u) @ w - (x - h * u) @ w) * dy).sum() / (2 * h), ((x @ (w + h * v) - x @ (w - h * v)) * dy).sum() / (2 * h))
    assert abs(float((dx.double() * u).sum() - num[0])) < 2.0 ** -4 * float((dy @ w.t()).norm() * 4)
    assert abs(float((dw.double() * v).sum() - num[1])) < 2.0 ** -4 * float((x.t() @ dy).norm() * 4)


@pytest.mark.gpu
def test_same_bits_again_captured_and_on_another_stream():
    from fine_grained_mixture_top_b200 import moe
    rt = routing(900, 6, 2, 0.1, 4)
    R = rt.struct.R_max
    x = torch.randn(900, 640, device="cuda").bfloat16()
    b, sb = rand_codes((6, 392, 640), 6), rand_scales((6, 4, 5), 8)
    used = rt["offsets"][-1:]

    def run(out):
        a, sa = moe.fp8_quantize_rows(x, row_src=rt["row_tok"], rows_used=used)
        return moe.fp8_gemm(a, sa, b, sb, routing=rt, out=out)
    outs = [torch.zeros(R, 392, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    run(outs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(outs[1])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2])
    outs[2].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert float(outs[0].abs().max()) > 0
    del graph
