"""Products whose last columns end inside the first half of a 128-column strip
(N mod 128 between 1 and 63, N no multiple of 8), with many tiles per pair of
CTAs and little work between two stores: what a tile stages must not meet a
store of the tile before that is still under way.  Each is compared with the
sum in 64 bits (tolerances as derived in test_gpu_fp8.py), then repeated: a
fixed order of sums gives the same bits every time."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_fp8 import block_sum, by_col, check, rand_codes, rand_scales, up   # noqa: E402

REPEATS = 100


def repeats(call, out, what):
    first = out.clone()
    for _ in range(REPEATS):
        out.fill_(7.0)
        call()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), what


@pytest.mark.gpu
@pytest.mark.parametrize("K", [100, 256])
@pytest.mark.parametrize("N", [2305, 2307, 2313, 2367])
def test_dense(N, K):
    from fine_grained_mixture_top_b200 import moe
    M = 4003
    a, b = rand_codes((M, K), N), rand_codes((N, K), K)
    kb = -(-K // 128)
    sa, sb = rand_scales((kb, M), 1), rand_scales((-(-N // 128), kb), 2)
    out = torch.full((M, up(N, 8)), 7.0, dtype=torch.bfloat16, device="cuda")

    def call():
        moe.fp8_gemm(a, sa, b, sb, out=out[:, :N])
    call()
    check(out[:, :N], *block_sum(a, sa, b, by_col(sb, N)))
    assert torch.all(out[:, N:] == 7)
    repeats(call, out, (N, K))
    assert moe.moe_get_status() == (0, 0)


def tiles_per_expert(per):
    """A routing whose expert e has per[e] rows (one choice per token)."""
    from fine_grained_mixture_top_b200 import moe
    idx = torch.repeat_interleave(torch.arange(len(per)), torch.tensor(per)).to(torch.int32)[:, None].contiguous()
    return moe.sort_pairs(idx.cuda(), torch.ones(idx.shape, device="cuda"), len(per))


# rows per expert: none, one block, a few
PER = [[0, 128, 1, 0, 300, 0, 128, 77, 0, 0, 128, 256] * 3, [0, 0, 0, 513, 0, 0] + [0, 60] * 17]


@pytest.mark.gpu
@pytest.mark.parametrize("per", PER, ids=["mixed", "sparse"])
@pytest.mark.parametrize("N", [1281, 1283, 1289, 1343])
def test_grouped_and_weight_gradients(N, per):
    from fine_grained_mixture_top_b200 import moe
    rt = tiles_per_expert(per)
    E, R, off = len(per), rt.struct.R_max, rt["offsets"].cpu().tolist()
    width = 200
    a, b = rand_codes((R, width), 1), rand_codes((E, N, width), 2)
    sa, sb = rand_scales((2, R), 3), rand_scales((E, -(-N // 128), 2), 4)
    out = torch.full((R, up(N, 8)), 7.0, dtype=torch.bfloat16, device="cuda")

    def grouped():
        moe.fp8_gemm(a, sa, b, sb, routing=rt, out=out[:, :N])
    grouped()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            check(out[lo:hi, :N], *block_sum(a[lo:hi], sa[:, lo:hi], b[e], by_col(sb[e], N)), e)
    assert torch.all(out[off[-1]:] == 7) and torch.all(out[:, N:] == 7)
    repeats(grouped, out, ("grouped", N))

    M = 300
    a, b = rand_codes((M, R), 5), rand_codes((N, R), 6)
    sa, sb = rand_scales((R // 128, M), 7), rand_scales((R // 128, N), 8)
    dw = torch.full((E, M, up(N, 8)), 7.0, dtype=torch.bfloat16, device="cuda")

    def gradients():
        moe.fp8_gemm_dw(a, sa, b, sb, routing=rt, out=dw[:, :, :N])
    gradients()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            assert torch.all(dw[e, :, :N] == 0), e
        else:
            t = slice(lo // 128, hi // 128)
            check(dw[e, :, :N], *block_sum(a[:, lo:hi], sa[t], b[:, lo:hi], sb[t]), e)
    assert torch.all(dw[:, :, N:] == 7)
    repeats(gradients, dw, ("gradients", N))
    assert moe.moe_get_status() == (0, 0)
