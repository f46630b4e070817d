"""What the row movement refuses, on the host, before anything is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    from fine_grained_mixture_top_b200 import build
    build.build()
    from fine_grained_mixture_top_b200 import moe as m
    return m


def _sizes(moe, T, E, K):
    P, R, ws = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
    rc = moe.lib().moe_sort_sizes(T, E, K, ctypes.byref(P), ctypes.byref(R), ctypes.byref(ws))
    return rc, P.value, R.value, ws.value


def test_sort_sizes(moe):
    assert _sizes(moe, 0, 4, 2) == (0, 0, 0, 0)
    assert _sizes(moe, 1, 64, 8) == (0, 8, 1024, 0)        # 8 experts at most have a row: 8 tiles, one launch
    rc, P, R, ws = _sizes(moe, 16384, 128, 8)
    assert (rc, P, R) == (0, 131072, 131072 + 128 * 127 // 128 * 128)
    assert ws >= 4 * P
    for T, E, K, code in ((-1, 4, 2, 1), (4, 0, 2, 1), (4, 4, 0, 1), (4, 1025, 2, 2), (4, 64, 33, 2),
                          (1 << 27, 64, 16, 2)):
        assert _sizes(moe, T, E, K)[0] == code, (T, E, K)
    L = moe.lib()
    assert L.moe_sort_sizes(4, 4, 2, None, None, None) == 1


def _routing(moe, **kw):
    """A routing of made-up aligned addresses: nothing here dereferences them."""
    st = moe.MoeRouting(**{k: 4096 for k in moe._ROUTING_PTRS}, P_max=8, R_max=1024)
    for k, v in kw.items():
        setattr(st, k, v)
    return ctypes.byref(st)


def test_c_entries_refuse(moe):
    L = moe.lib()
    sort = lambda rt, T=4, E=8, K=2, ws=None, n=0: L.moe_sort_pairs(T, E, K, rt, ws, n, None)   # noqa: E731
    assert sort(None) == 1
    for name in ("topk_idx", "topk_gate", "tok_ptr", "pair_expert", "pair_gate", "pair_row", "counts", "offsets",
                 "row_tok", "row_gate", "tile_expert"):
        assert sort(_routing(moe, **{name: None})) == 1, name
    assert sort(_routing(moe, row_tok=4100)) == 1            # misaligned
    assert sort(_routing(moe, topk_idx=4098)) == 1
    assert sort(_routing(moe, P_max=7)) == 1 and sort(_routing(moe, R_max=1023)) == 1
    assert sort(_routing(moe, R_max=896)) == 1               # 8 experts with a row each need 8 tiles
    assert sort(_routing(moe), E=2000) == 2
    big = _routing(moe, P_max=20000, R_max=40064)
    assert sort(big, T=10000) == 3 and sort(big, T=10000, ws=4096, n=100) == 3
    assert sort(big, T=10000, ws=4100, n=1 << 30) == 1
    for fn in (L.moe_permute, L.moe_permute_bwd, L.moe_unpermute):
        call = lambda rt=None, T=4, E=8, type=0, width=64, a=4096, lda=64, b=8192, ldb=64: fn(   # noqa: E731
            T, E, _routing(moe) if rt is None else rt, type, width, a, lda, b, ldb, None)
        assert call(rt=_routing(moe, pair_row=None)) == 1
        assert call(type=7) == 1 and call(T=-1) == 1 and call(width=0) == 1
        assert call(E=0) == 2 and call(E=1025) == 2 and call(width=(1 << 20) + 1, lda=1 << 21, ldb=1 << 21) == 2
        assert call(a=None) == 1 and call(b=None) == 1
        assert call(lda=63) == 1 and call(ldb=63) == 1       # rows would overlap
        assert call(a=4097) == 1                             # not aligned to its elements
        assert call(T=0, a=None, b=None) == 0                # nothing to move
    assert L.moe_permute_bwd(4, 8, _routing(moe), 3, 64, 4096, 64, 8192, 64, None) == 2   # codes are not summed
    assert L.moe_unpermute(4, 8, _routing(moe), 3, 64, 4096, 64, 8192, 64, None) == 2
    bwd = lambda rt, K=2, type=0, d=4096, topk=4096: L.moe_unpermute_bwd(   # noqa: E731
        4, 8, K, rt, type, 64, d, 64, 8192, 64, 16384, 64, None, topk, None)
    assert bwd(_routing(moe), type=3) == 2 and bwd(_routing(moe), K=33) == 2
    assert bwd(_routing(moe), d=None) == 1 and bwd(_routing(moe, topk_idx=None)) == 1
    assert moe.last_error() == ""


def test_binding_refuses(moe):
    idx, gate = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.sort_pairs(idx, gate, 8)
    with pytest.raises(TypeError, match="topk_idx"):
        moe.sort_pairs(idx.long(), gate, 8)
    with pytest.raises(TypeError, match="topk_gate"):
        moe.sort_pairs(idx, gate.half(), 8)
    with pytest.raises(ValueError, match="topk_gate"):
        moe.sort_pairs(idx, gate[:3], 8)
    with pytest.raises(ValueError, match="contiguous"):
        moe.sort_pairs(torch.zeros(2, 4, dtype=torch.int32).t(), gate, 8)
    rt = moe.Routing({"tok_ptr": torch.zeros(5), "counts": torch.zeros(8), "topk_idx": idx},
                     moe.MoeRouting(P_max=8, R_max=1024))
    x = torch.zeros(4, 16)
    with pytest.raises(TypeError):
        moe.permute(rt, x.double())
    with pytest.raises(ValueError, match="src"):
        moe.permute(rt, x[:3])
    with pytest.raises(ValueError, match="contiguous"):
        moe.permute(rt, torch.zeros(16, 4).t())
    with pytest.raises(ValueError, match="overlap"):
        moe.permute(rt, torch.zeros(1, 16).expand(4, 16))
    with pytest.raises(ValueError, match="CUDA device"):
        moe.permute(rt, x)
    with pytest.raises(TypeError):
        moe.unpermute(rt, torch.zeros(1024, 16).to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="rows"):
        moe.unpermute(rt, torch.zeros(1000, 16))
    with pytest.raises(TypeError, match="dout"):
        moe.unpermute_bwd(rt, x.half(), torch.zeros(1024, 16))
    rows = torch.zeros(1024, 16)
    with pytest.raises(ValueError, match="must not be rows"):
        moe.unpermute_bwd(rt, x, rows, drows=rows)
    rt.struct.P_max = 8 + 127 * 8        # capacities of token rounding
    with pytest.raises(ValueError, match="pairs=True"):
        moe.unpermute_bwd(rt, x, rows)
