"""The workspace that a caller gives to sort_pairs is checked whether or not a
routing comes with it, on the host, before its address goes anywhere."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    from fine_grained_mixture_top_b200 import build
    build.build()
    from fine_grained_mixture_top_b200 import moe as m
    return m


@pytest.mark.parametrize("with_routing", [False, True])
def test_workspace(moe, with_routing):
    idx, gate = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    rt = moe.Routing({}, moe.MoeRouting()) if with_routing else None
    for ws in (torch.zeros(4096, dtype=torch.float16), torch.zeros(1, dtype=torch.uint8).expand(4096),
               torch.zeros(8192, dtype=torch.uint8)[::2], torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="ws"):
            moe.sort_pairs(idx, gate, 8, routing=rt, ws=ws)
    with pytest.raises(ValueError, match="CUDA device"):      # a proper one: refused for the device alone
        moe.sort_pairs(idx, gate, 8, routing=rt, ws=torch.zeros(4096, dtype=torch.uint8))


@pytest.mark.gpu
def test_workspace_on_another_device():
    from fine_grained_mixture_top_b200 import moe
    idx, gate = torch.zeros(4000, 2, dtype=torch.int32, device="cuda"), torch.zeros(4000, 2, device="cuda")
    with pytest.raises(ValueError, match="ws"):
        moe.sort_pairs(idx, gate, 8, ws=torch.zeros(1 << 20, dtype=torch.uint8))
    rt = moe.sort_pairs(idx, gate, 8, ws=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    assert int(rt["counts"][0]) == 8000
    with pytest.raises(moe.MoEError):                          # too small
        moe.sort_pairs(idx, gate, 8, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
