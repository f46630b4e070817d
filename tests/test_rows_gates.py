"""Which routings have a gate gradient per choice: those whose pairs are the
kept choices.  Token rounding makes other pairs, in expert order."""
import ctypes
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    from fine_grained_mixture_top_b200 import build
    build.build()
    from fine_grained_mixture_top_b200 import moe as m
    return m


def test_rounding_is_told_by_the_call_that_rounds(moe, monkeypatch):
    """With K = E the pair capacities of rounding are those of the choices, so
    that they tell nothing (host only: the library's entries are stubs here)."""
    T = E = K = 4
    real = moe.lib()
    dims, opts = moe.dims_of(T, 128, E, 64, K), moe.opts_of(1)
    assert moe.query_sizes(dims, opts).P_max == T * K
    rt = moe.Routing({"tok_ptr": torch.zeros(T + 1), "counts": torch.zeros(E), "topk_idx": torch.zeros(T, K)},
                     moe.MoeRouting(P_max=T * K, R_max=512))
    x, rows, ws = torch.zeros(T, 16), torch.zeros(512, 16), torch.zeros(16, dtype=torch.uint8)
    stream = types.SimpleNamespace(cuda_stream=0)
    monkeypatch.setattr(moe, "_lib", types.SimpleNamespace(
        moe_route=lambda *a: 0, moe_token_round=lambda *a: 0, moe_route_given=lambda *a: 0, moe_route_noalloc=lambda *a: 0,
        moe_status_str=real.moe_status_str))
    with pytest.raises(ValueError, match="CUDA device"):      # accepted, up to the device
        moe.unpermute_bwd(rt, x, rows)
    moe.moe_route(dims, opts, x, x, None, rt, ws, stream=stream)
    moe.moe_token_round(dims, opts, rt, ws, stream=stream)
    with pytest.raises(ValueError, match="pairs=True"):
        moe.unpermute_bwd(rt, x, rows)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.unpermute_bwd(rt, x, rows, pairs=True)
    for again in (lambda: moe.moe_route(dims, opts, x, x, None, rt, ws, stream=stream),
                  lambda: moe.moe_route_noalloc(dims, opts, x, x, None, rt, stream=stream),
                  lambda: moe.moe_route_given(dims, opts, rt, ws, stream=stream)):
        moe.moe_token_round(dims, opts, rt, ws, stream=stream)
        again()
        with pytest.raises(ValueError, match="CUDA device"):
            moe.unpermute_bwd(rt, x, rows)


@pytest.mark.gpu
def test_gate_gradients_of_a_rounded_routing_over_all_experts():
    """T = 300, E = K = 4: refused per choice, right in pair order."""
    from fine_grained_mixture_top_b200 import moe
    from workloads import MoEConfig, make_inputs
    cfg = MoEConfig("round_all", T=300, d=128, E=4, n=64, K=4, w_std=0.05, bias="normal", seed=5, round_mode=1)
    inp = make_inputs(cfg, "cuda")
    layer = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, round_mode=1, seed=cfg.seed)
    layer.route(inp["X"], inp["Wr"], inp["bias"])
    rt = layer.routing
    assert rt.struct.P_max == cfg.T * cfg.K
    rows = moe.permute(rt, inp["X"])
    with pytest.raises(ValueError, match="pairs=True"):
        moe.unpermute_bwd(rt, inp["dO"], rows)
    _, dg = moe.unpermute_bwd(rt, inp["dO"], rows, pairs=True)
    P = int(rt["tok_ptr"][-1])
    pt = np.repeat(np.arange(cfg.T), np.diff(rt["tok_ptr"].cpu().numpy()))
    x, do = inp["X"].double().cpu().numpy(), inp["dO"].double().cpu().numpy()
    ref, mag = (do[pt] * x[pt]).sum(1), np.abs(do[pt] * x[pt]).sum(1)
    # cfg.d terms in fp32, a rounding per product and per sum
    assert np.all(np.abs(dg[:P].double().cpu().numpy() - ref) <= (cfg.d + 1) * 2.0 ** -24 * mag)


def choices(T, E, K, drop, seed):
    rs = np.random.RandomState(seed)
    idx = np.argsort(rs.rand(T, E), axis=1)[:, :K].astype(np.int32)
    idx[rs.rand(T, K) < drop] = -1
    return torch.from_numpy(idx).cuda(), torch.from_numpy(rs.rand(T, K).astype(np.float32)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,drop", [(1, 3, 2, 0.5), (700, 9, 4, 0.3), (5000, 40, 32, 0.2), (3000, 17, 1, 0.5),
                                        (513, 8, 8, 0.0), (300, 5, 3, 1.0)])
def test_gate_gradients_from_the_routing_alone(T, E, K, drop):
    """The caller's selection is another one by the time of the gradient."""
    from fine_grained_mixture_top_b200 import moe
    idx, gate = choices(T, E, K, drop, T)
    kept = (idx >= 0).clone()
    rt = moe.sort_pairs(idx, gate, E)
    pairs = int(rt["tok_ptr"][-1])
    slot = kept.nonzero()[:, 1].to(torch.int32)
    assert torch.equal(rt["pair_slot"][:pairs], slot) and torch.all(rt["pair_slot"][pairs:] == -1)
    x, do = torch.randn(T, 48, device="cuda"), torch.randn(T, 48, device="cuda")
    rows = moe.permute(rt, x)
    want = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    t, k = kept.nonzero(as_tuple=True)
    want[t, k] = (do[t].double() * x[t].double()).sum(1)
    mag[t, k] = (do[t].double() * x[t].double()).abs().sum(1)

    def right(dg):       # 48 terms in fp32, a rounding per product and per sum
        assert torch.all((dg.double() - want).abs() <= 49 * 2.0 ** -24 * mag)
    nan = lambda: torch.full((T, K), float("nan"), device="cuda")   # noqa: E731
    first = moe.unpermute_bwd(rt, do, rows, dgate=nan())[1]
    right(first)
    rt.struct.pair_slot = None       # a routing without places: from the selection, while it is there
    right(moe.unpermute_bwd(rt, do, rows, dgate=nan())[1])
    rt.struct.pair_slot = rt["pair_slot"].data_ptr()
    idx.copy_(choices(T, E, K, 0.6, T + 1)[0])
    gate.fill_(float("nan"))
    assert torch.equal(moe.unpermute_bwd(rt, do, rows, dgate=nan())[1], first)
    idx2, gate2 = choices(T, E, K, drop, T + 2)      # the same buffers for another selection
    kept2 = idx2 >= 0
    moe.sort_pairs(idx2, gate2, E, routing=rt)
    n = int(kept2.sum())
    assert torch.equal(rt["pair_slot"][:n], kept2.nonzero()[:, 1].to(torch.int32))
    assert torch.all(rt["pair_slot"][n:] == -1)


@pytest.mark.gpu
def test_gate_gradients_of_a_given_selection():
    """moe_route_given keeps every choice: its routing needs no selection either."""
    from fine_grained_mixture_top_b200 import moe
    T, E, K, d = 260, 6, 3, 128
    layer = moe.MoELayer(T, d, E, 64, K)
    idx, gate = choices(T, E, K, 0.0, 8)
    layer.routing["topk_idx"].copy_(idx)
    layer.routing["topk_gate"].copy_(gate)
    moe.moe_route_given(layer.dims, layer.opts, layer.routing, layer.ws_route)
    x, do = torch.randn(T, d, device="cuda"), torch.randn(T, d, device="cuda")
    rows = moe.permute(layer.routing, x)
    first = moe.unpermute_bwd(layer.routing, do, rows)[1]
    ref = (x.double() * do.double()).sum(1, keepdim=True).expand(T, K)
    assert torch.all((first.double() - ref).abs() <= (d + 1) * 2.0 ** -24 * (x * do).double().abs().sum(1, keepdim=True))
    layer.routing["topk_idx"].fill_(-1)
    dg = torch.full((T, K), float("nan"), device="cuda")
    assert torch.equal(moe.unpermute_bwd(layer.routing, do, rows, dgate=dg)[1], first)


def test_a_misaligned_place_array_is_refused(moe):
    st = moe.MoeRouting(**{k: 4096 for k in moe._ROUTING_PTRS}, P_max=8, R_max=1024, pair_slot=4100)
    ref = ctypes.byref(st)
    assert moe.lib().moe_sort_pairs(4, 8, 2, ref, None, 0, None) == 1
    assert moe.lib().moe_unpermute_bwd(4, 8, 2, ref, 0, 64, 4096, 64, 8192, 64, 16384, 64, None, 4096, None) == 1
