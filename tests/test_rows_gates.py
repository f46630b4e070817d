"""Which routings have a gate gradient per choice: those whose pairs are the
kept choices.  Token rounding makes other pairs, in expert order."""
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
