"""The layer's forward with 8-bit products (MoELayer.forward_fp8): routing, the
gathering quantizer, grouped products, SwiGLU quantizer and weighted sum run
together, against the same steps in 64 bits on the operands as quantized."""
import numpy as np
import pytest

from workloads import MoEConfig, make_inputs

import parity as P

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn

CFGS = [
    MoEConfig("fp8_small", T=300, d=256, E=8, n=128, K=2, w_std=0.05, bias="normal", seed=71),
    MoEConfig("fp8_ragged", T=1000, d=384, E=12, n=192, K=3, w_std=0.05, seed=72),
    MoEConfig("fp8_round", T=900, d=256, E=6, n=64, K=2, w_std=0.05, bias="normal", seed=73, round_mode=1),
    MoEConfig("fp8_one", T=1, d=128, E=5, n=64, K=3, w_std=0.05, seed=74),
]


def quantized(x, br, bc):
    """x [R, C] (64 bits) on its br x bc blocks' E4M3 grids."""
    R, C = x.shape
    t = torch.zeros(-(-R // br) * br, -(-C // bc) * bc)
    t[:R, :C] = x.float()
    t = t.view(t.shape[0] // br, br, t.shape[1] // bc, bc)
    amax = t.abs().amax((1, 3), keepdim=True).clamp_min(2.0 ** -110)
    f = torch.full_like(amax, 448.0)
    q = (t * (f / amax)).to(E4M3).double() * (amax / f).double()
    return q.reshape(q.shape[0] * br, -1)[:R, :C]


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", CFGS, ids=[c.name for c in CFGS])
def test_forward_fp8(cfg):
    from fine_grained_mixture_top_b200 import moe
    inp = make_inputs(cfg, "cuda")
    layer = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, round_mode=cfg.round_mode, seed=cfg.seed)
    layer.route(inp["X"], inp["Wr"], inp["bias"])
    wq = layer.quantize_weights_fp8(inp["W1"], inp["W2"])
    O = layer.forward_fp8(inp["X"], wq)
    assert O.data_ptr() == layer.O.data_ptr()
    torch.cuda.synchronize()
    assert moe.moe_get_status()[0] == 0
    rt = {k: v.cpu().long() if v.dtype == torch.int32 else v.cpu().double() for k, v in layer.routing.tensors.items()
          if v is not None}
    off, used = rt["offsets"], int(rt["offsets"][-1])
    X, H = inp["X"].double().cpu(), layer.H.double().cpu()
    tok = rt["row_tok"][:used]
    xq = torch.where((tok >= 0)[:, None], quantized(X, 1, 128)[tok.clamp_min(0)], torch.zeros((), dtype=torch.float64))
    Href, Y = torch.zeros(used, 2 * cfg.n, dtype=torch.float64), torch.zeros(used, cfg.d, dtype=torch.float64)
    g, u = H[:used, :cfg.n], H[:used, cfg.n:]          # the second half of the layer from the H it kept
    aq = quantized(g * torch.sigmoid(g) * u, 1, 128)
    for e in range(cfg.E):
        r = slice(int(off[e]), int(off[e + 1]))
        Href[r] = xq[r] @ quantized(inp["W1"][e].double().cpu(), 128, 128)
        Y[r] = aq[r] @ quantized(inp["W2"][e].double().cpu(), 128, 128)
    pairs = int(rt["tok_ptr"][-1])
    pt = torch.repeat_interleave(torch.arange(cfg.T), torch.diff(rt["tok_ptr"]))
    Oref = torch.zeros(cfg.T, cfg.d, dtype=torch.float64).index_add_(
        0, pt, Y[rt["pair_row"][:pairs]] * rt["pair_gate"][:pairs, None])
    # one rounding to bf16 (2^-8 at most, H), three of them with those of Y and O and a code that may fall to the
    # other side of a tie (O): normwise well below 2^-7
    for got, ref in ((H[:used], Href), (O.double().cpu(), Oref)):
        assert float((got - ref).norm() / ref.norm()) < 2.0 ** -7
    # and near the unquantized layer: each operand is within 2^-4 of its value
    layer2 = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, round_mode=cfg.round_mode, seed=cfg.seed)
    layer2.route(inp["X"], inp["Wr"], inp["bias"])
    full = layer2.forward(inp["X"], inp["W1"], inp["W2"]).double().cpu()
    assert float((O.double().cpu() - full).norm() / full.norm()) < 2.0 ** -3
    # the backward takes the H that was kept
    grads = layer.backward(inp["dO"], inp["X"], inp["Wr"], inp["W1"], inp["W2"])
    torch.cuda.synchronize()
    assert moe.moe_get_status()[0] == 0
    for x in grads:
        assert torch.isfinite(x.float()).all()


@pytest.mark.gpu
def test_an_expert_path_of_its_own_with_gradients():
    """Sorted rows through a two-layer expert of the caller's own in 8 bits, and
    all gradients back (rows, weights, gates, tokens), against the same chain in
    64 bits without quantization: every product is within a few percent."""
    from fine_grained_mixture_top_b200 import moe
    T, E, K, d, n = 700, 5, 2, 256, 192
    rs = np.random.RandomState(3)
    idx = np.argsort(rs.rand(T, E), axis=1)[:, :K].astype(np.int32)
    idx[rs.rand(T, K) < 0.1] = -1
    gate = rs.rand(T, K).astype(np.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dout = (torch.randn(T, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    W = (torch.randn(E, d, n, generator=g, device="cuda") * 0.05).bfloat16()
    V = (torch.randn(E, n, d, generator=g, device="cuda") * 0.05).bfloat16()
    rt = moe.sort_pairs(torch.from_numpy(idx).cuda(), torch.from_numpy(gate).cuda(), E)
    used = rt["offsets"][E:]
    rows = moe.permute(rt, x)

    def product(a, w, transpose):
        return moe.fp8_gemm(*moe.fp8_quantize_rows(a, rows_used=used), *moe.fp8_quantize_blocks(w, transpose=transpose),
                            routing=rt)
    h = product(rows, W, True)
    y = product(h, V, True)
    out = moe.unpermute(rt, y)
    dy, dgate = moe.unpermute_bwd(rt, dout, y)
    cols = lambda t: moe.fp8_quantize_cols(t, rows_used=used)   # noqa: E731
    dV = moe.fp8_gemm_dw(*cols(h), *cols(dy), routing=rt)
    dh = product(dy, V, False)
    dW = moe.fp8_gemm_dw(*cols(rows), *cols(dh), routing=rt)
    dx = moe.permute_bwd(rt, product(dh, W, False))
    torch.cuda.synchronize()
    assert moe.moe_get_status() == (0, 0)

    X = x.double().requires_grad_()
    Wd, Vd = W.double().requires_grad_(), V.double().requires_grad_()
    G = torch.from_numpy(gate).cuda().double().requires_grad_()
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (torch.from_numpy(idx).cuda() == e).nonzero(as_tuple=True)
        ref = ref.index_add(0, t, (X[t] @ Wd[e] @ Vd[e]) * G[t, k][:, None])
    ref.backward(dout.double())
    for name, got, want in (("out", out, ref), ("dx", dx, X.grad), ("dW", dW, Wd.grad), ("dV", dV, Vd.grad),
                            ("dgate", dgate, G.grad)):
        err = float((got.double() - want.detach()).norm() / want.detach().norm())
        # two products of operands within 2^-4 each (errors of both signs), and their gradients
        assert err < 2.0 ** -3, (name, err)
