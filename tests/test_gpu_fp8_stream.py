"""MoELayer.forward_fp8 on a stream given by name: its buffers belong to that
stream from the first call on, and the result is that of the current stream."""
import pytest

torch = pytest.importorskip("torch")


def streams_of(tensors):
    """The streams whose allocations hold these tensors."""
    found = set()
    for t in tensors:
        p = t.data_ptr()
        found |= {seg["stream"] for seg in torch.cuda.memory_snapshot()
                  if seg["address"] <= p < seg["address"] + seg["total_size"]}
    return found


@pytest.mark.gpu
def test_forward_fp8_on_a_given_stream():
    from fine_grained_mixture_top_b200 import moe
    from workloads import MoEConfig, make_inputs
    cfg = MoEConfig("fp8_stream", T=1000, d=512, E=12, n=128, K=3, w_std=0.05, seed=75)
    inp = make_inputs(cfg, "cuda")

    def layer():
        m = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, seed=cfg.seed)
        m.route(inp["X"], inp["Wr"], inp["bias"])
        return m, m.quantize_weights_fp8(inp["W1"], inp["W2"])
    m, wq = layer()
    ref, refH = m.forward_fp8(inp["X"], wq).clone(), m.H.clone()
    used = int(m.routing["offsets"][-1])
    assert streams_of(m.ws_fp8.values()) == {torch.cuda.current_stream().cuda_stream}
    m, wq = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        junk = torch.full((1 << 24,), 1, device="cuda")   # the current stream goes on taking and freeing memory
        O = m.forward_fp8(inp["X"], wq, stream=side)
        del junk
    assert streams_of(m.ws_fp8.values()) == {side.cuda_stream}
    side.synchronize()
    assert torch.equal(O, ref) and torch.equal(m.H[:used], refH[:used])
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    other = torch.empty_like(ref)
    assert m.forward_fp8(inp["X"], wq, stream=side, O=other).data_ptr() == other.data_ptr()
    side.synchronize()
    assert torch.equal(other, ref)
    # captured on a stream of its own, replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward_fp8(inp["X"], wq, O=other)
    other.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, ref)
    assert moe.moe_get_status()[0] == 0
    del graph


@pytest.mark.gpu
def test_mxfp8_workspaces_on_a_given_stream():
    from fine_grained_mixture_top_b200 import moe
    from workloads import MoEConfig, make_inputs
    cfg = MoEConfig("mx_stream", T=500, d=256, E=8, n=128, K=2, w_std=0.05, seed=76)
    inp = make_inputs(cfg, "cuda")

    def layer():
        m = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, seed=cfg.seed)
        m.route(inp["X"], inp["Wr"], inp["bias"])
        return m
    m = layer()
    ref = m.forward(inp["X"], inp["W1"], inp["W2"], mxfp8=True).clone()
    assert streams_of([m.ws_fwd_mx]) == {torch.cuda.current_stream().cuda_stream}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    m = layer()
    torch.cuda.synchronize()
    O = m.forward(inp["X"], inp["W1"], inp["W2"], mxfp8=True, stream=side)
    side.synchronize()
    assert streams_of([m.ws_fwd_mx]) == {side.cuda_stream} and torch.equal(O, ref)
    m = layer()
    torch.cuda.synchronize()
    wq = m.quantize_weights_mxfp8(inp["W1"], inp["W2"], stream=side)
    O = m.forward_mxfp8_q(inp["X"], wq, stream=side)
    side.synchronize()
    assert streams_of([wq, m.ws_fwd_mx]) == {side.cuda_stream} and torch.equal(O, ref)
