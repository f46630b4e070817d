"""Rows sorted by expert and back (moe_sort_pairs, moe_permute, moe_unpermute
and their gradients) against a plain computation in 64 bits.

Tolerances: an output is rounded once from an fp32 sum, so it is off by at most
eps/2 of the type relative to the value, plus the sum's own error, at most
n 2^-24 times the sum of the terms' magnitudes for n terms and one rounding per
product (sums here are at most 32 terms, or `width` terms for a gate gradient)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def selection(T, E, K, seed, drop=0.0, distinct=True):
    rs = np.random.RandomState(seed)
    if distinct:
        idx = np.argsort(rs.rand(T, E) - 2 * (rs.rand(E) < 0.2), axis=1)[:, :K].astype(np.int32)
    else:
        idx = rs.randint(0, E, (T, K)).astype(np.int32)
    gate = rs.rand(T, K).astype(np.float32)
    lost = rs.rand(T, K) < drop
    idx[lost] = rs.choice([-1, E, -2 ** 31, 2 ** 31 - 1], lost.sum())
    return idx, gate


def plain_sort(idx, gate, E, P_max, R_max):
    """The routing by counting, one choice after another."""
    T, K = idx.shape
    members = [[] for _ in range(E)]
    pairs = []
    tok_ptr = [0]
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if 0 <= e < E:
                members[e].append(len(pairs))
                pairs.append((t, e, gate[t, k]))
        tok_ptr.append(len(pairs))
    out = {"tok_ptr": np.array(tok_ptr), "counts": np.array([len(m) for m in members]),
           "pair_row": np.full(P_max, -1), "pair_expert": np.full(P_max, -1), "pair_gate": np.zeros(P_max, np.float32),
           "row_tok": np.full(R_max, -1), "row_gate": np.zeros(R_max, np.float32),
           "tile_expert": np.full(R_max // 128, -1), "offsets": np.zeros(E + 1, np.int64)}
    off = 0
    for e, m in enumerate(members):
        for i, p in enumerate(m):
            out["pair_row"][p], out["pair_expert"][p], out["pair_gate"][p] = off + i, e, pairs[p][2]
            out["row_tok"][off + i], out["row_gate"][off + i] = pairs[p][0], pairs[p][2]
        size = -(-len(m) // 128) * 128
        out["tile_expert"][off // 128:(off + size) // 128] = e
        off += size
        out["offsets"][e + 1] = off
    return out


def sorted_on_gpu(idx, gate, E, **kw):
    from fine_grained_mixture_top_b200 import moe
    return moe.sort_pairs(torch.from_numpy(idx).cuda(), torch.from_numpy(gate).cuda(), E, **kw)


def check_sort(rt, idx, gate, E):
    ref = plain_sort(idx, gate, E, rt.struct.P_max, rt.struct.R_max)
    for k, v in ref.items():
        np.testing.assert_array_equal(rt[k].cpu().numpy(), v, err_msg=k)
    return ref


SORTS = [  # T, E, K, drop, distinct
    (1, 1, 1, 0.0, True), (1, 64, 8, 0.0, True), (7, 5, 3, 0.5, True), (129, 3, 2, 0.0, True),
    (300, 1024, 32, 0.1, True), (256, 8, 32, 0.0, False),       # one chunk exactly full, experts chosen twice
    (8193, 17, 1, 0.0, False), (5000, 128, 8, 0.2, True), (4096, 1023, 5, 0.3, False), (20000, 2, 2, 0.0, True),
    (600, 40, 4, 1.0, True), (16385, 1, 1, 0.5, False),
    (2048, 9, 1, 0.1, False), (2049, 1024, 1, 0.0, False), (131072, 600, 2, 0.05, False), (87382, 33, 3, 0.2, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,drop,distinct", SORTS)
def test_sort(T, E, K, drop, distinct):
    idx, gate = selection(T, E, K, T + E, drop, distinct)
    rt = sorted_on_gpu(idx, gate, E)
    check_sort(rt, idx, gate, E)
    # the same buffers again, another selection: nothing of the first is left
    idx2, gate2 = selection(T, E, K, T + E + 1, min(1.0, drop + 0.3), distinct)
    rt2 = sorted_on_gpu(idx2, gate2, E, routing=rt)
    assert rt2 is rt
    check_sort(rt, idx2, gate2, E)


@pytest.mark.gpu
def test_no_tokens():
    from fine_grained_mixture_top_b200 import moe
    rt = sorted_on_gpu(np.zeros((0, 4), np.int32), np.zeros((0, 4), np.float32), 6)
    check_sort(rt, np.zeros((0, 4), np.int32), np.zeros((0, 4), np.float32), 6)
    rows = moe.permute(rt, torch.zeros(0, 32, device="cuda"))
    assert rows.shape == (0, 32)
    assert moe.unpermute(rt, rows).shape == (0, 32)
    assert moe.permute_bwd(rt, rows).shape == (0, 32)
    drows, dgate = moe.unpermute_bwd(rt, torch.zeros(0, 32, device="cuda"), rows)
    assert drows.shape == (0, 32) and dgate.shape == (0, 4)


ROWS = [  # T, E, K, drop, width, column offset (elements) of every row tensor
    (1, 4, 1, 0.0, 8, 0), (5, 64, 8, 0.0, 2048, 0), (37, 9, 3, 0.4, 1001, 0), (200, 16, 2, 0.0, 264, 3),
    (64, 200, 32, 0.2, 72, 0), (300, 7, 4, 0.1, 1, 0), (150, 12, 6, 1.0, 130, 0), (1000, 33, 8, 0.05, 7168, 0),
    (90, 5, 5, 0.0, 66, 2),
]


def strided(shape, dtype, off, fill=None):
    """A [rows, width] view whose rows are not adjacent and start `off`
    elements into a wider tensor; the rest of that tensor must stay as it is."""
    rows, width = shape
    base = torch.full((rows, width + (off + 5 if off else 0)), 7.0, dtype=dtype, device="cuda")
    view = base[:, off:off + width] if off else base
    if fill is not None:
        view.copy_(fill)
    return base, view


def close(got, ref, mag, n, dtype):
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + (n + 1) * 2.0 ** -24 * mag
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25   # half a step of the subnormals
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,E,K,drop,width,off", ROWS)
def test_rows_and_gradients(T, E, K, drop, width, off, dtype):
    from fine_grained_mixture_top_b200 import moe
    dt = DTYPES[dtype]
    idx, gate = selection(T, E, K, 3 * T + width, drop)
    rt = sorted_on_gpu(idx, gate, E)
    ref = plain_sort(idx, gate, E, rt.struct.P_max, rt.struct.R_max)
    R, used = rt.struct.R_max, int(ref["offsets"][-1])
    g = torch.Generator().manual_seed(T + width)
    x = torch.randn(T, width, generator=g).to(dt)
    xb, xv = strided((T, width), dt, off, x.cuda())
    rb, rv = strided((R, width), dt, off)
    out = moe.permute(rt, xv, rows=rv)
    assert out.data_ptr() == rv.data_ptr()
    want = torch.full_like(rb, 7.0).cpu()
    tok = torch.from_numpy(ref["row_tok"][:used])
    cols = slice(off, off + width) if off else slice(None)
    want[:used, cols] = torch.where((tok >= 0)[:, None], x[tok.clamp_min(0)], torch.zeros((), dtype=dt))
    assert torch.equal(rb.cpu(), want)              # bit for bit, rows past the last segment and the gaps untouched
    assert torch.equal(xb.cpu()[:, cols], x)

    y = torch.randn(R, width, generator=g).to(dt)
    yb, yv = strided((R, width), dt, off, y.cuda())
    y64 = y.double().numpy()
    P = int(ref["tok_ptr"][-1])
    pt = np.repeat(np.arange(T), np.diff(ref["tok_ptr"]))
    pr, pg = ref["pair_row"][:P], ref["pair_gate"][:P].astype(np.float64)
    for name, w in (("unpermute", pg), ("permute_bwd", np.ones(P))):
        o64, mag = np.zeros((T, width)), np.zeros((T, width))
        np.add.at(o64, pt, y64[pr] * w[:, None])
        np.add.at(mag, pt, np.abs(y64[pr] * w[:, None]))
        ob, ov = strided((T, width), dt, off)
        getattr(moe, name)(rt, yv, ov)
        close(ov, o64, mag, K, dt)
        if off:
            assert torch.all(ob[:, :off] == 7) and torch.all(ob[:, off + width:] == 7)

    do = torch.randn(T, width, generator=g).to(dt)
    dob, dov = strided((T, width), dt, off, do.cuda())
    db, dv = strided((R, width), dt, off)
    drows, dgate = moe.unpermute_bwd(rt, dov, yv, drows=dv)
    do64 = do.double().numpy()
    d64 = np.zeros((used, width))
    d64[pr] = do64[pt] * pg[:, None]
    close(dv[:used], d64, np.abs(d64), 0, dt)
    assert torch.all(dv[used:] == 7)
    g64 = (do64[pt] * y64[pr]).sum(1)
    gmag = np.abs(do64[pt] * y64[pr]).sum(1)
    full, fmag = np.zeros((T, K)), np.zeros((T, K))
    kept = (idx >= 0) & (idx < E)
    full[kept], fmag[kept] = g64, gmag
    assert dgate.shape == (T, K)
    close(dgate, full, fmag, width, torch.float32)
    assert torch.all(dgate.cpu()[torch.from_numpy(~kept)] == 0)
    pairs = torch.full((rt.struct.P_max,), 5.0, device="cuda")
    moe.unpermute_bwd(rt, dov, yv, drows=dv, dgate=pairs, pairs=True)
    assert torch.equal(pairs[:P].cpu(), dgate.cpu()[torch.from_numpy(kept)])
    assert torch.all(pairs[P:] == 5)


@pytest.mark.gpu
def test_codes_are_moved_bit_for_bit():
    from fine_grained_mixture_top_b200 import moe
    for width in (48, 20, 33):
        idx, gate = selection(70, 6, 3, width, 0.2)
        rt = sorted_on_gpu(idx, gate, 6)
        x = torch.randint(0, 256, (70, width), dtype=torch.uint8)
        rows = moe.permute(rt, x.cuda().view(torch.float8_e4m3fn)).view(torch.uint8).cpu()
        tok = rt["row_tok"].cpu()[:int(rt["offsets"][-1])].long()
        want = torch.where((tok >= 0)[:, None], x[tok.clamp_min(0)], torch.zeros((), dtype=torch.uint8))
        assert torch.equal(rows[:tok.numel()], want)


@pytest.mark.gpu
def test_gradients_against_differences():
    """L = <dout, unpermute(permute(x) * s)> for fixed row factors s: its
    gradients in x and in the gates, by central differences of the float64
    forward, against the backward calls chained."""
    from fine_grained_mixture_top_b200 import moe
    T, E, K, width = 6, 4, 2, 16
    idx, gate = selection(T, E, K, 5, 0.2)
    rt = sorted_on_gpu(idx, gate, E)
    ref = plain_sort(idx, gate, E, rt.struct.P_max, rt.struct.R_max)
    rs = np.random.RandomState(0)
    x, do = rs.randn(T, width).astype(np.float32), rs.randn(T, width).astype(np.float32)
    s = rs.rand(rt.struct.R_max, 1).astype(np.float32)
    kept = (idx >= 0) & (idx < E)

    def loss(x, gate):
        out = np.zeros((T, width))
        p = 0
        for t in range(T):
            for k in range(K):
                if kept[t, k]:
                    out[t] += gate[t, k] * x[t] * s[ref["pair_row"][p], 0]
                    p += 1
        return (out * do).sum()

    sd = torch.from_numpy(s).cuda()
    rows = moe.permute(rt, torch.from_numpy(x).cuda())
    used = int(ref["offsets"][-1])
    rows[used:] = 0
    y = rows * sd
    drows, dgate = moe.unpermute_bwd(rt, torch.from_numpy(do).cuda(), y)
    drows[used:] = 0
    dx = moe.permute_bwd(rt, drows * sd).cpu().numpy()
    h = 1e-4
    for arr, got in ((x, dx), (gate, dgate.cpu().numpy())):
        num = np.zeros(arr.shape)
        for i in np.ndindex(*arr.shape):
            vals = []
            for sign in (1, -1):
                a = arr.astype(np.float64)
                a[i] += sign * h
                vals.append(loss(a, gate.astype(np.float64)) if arr is x else loss(x.astype(np.float64), a))
            num[i] = (vals[0] - vals[1]) / (2 * h)
        # the loss is linear in each argument: differences are exact up to 1e-11, fp32 sums to 2^-20 of unit terms
        np.testing.assert_allclose(got, num, atol=5e-5)


@pytest.mark.gpu
def test_rows_of_the_layers_own_routing():
    """permute / unpermute on the routing of moe_route and of token rounding:
    unpermute is the layer's aggregation."""
    from fine_grained_mixture_top_b200 import moe
    from workloads import MoEConfig, make_inputs
    for mode in (0, 1):
        cfg = MoEConfig("rows", T=900, d=256, E=16, n=64, K=4, w_std=0.05, bias="normal", seed=61, round_mode=mode)
        inp = make_inputs(cfg, "cuda")
        layer = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K, round_mode=mode, seed=cfg.seed)
        layer.route(inp["X"], inp["Wr"], inp["bias"])
        rt = layer.routing
        used, P = int(rt["offsets"][-1]), int(rt["tok_ptr"][-1])
        rows = moe.permute(rt, inp["X"])
        tok = rt["row_tok"][:used].long()
        want = torch.where((tok >= 0)[:, None], inp["X"][tok.clamp_min(0)], torch.zeros((), dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(rows[:used], want)
        out = moe.unpermute(rt, rows).double().cpu()
        pt = torch.repeat_interleave(torch.arange(cfg.T), torch.diff(rt["tok_ptr"].cpu()).long())
        y = rows.double().cpu()[rt["pair_row"][:P].cpu().long()] * rt["pair_gate"][:P].double().cpu()[:, None]
        ref = torch.zeros(cfg.T, cfg.d, dtype=torch.float64).index_add_(0, pt, y)
        mag = torch.zeros(cfg.T, cfg.d, dtype=torch.float64).index_add_(0, pt, y.abs())
        assert torch.all((out - ref).abs() <= 2.0 ** -8 * ref.abs() + 17 * 2.0 ** -24 * mag)
        if mode:
            drows, dg = moe.unpermute_bwd(rt, inp["dO"], rows, pairs=True)
            g64 = (inp["dO"].double().cpu()[pt] * rows.double().cpu()[rt["pair_row"][:P].cpu().long()]).sum(1)
            assert torch.all((dg[:P].double().cpu() - g64).abs() <= 257 * 2.0 ** -24 * 256 * 16)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    from fine_grained_mixture_top_b200 import moe
    T, E, K, width = 3000, 20, 4, 96
    idx, gate = selection(T, E, K, 9, 0.1)
    ti, tg = torch.from_numpy(idx).cuda(), torch.from_numpy(gate).cuda()
    x = torch.randn(T, width, device="cuda")
    rt = moe.sort_pairs(ti, tg, E)
    rows = torch.zeros(rt.struct.R_max, width, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):   # enqueued on the side stream, seen there without a synchronize in between
        moe.sort_pairs(ti, tg, E, routing=rt, ws=ws)
        moe.permute(rt, x, rows=rows)
        out = moe.unpermute(rt, rows)
    side.synchronize()
    ref = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.sort_pairs(ti, tg, E, routing=rt, ws=ws)
        moe.permute(rt, x, rows=rows)
        out2 = moe.unpermute(rt, rows)
    idx2, gate2 = selection(T, E, K, 10, 0.4)
    ti.copy_(torch.from_numpy(idx2))
    tg.copy_(torch.from_numpy(gate2))
    graph.replay()
    torch.cuda.synchronize()
    check_sort(rt, idx2, gate2, E)
    assert not torch.equal(out2, ref)
    ti.copy_(torch.from_numpy(idx))
    tg.copy_(torch.from_numpy(gate))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, ref)   # the same bits from the same inputs, run after run
    del graph


@pytest.mark.gpu
def test_nan_and_infinity_stay_in_their_rows():
    from fine_grained_mixture_top_b200 import moe
    idx = np.array([[0, 1], [1, 0], [-1, -1]], np.int32)
    gate = np.ones((3, 2), np.float32)
    rt = sorted_on_gpu(idx, gate, 2)
    x = torch.ones(3, 16, device="cuda")
    x[1, 3] = float("nan")
    x[2, :] = float("inf")      # a token without choices reaches nothing
    rows = moe.permute(rt, x)
    used = int(rt["offsets"][-1])
    assert int(torch.isnan(rows[:used]).sum()) == 2 and not torch.isinf(rows[:used]).any()
    out = moe.unpermute(rt, rows)
    assert torch.equal(out[0], torch.full((16,), 2.0, device="cuda"))
    assert torch.isnan(out[1, 3]) and int(torch.isnan(out).sum()) == 1
    assert torch.all(out[2] == 0)


@pytest.mark.gpu
def test_a_stream_given_by_name_and_what_is_refused():
    """With `stream` the whole call belongs to it, allocations too: work queued
    before it on another stream is not waited for, memory it takes is not shared."""
    from fine_grained_mixture_top_b200 import moe
    T, E, K, width = 20000, 12, 3, 128
    idx, gate = selection(T, E, K, 21, 0.1)
    ti, tg = torch.from_numpy(idx).cuda(), torch.from_numpy(gate).cuda()
    x = torch.randn(T, width, device="cuda")
    ref = moe.unpermute(rt := moe.sort_pairs(ti, tg, E), moe.permute(rt, x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        junk = torch.full((1 << 22,), 1, device="cuda")      # the current stream keeps taking and freeing memory
        r = moe.sort_pairs(ti, tg, E, stream=s)
        rows = moe.permute(r, x, stream=s)
        outs.append(moe.unpermute(r, rows, stream=s))
        del junk, r, rows
    s.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    from workloads import MoEConfig, make_inputs
    cfg = MoEConfig("rows2", T=64, d=128, E=4, n=64, K=2, seed=1)
    layer = moe.MoELayer(cfg.T, cfg.d, cfg.E, cfg.n, cfg.K)
    with pytest.raises(ValueError, match="sort_pairs"):
        moe.sort_pairs(ti[:64, :2].contiguous(), tg[:64, :2].contiguous(), 4, routing=layer.routing)
    with pytest.raises(ValueError, match="another"):
        moe.sort_pairs(ti, tg, E + 1, routing=rt)
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError, match="stream"):
            moe.permute(rt, x, stream=torch.cuda.Stream(device=1))
