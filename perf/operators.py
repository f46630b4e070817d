"""Cases for the layer's row movement and its 8-bit products.

permute    tokens sorted by the experts they chose, the rows in that order,
           and the gradient of the tokens
unpermute  the weighted sum of each token's rows, and the gradients of the
           rows and of the weights
quantize   E4M3 codes with one fp32 scale per block of 128: rows (gathered or
           behind the SwiGLU product if asked), columns of row blocks, and
           128 x 128 blocks of expert weights
product    matrix products of such codes: dense, grouped by expert, and the
           weight gradient of the groups

`own` picks who computes a pass: elementary torch operations in 32 bits, or
the library's kernels.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TILE = 128          # rows per tile of an expert's segment, values per scale block
AMAX_FLOOR = 2.0 ** -110
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of eight sequences on a layer of 64 experts
        dict(name="permute_decode", op="permute", dir="fwd", type="bf16", T=8, d=2048, E=64, K=8, drop=0.0, skew=0.0),
        # the training batch of the 7B-class layer
        dict(name="permute_batch", op="permute", dir="fwd", type="bf16", T=16384, d=1536, E=128, K=8, drop=0.0,
             skew=0.5),
        # tokens over their expert's capacity dropped, an odd width, the gradient of the tokens
        dict(name="permute_grad_ragged", op="permute", dir="bwd", type="fp16", T=5003, d=1001, E=37, K=6, drop=0.1,
             skew=0.5),
        # a small decoding batch at the widest model dimension here
        dict(name="unpermute_decode", op="unpermute", dir="fwd", type="bf16", T=32, d=7168, E=256, K=8, drop=0.0,
             skew=0.0),
        # the largest layer's prefill or training batch
        dict(name="unpermute_batch", op="unpermute", dir="fwd", type="bf16", T=8192, d=7168, E=256, K=8, drop=0.0,
             skew=1.0),
        # the backward of the 7B-class layer's combine
        dict(name="unpermute_grad", op="unpermute", dir="bwd", type="bf16", T=16384, d=1536, E=128, K=8, drop=0.0,
             skew=0.5),
        # activations on their way into the first product: gathered by expert and quantized
        dict(name="quantize_gathered", op="quantize", form="gather", type="bf16", rows=16384, cols=2048, E=64, K=8),
        # expert weights after an optimizer step
        dict(name="quantize_weights", op="quantize", form="blocks_t", type="bf16", E=128, rows=1536, cols=512),
        # a dense projection for a few decoded tokens: the weights' bytes are all that counts
        dict(name="product_decode", op="product", form="dense", M=16, N=4096, Kd=7168),
        # a dense projection with no whole tile in any direction
        dict(name="product_ragged", op="product", form="dense", M=1001, N=1528, Kd=2000),
        # the up-projection of the OLMoE-shaped layer's training batch
        dict(name="product_grouped", op="product", form="grouped", T=32768, E=64, K=8, N=2048, Kd=2048, skew=0.5),
        # the first weight gradient of the 7B-class layer
        dict(name="product_dw", op="product", form="dw", T=16384, E=128, K=8, M=1536, N=512, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "quantize", "product", "product"])
    if op in ("permute", "unpermute"):
        while True:
            c = dict(op=op, dir=rng.choice(["fwd", "bwd"]), type=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     T=_log(rng, 1, 32768), d=_log(rng, 64, 8192), E=_log(rng, 1, 512), K=rng.randint(1, 8),
                     drop=rng.choice([0.0, 0.0, 0.2]), skew=rng.choice([0.0, 0.5, 1.0]))
            if rng.random() < 0.5:
                c["d"] = max(64, c["d"] // 64 * 64)
            c["K"] = min(c["K"], c["E"])
            if c["T"] * c["K"] * c["d"] * (4 if c["type"] == "fp32" else 2) <= 8192 * 8 * 7168 * 2:
                return c
    if op == "quantize":
        while True:
            form = rng.choice(["rows", "gather", "swiglu", "cols", "blocks", "blocks_t"])
            c = dict(op=op, form=form, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     rows=_log(rng, 1, 32768), cols=_log(rng, 16, 8192), E=1, K=1)
            if form == "gather":
                c |= dict(E=_log(rng, 1, 256), K=rng.randint(1, 8))
                c["K"] = min(c["K"], c["E"])
            if form in ("blocks", "blocks_t"):
                c |= dict(E=_log(rng, 1, 128), rows=_log(rng, 64, 7168), cols=_log(rng, 64, 4096))
            if c["E"] * 128 * c["cols"] + c["E"] ** (form[:6] == "blocks") * c["rows"] * c["K"] * c["cols"] <= 2.4e8:
                return c
    while True:
        form = rng.choice(["dense", "dense", "grouped", "dw"])
        if form == "dense":
            c = dict(op=op, form=form, M=_log(rng, 1, 16384), N=_log(rng, 64, 8192), Kd=_log(rng, 64, 8192))
            work = c["M"] * c["N"] * c["Kd"]
        else:
            c = dict(op=op, form=form, T=_log(rng, 1, 32768), E=_log(rng, 1, 256), K=rng.randint(1, 8),
                     N=_log(rng, 64, 4096), skew=rng.choice([0.0, 0.5, 1.0]))
            c["K"] = min(c["K"], c["E"])
            side = c["M" if form == "dw" else "Kd"] = _log(rng, 64, 4096)
            work = (c["T"] * c["K"] + 64 * c["E"]) * c["N"] * side
            if c["E"] * c["N"] * side > 4.5e8:
                continue
        if work <= 32768 * 8 * 2048 * 2048:
            return c


# -------------------------------------------------------------------- inputs
def _up(x, m):
    return -(-x // m) * m


def _selection(c, g):
    """Distinct experts per token, some far more popular than others where
    the case is skewed, gates that sum to one, and dropped choices as -1."""
    T, E, K = c["T"], c["E"], c["K"]
    pop = torch.randn(E, generator=g, device="cuda") * c["skew"] * 2
    score = torch.rand(T, E, generator=g, device="cuda").log().neg().log().neg() + pop
    top = score.topk(K, dim=1)
    idx = top.indices.to(torch.int32)
    gate = torch.softmax(top.values, dim=1).float().contiguous()
    if c.get("drop"):
        idx = torch.where(torch.rand(T, K, generator=g, device="cuda") < c["drop"], torch.full_like(idx, -1), idx)
    return idx.contiguous(), gate


def _sorted(idx, gate, E):
    """The routing of a selection: pairs in token order, rows in expert order
    with each expert's segment padded to whole tiles."""
    T, K = idx.shape
    P = T * K
    R = _up(P + (TILE - 1) * min(E, P), TILE)
    dev = idx.device
    key = idx.reshape(-1).long()
    kept = (key >= 0) & (key < E)
    key = torch.where(kept, key, E)
    order = torch.sort(key, stable=True).indices
    n = torch.zeros(E + 1, dtype=torch.long, device=dev).scatter_add_(0, key, torch.ones_like(key))
    counts = n[:E]
    start = torch.cumsum(n, 0) - n
    seg = (counts + TILE - 1) // TILE * TILE
    offsets = torch.zeros(E + 1, dtype=torch.long, device=dev)
    offsets[1:] = torch.cumsum(seg, 0)
    rank = torch.empty_like(key).scatter_(0, order, torch.arange(P, device=dev)) - start[key]
    row = torch.where(kept, offsets[key] + rank, R)               # R: a row that is cut off again
    pair = torch.where(kept, torch.cumsum(kept, 0) - 1, P)
    i32 = torch.int32
    row_tok = torch.full((R + 1,), -1, dtype=i32, device=dev)
    row_tok.scatter_(0, row, torch.where(kept, torch.arange(P, device=dev) // K, -1).to(i32))
    row_gate = torch.zeros(R + 1, device=dev).scatter_(0, row, torch.where(kept, gate.reshape(-1), 0.0))
    pair_row = torch.full((P + 1,), -1, dtype=i32, device=dev)
    pair_row.scatter_(0, pair, torch.where(kept, row, -1).to(i32))
    pair_gate = torch.zeros(P + 1, device=dev).scatter_(0, pair, torch.where(kept, gate.reshape(-1), 0.0))
    tok_ptr = torch.zeros(T + 1, dtype=i32, device=dev)
    tok_ptr[1:] = torch.cumsum(kept.reshape(T, K).sum(1), 0)
    row_tok[R] = -1
    pair_row[P] = -1
    return {"counts": counts.to(i32), "offsets": offsets.to(i32), "row_tok": row_tok[:R], "row_gate": row_gate[:R],
            "pair_row": pair_row[:P], "pair_gate": pair_gate[:P], "tok_ptr": tok_ptr,
            "slot_row": torch.where(kept, row, -1).reshape(T, K)}


def _values(g, shape, dtype):
    """Activations: normal, with a few channels ten times as large."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., :: 97] *= 10.0
    return x.to(dtype)


def _codes(g, rows, cols, pad_rows=None):
    """Codes [rows, cols] with a row stride that is a multiple of 16, and
    their scales [ceil(cols / 128), rows], as the quantizer leaves them."""
    store = torch.zeros(rows, _up(cols, 16), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(-(-cols // TILE), rows, device="cuda")
    step = max(1, (1 << 27) // max(1, _up(cols, TILE)))
    for r in range(0, rows, step):
        x = torch.randn(min(step, rows - r), _up(cols, TILE), generator=g, device="cuda")
        x[:, cols:] = 0
        x = x.view(x.shape[0], -1, TILE)
        s = x.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
        store[r:r + step, :cols] = (x / s[:, :, None]).reshape(x.shape[0], -1)[:, :cols].to(torch.float8_e4m3fn)
        scales[:, r:r + step] = s.t() * torch.exp2(torch.randn(1, x.shape[0], generator=g, device="cuda"))
    return store[:, :cols], scales


def _weights(g, E, N, K):
    """Expert weights as codes [E, N, K] and scales [E, ceil(N / 128), ceil(K / 128)]."""
    store = torch.zeros(E, N, _up(K, 16), dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        store[e, :, :K] = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp_(-448, 448).to(
            torch.float8_e4m3fn)
    s = torch.rand(E, -(-N // TILE), -(-K // TILE), generator=g, device="cuda") * 2e-4 + 1e-4
    return store[:, :, :K], s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("permute", "unpermute"):
        dtype = TYPES[c["type"]]
        s["idx"], s["gate"] = _selection(c, g)
        s["rt"] = _sorted(s["idx"], s["gate"], c["E"])
        R = s["rt"]["row_tok"].numel()
        used = (torch.arange(R, device="cuda") < s["rt"]["offsets"][-1])[:, None]
        if c["op"] == "permute" and c["dir"] == "fwd":
            s["x"] = _values(g, (c["T"], c["d"]), dtype)
            s["rows"] = torch.zeros(R, c["d"], dtype=dtype, device="cuda")
        else:
            s["rows"] = torch.where(used, _values(g, (R, c["d"]), dtype), 0).to(dtype)
        if c["op"] == "unpermute" and c["dir"] == "bwd":
            s["dout"] = _values(g, (c["T"], c["d"]), dtype)
            s["drows"] = torch.zeros(R, c["d"], dtype=dtype, device="cuda")
        if own:   # the handle that a program keeps for its batch size
            from fine_grained_mixture_top_b200 import moe
            s["handle"] = moe.sort_pairs(s["idx"], s["gate"], c["E"])
    elif c["op"] == "quantize":
        dtype = TYPES[c["type"]]
        if c["form"] in ("blocks", "blocks_t"):
            s["w"] = (torch.randn(c["E"], c["rows"], c["cols"], generator=g, device="cuda") * 0.02).to(dtype)
        else:
            s["x"] = _values(g, (c["rows"], c["cols"] * (2 if c["form"] == "swiglu" else 1)), dtype)
        if c["form"] == "gather":
            idx, gate = _selection(dict(T=c["rows"], E=c["E"], K=c["K"], skew=0.5), g)
            rt = _sorted(idx, gate, c["E"])
            s["row_src"], s["rows_used"] = rt["row_tok"].contiguous(), rt["offsets"][-1:].clone()
            R = rt["row_tok"].numel()
            s["codes"] = torch.zeros(R, _up(c["cols"], 16), dtype=torch.float8_e4m3fn, device="cuda")[:, :c["cols"]]
            s["scales"] = torch.zeros(-(-c["cols"] // TILE), R, device="cuda")
    elif c["form"] == "dense":
        s["a"], s["sa"] = _codes(g, c["M"], c["Kd"])
        s["b"], s["sb"] = _weights(g, 1, c["N"], c["Kd"])
        s["b"], s["sb"] = s["b"][0], s["sb"][0]
    else:
        idx, gate = _selection(c, g)
        rt = _sorted(idx, gate, c["E"])
        R = rt["row_tok"].numel()
        s["offsets"] = rt["offsets"].tolist()      # a program of plain products knows its groups on the host
        real = rt["row_tok"] >= 0
        if c["form"] == "grouped":
            s["a"], s["sa"] = _codes(g, R, c["Kd"])
            s["a"].view(torch.uint8).mul_(real[:, None].to(torch.uint8))
            s["b"], s["sb"] = _weights(g, c["E"], c["N"], c["Kd"])
            s["out"] = torch.zeros(R, _up(c["N"], 8), dtype=torch.bfloat16, device="cuda")[:, :c["N"]]
        else:
            s["a"], s["sa"] = _codes(g, c["M"], R)
            s["b"], s["sb"] = _codes(g, c["N"], R)
            s["a"].view(torch.uint8).mul_(real[None, :].to(torch.uint8))
            s["b"].view(torch.uint8).mul_(real[None, :].to(torch.uint8))
        if own:
            from fine_grained_mixture_top_b200 import moe
            s["handle"] = moe.sort_pairs(idx, gate, c["E"])
    return s


# ---------------------------------------------------------------- plain form
def _row_scales(s, rows, cols):
    """[ceil(cols / 128), rows] scales as [rows, cols] factors."""
    return s.t().repeat_interleave(TILE, dim=1)[:rows, :cols]


def _block_scales(s, rows, cols):
    return s.repeat_interleave(TILE, dim=-2).repeat_interleave(TILE, dim=-1)[..., :rows, :cols]


def _gather(src, index):
    """src[index], zeros where the index is -1."""
    out = src[index.clamp_min(0).long()]
    return torch.where((index >= 0)[..., None], out, torch.zeros((), dtype=out.dtype, device=out.device))


def _pair_sum(rows, slot_row, weight):
    """Per token, the sum of its rows times their weights: one choice of
    every token at a time, so that no [T, K, d] tensor is made."""
    out = torch.zeros(slot_row.shape[0], rows.shape[1], device=rows.device)
    for k in range(slot_row.shape[1]):
        r = _gather(rows, slot_row[:, k]).float()
        out += r if weight is None else r * weight[:, k:k + 1]
    return out


def _codes_of(x, axis_blocks):
    """x [..., B, 128, ...] split along axis_blocks + 1: codes and scales."""
    amax = x.abs().amax(axis_blocks + 1, keepdim=True).clamp_min(AMAX_FLOOR)
    return (x * (E4M3_MAX / amax)).to(torch.float8_e4m3fn), (amax / E4M3_MAX)


def _pad(x, dim, m):
    n = _up(x.shape[dim], m) - x.shape[dim]
    if n == 0:
        return x
    shape = list(x.shape)
    shape[dim] = n
    return torch.cat([x, torch.zeros(shape, dtype=x.dtype, device=x.device)], dim)


def _plain_quantize(s):
    c, form = s["case"], s["case"]["form"]
    if form in ("blocks", "blocks_t"):
        w = s["w"].float()
        w = w.transpose(1, 2) if form == "blocks_t" else w
        E, a, b = w.shape
        w = _pad(_pad(w, 1, TILE), 2, TILE)
        t = w.reshape(E, w.shape[1] // TILE, TILE, w.shape[2] // TILE, TILE)
        amax = t.abs().amax((2, 4), keepdim=True).clamp_min(AMAX_FLOOR)
        q = (t * (E4M3_MAX / amax)).to(torch.float8_e4m3fn).reshape(w.shape)[:, :a, :b]
        return {"codes": q.contiguous(), "scales": (amax / E4M3_MAX)[:, :, 0, :, 0].contiguous()}
    x = s["x"].float()
    if form == "swiglu":
        h, u = x[:, :c["cols"]], x[:, c["cols"]:]
        x = h / (1 + torch.exp(-h)) * u
    if form == "cols":
        rows, cols = x.shape
        x = _pad(x, 0, TILE)
        q, sc = _codes_of(x.view(-1, TILE, cols), 0)
        return {"codes": q.reshape(-1, cols).t()[:, :rows].contiguous(), "scales": sc[:, 0].contiguous()}
    rows, cols = x.shape
    x = _pad(x, 1, TILE)
    q, sc = _codes_of(x.view(rows, -1, TILE), 1)
    q, sc = q.reshape(rows, -1)[:, :cols], sc[:, :, 0]
    if form == "gather":
        src = s["row_src"]
        used = torch.arange(src.numel(), device=src.device) < s["rows_used"]
        real = src >= 0
        q = _gather(q.contiguous().view(torch.uint8), src).view(torch.float8_e4m3fn)
        sc = torch.where(real[:, None], sc[src.clamp_min(0).long()], (AMAX_FLOOR / E4M3_MAX) * used[:, None])
    return {"codes": q.contiguous(), "scales": sc.t().contiguous()}


def _plain_product(s):
    c, form = s["case"], s["case"]["form"]
    a, sa, b, sb = s["a"], s["sa"], s["b"], s["sb"]
    if form == "dense":
        A = a.float() * _row_scales(sa, *a.shape)
        B = b.float() * _block_scales(sb, *b.shape)
        return {"out": (A @ B.t()).to(torch.bfloat16)}
    off = s["offsets"]
    if form == "grouped":
        out = torch.zeros_like(s["out"])
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                A = a[lo:hi].float() * _row_scales(sa[:, lo:hi], hi - lo, c["Kd"])
                B = b[e].float() * _block_scales(sb[e], c["N"], c["Kd"])
                out[lo:hi] = (A @ B.t()).to(torch.bfloat16)
        return {"out": out}
    out = torch.zeros(c["E"], c["M"], c["N"], dtype=torch.bfloat16, device=a.device)
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            A = a[:, lo:hi].float() * _row_scales(sa[lo // TILE:hi // TILE], c["M"], hi - lo)
            B = b[:, lo:hi].float() * _row_scales(sb[lo // TILE:hi // TILE], c["N"], hi - lo)
            out[e] = (A @ B.t()).to(torch.bfloat16)
    return {"out": out}


def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "permute":
        if c["dir"] == "fwd":
            rt = _sorted(s["idx"], s["gate"], c["E"])
            return {"rows": _gather(s["x"], rt["row_tok"]), "counts": rt["counts"], "offsets": rt["offsets"],
                    "row_tok": rt["row_tok"], "pair_row": rt["pair_row"], "tok_ptr": rt["tok_ptr"]}
        return {"dx": _pair_sum(s["rows"], s["rt"]["slot_row"], None).to(s["rows"].dtype)}
    if c["op"] == "unpermute":
        if c["dir"] == "fwd":
            return {"out": _pair_sum(s["rows"], s["rt"]["slot_row"], s["gate"]).to(s["rows"].dtype)}
        rt = s["rt"]
        drows = (_gather(s["dout"], rt["row_tok"]).float() * rt["row_gate"][:, None]).to(s["rows"].dtype)
        row_dot = (_gather(s["dout"], rt["row_tok"]).float() * s["rows"].float()).sum(1)
        slot = rt["slot_row"]
        return {"drows": drows, "dgate": torch.where(slot >= 0, row_dot[slot.clamp_min(0)], 0.0)}
    return _plain_quantize(s) if c["op"] == "quantize" else _plain_product(s)


def _run_own(s):
    from fine_grained_mixture_top_b200 import moe
    c = s["case"]
    if c["op"] == "permute":
        if c["dir"] == "fwd":
            rt = moe.sort_pairs(s["idx"], s["gate"], c["E"], routing=s["handle"])
            rows = moe.permute(rt, s["x"], rows=s["rows"])
            return {"rows": rows, "counts": rt["counts"], "offsets": rt["offsets"], "row_tok": rt["row_tok"],
                    "pair_row": rt["pair_row"], "tok_ptr": rt["tok_ptr"]}
        return {"dx": moe.permute_bwd(s["handle"], s["rows"])}
    if c["op"] == "unpermute":
        if c["dir"] == "fwd":
            return {"out": moe.unpermute(s["handle"], s["rows"])}
        drows, dgate = moe.unpermute_bwd(s["handle"], s["dout"], s["rows"], drows=s["drows"])
        return {"drows": drows, "dgate": dgate}
    if c["op"] == "quantize":
        form = c["form"]
        if form in ("blocks", "blocks_t"):
            q, sc = moe.fp8_quantize_blocks(s["w"], transpose=form == "blocks_t")
        elif form == "cols":
            q, sc = moe.fp8_quantize_cols(s["x"])
        elif form == "gather":
            q, sc = moe.fp8_quantize_rows(s["x"], row_src=s["row_src"], rows_used=s["rows_used"], codes=s["codes"],
                                          scales=s["scales"])
        else:
            q, sc = moe.fp8_quantize_rows(s["x"], swiglu=form == "swiglu")
        return {"codes": q, "scales": sc}
    if c["form"] == "dense":
        return {"out": moe.fp8_gemm(s["a"], s["sa"], s["b"], s["sb"])}
    if c["form"] == "grouped":
        return {"out": moe.fp8_gemm(s["a"], s["sa"], s["b"], s["sb"], routing=s["handle"], out=s["out"])}
    return {"out": moe.fp8_gemm_dw(s["a"], s["sa"], s["b"], s["sb"], routing=s["handle"])}


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    if c["op"] in ("permute", "unpermute"):
        es = 4 if c["type"] == "fp32" else 2
        P = c["T"] * c["K"] * (1 - c["drop"])
        rows, toks = P * c["d"] * es, c["T"] * c["d"] * es
        if c["op"] == "unpermute" and c["dir"] == "bwd":
            return {"bytes": 2 * rows + toks + 16 * P, "flops": 3 * P * c["d"]}
        return {"bytes": rows + toks + 16 * P, "flops": P * c["d"]}
    if c["op"] == "quantize":
        es = 4 if c["type"] == "fp32" else 2
        if c["form"] in ("blocks", "blocks_t"):
            n = c["E"] * c["rows"] * c["cols"]
            return {"bytes": n * (es + 1), "flops": 3 * n}
        n = c["rows"] * c["cols"]
        k = c["K"]
        return {"bytes": n * es * (2 if c["form"] == "swiglu" else 1) + n * k * (1 + 4 / TILE), "flops": 3 * n * k}
    if c["form"] == "dense":
        m, n, k, e = c["M"], c["N"], c["Kd"], 1
    elif c["form"] == "grouped":
        m, n, k, e = c["T"] * c["K"], c["N"], c["Kd"], min(c["E"], c["T"] * c["K"])
    else:
        rows = c["T"] * c["K"]
        return {"bytes": rows * (c["M"] + c["N"]) * (1 + 4 / TILE) + 2 * c["E"] * c["M"] * c["N"],
                "flops": 2 * rows * c["M"] * c["N"]}
    return {"bytes": m * k * (1 + 4 / TILE) + e * n * k + 2 * m * n, "flops": 2 * m * n * k}


# ------------------------------------------------------------- in 64 bits
def _exact_route(s):
    """Row of every choice (-1 dropped) and token of every row, by counting."""
    c = s["case"]
    idx = s["idx"].cpu().reshape(-1).numpy()
    E, K = c["E"], c["K"]
    P = idx.size
    lists = [[] for _ in range(E)]
    for p, e in enumerate(idx.tolist()):
        if 0 <= e < E:
            lists[e].append(p)
    R = _up(P + (TILE - 1) * min(E, P), TILE)
    slot, tok, off = [-1] * P, [-1] * R, 0
    for members in lists:
        for i, p in enumerate(members):
            slot[p], tok[off + i] = off + i, p // K
        off += _up(len(members), TILE)
    return torch.tensor(slot, device="cuda").view(-1, K), torch.tensor(tok, device="cuda")


def _exact_move(s):
    c = s["case"]
    slot, tok = _exact_route(s)
    if c["op"] == "permute" and c["dir"] == "fwd":
        x = s["x"].double()
        rows = torch.zeros(tok.numel(), c["d"], dtype=torch.float64, device="cuda")
        real = tok >= 0
        rows[real] = x[tok[real]]
        return {"rows": rows, "counts": None, "offsets": None, "row_tok": None, "pair_row": None, "tok_ptr": None}
    if c["dir"] == "fwd" or c["op"] == "permute":
        w = s["gate"].double() if c["op"] == "unpermute" else torch.ones_like(s["gate"]).double()
        out = torch.zeros(c["T"], c["d"], dtype=torch.float64, device="cuda")
        t, k = (slot >= 0).nonzero(as_tuple=True)
        out.index_add_(0, t, s["rows"][slot[t, k]].double() * w[t, k][:, None])
        return {"dx" if c["op"] == "permute" else "out": out}
    t, k = (slot >= 0).nonzero(as_tuple=True)
    drows = torch.zeros(tok.numel(), c["d"], dtype=torch.float64, device="cuda")
    dgate = torch.zeros(c["T"], c["K"], dtype=torch.float64, device="cuda")
    for i in range(0, t.numel(), 16384):
        ti, ki = t[i:i + 16384], k[i:i + 16384]
        r = slot[ti, ki]
        do = s["dout"][ti].double()
        drows[r] = do * s["gate"][ti, ki].double()[:, None]
        dgate[ti, ki] = (do * s["rows"][r].double()).sum(1)
    return {"drows": drows, "dgate": dgate}


def _nearest_e4m3(v):
    """The E4M3 value nearest to v (|v| <= 448), ties to the even one."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_quantize(s):
    c, form = s["case"], s["case"]["form"]
    floor = torch.tensor(AMAX_FLOOR, dtype=torch.float64, device="cuda")
    if form in ("blocks", "blocks_t"):
        codes, scales = [], []
        for w in s["w"]:
            w = (w.t() if form == "blocks_t" else w).double()
            sc = torch.stack([torch.stack([torch.maximum(q.abs().max(), floor) for q in r.split(TILE, 1)])
                              for r in w.split(TILE, 0)]) / E4M3_MAX
            codes.append(_nearest_e4m3(w / _block_scales(sc, *w.shape)).float())
            scales.append(sc)
        return {"codes": torch.stack(codes).double(), "scales": torch.stack(scales)}
    x = s["x"].double()
    if form == "swiglu":
        x = x[:, :c["cols"]] * torch.sigmoid(x[:, :c["cols"]]) * x[:, c["cols"]:]
    if form == "cols":
        x = x.t()
    sc = torch.stack([torch.maximum(b.abs().amax(1), floor) for b in x.split(TILE, 1)]) / E4M3_MAX
    q = torch.cat([_nearest_e4m3(b / sc[i][:, None]) for i, b in enumerate(x.split(TILE, 1))], 1)
    if form == "gather":
        src = s["row_src"].long()
        n = int(s["rows_used"])
        codes = torch.zeros(src.numel(), c["cols"], dtype=torch.float32, device="cuda")
        scales = torch.zeros(sc.shape[0], src.numel(), dtype=torch.float64, device="cuda")
        scales[:, :n] = floor / E4M3_MAX
        real = (src >= 0).nonzero()[:, 0]
        codes[real] = q[src[real]].float()
        scales[:, real] = sc[:, src[real]]
        return {"codes": codes.double(), "scales": scales}
    return {"codes": q, "scales": sc}


def _exact_block_sum(a, sa, b, sb):
    """sum over blocks of 128 of (a_block . b_block) * sa * sb, sb per row of b."""
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device="cuda")
    for i in range(-(-a.shape[1] // TILE)):
        k = slice(i * TILE, (i + 1) * TILE)
        out += (a[:, k].double() @ b[:, k].double().t()) * sa[i].double()[:, None] * sb[i].double()[None, :]
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] in ("permute", "unpermute"):
        return _exact_move(s)
    if c["op"] == "quantize":
        return _exact_quantize(s)
    col = lambda sb, n: sb.t().repeat_interleave(TILE, dim=1)[:, :n]  # noqa: E731
    if c["form"] == "dense":
        return {"out": _exact_block_sum(s["a"], s["sa"], s["b"], col(s["sb"], c["N"]))}
    off = s["offsets"]
    spans = [(e, off[e], off[e + 1]) for e in range(c["E"]) if off[e + 1] > off[e]]
    if c["form"] == "grouped":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            out[lo:hi] = _exact_block_sum(s["a"][lo:hi], s["sa"][:, lo:hi], s["b"][e], col(s["sb"][e], c["N"]))
        return {"out": out}
    out = torch.zeros(c["E"], c["M"], c["N"], dtype=torch.float64, device="cuda")
    for e, lo, hi in spans:
        t = slice(lo // TILE, hi // TILE)
        out[e] = _exact_block_sum(s["a"][:, lo:hi], s["sa"][t], s["b"][:, lo:hi], s["sb"][t])
    return {"out": out}
