"""Python binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; torch supplies the
device memory and the stream.  There is no fallback: if the shared library is
missing the import of this module's functions raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_DEBUG=1 in the environment loads the debug build instead (device-side
# routing checks reported through moe_get_status; same results otherwise)
LIB_PATH = os.path.join(_PKG, "libmoe_debug.so" if os.environ.get("MOE_DEBUG") == "1" else "libmoe.so")

c_void_p = ctypes.c_void_p
c_int32 = ctypes.c_int32
c_int64 = ctypes.c_int64

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, \
    MOE_ERR_DEVICE_CHECK, MOE_ERR_SCRATCH_LIMIT = range(8)


class MoeDims(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d", c_int32), ("E", c_int32), ("n", c_int32), ("K", c_int32)]


class MoeOpts(ctypes.Structure):
    _fields_ = [("round_mode", c_int32), ("router_grad", c_int32), ("seed", ctypes.c_uint64)]


_ROUTING_PTRS = ["logits", "probs", "topk_idx", "topk_gate", "tok_ptr", "pair_expert", "pair_gate", "pair_row",
                 "counts", "offsets", "row_tok", "row_gate", "tile_expert"]


class MoeRouting(ctypes.Structure):
    _fields_ = [(name, c_void_p) for name in _ROUTING_PTRS] + [("P_max", c_int64), ("R_max", c_int64),
                                                                ("pair_dS", c_void_p),
                                                                ("pair_slot", c_void_p)]


class MoeSizes(ctypes.Structure):
    _fields_ = [("P_max", c_int64), ("R_max", c_int64), ("route_ws", ctypes.c_size_t),
                ("fwd_ws", ctypes.c_size_t), ("bwd_ws", ctypes.c_size_t), ("h_elems", c_int64),
                ("fwd_mx_ws", ctypes.c_size_t), ("mx_weights_bytes", ctypes.c_size_t)]


class MoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = f"{what}: {status_str(code)} ({code})"
        if code == MOE_ERR_CUDA:
            msg += f": {last_error()}"
        super().__init__(msg)
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by fine_grained_mixture_top_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run python -m "
                               "fine_grained_mixture_top_b200.build" +
                               (" --debug" if LIB_PATH.endswith("_debug.so") else ""))
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.moe_query_sizes.argtypes = [P(MoeDims), P(MoeOpts), P(MoeSizes)]
        L.moe_route.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, P(MoeRouting), c_void_p,
                                ctypes.c_size_t, c_void_p]
        L.moe_route_noalloc.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, P(MoeRouting),
                                         c_void_p]
        L.moe_route_noalloc.restype = c_int32
        L.moe_token_round.argtypes = [P(MoeDims), P(MoeOpts), P(MoeRouting), c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_forward.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, P(MoeRouting), c_void_p,
                                  c_void_p, c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_forward_mxfp8.argtypes = L.moe_forward.argtypes
        L.moe_mx_quantize_weights.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, ctypes.c_size_t,
                                              c_void_p]
        L.moe_forward_mxfp8_q.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, P(MoeRouting), c_void_p,
                                          c_void_p, c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_backward.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   P(MoeRouting), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   ctypes.c_size_t, c_void_p]
        L.moe_backward_ev.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      P(MoeRouting), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                      ctypes.c_size_t, P(c_void_p), c_void_p]
        L.moe_set_sm_budget.argtypes = [c_int32]
        L.moe_route_given.argtypes = [P(MoeDims), P(MoeOpts), P(MoeRouting), c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_ep_pack.argtypes = [P(MoeDims), P(MoeOpts), P(MoeRouting), c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_ep_combine.argtypes = [P(MoeDims), P(MoeOpts), P(MoeRouting), c_void_p, c_void_p, c_void_p, c_void_p]
        L.moe_router_backward.argtypes = [P(MoeDims), P(MoeOpts), c_void_p, c_void_p, P(MoeRouting), c_void_p,
                                          c_void_p, c_void_p, c_void_p, c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_sort_sizes.argtypes = [c_int64, c_int32, c_int32, P(c_int64), P(c_int64), P(ctypes.c_size_t)]
        L.moe_sort_pairs.argtypes = [c_int64, c_int32, c_int32, P(MoeRouting), c_void_p, ctypes.c_size_t, c_void_p]
        L.moe_permute.argtypes = [c_int64, c_int32, P(MoeRouting), c_int32, c_int64, c_void_p, c_int64, c_void_p,
                                  c_int64, c_void_p]
        L.moe_permute_bwd.argtypes = L.moe_permute.argtypes
        L.moe_unpermute.argtypes = L.moe_permute.argtypes
        L.moe_unpermute_bwd.argtypes = [c_int64, c_int32, c_int32, P(MoeRouting), c_int32, c_int64, c_void_p, c_int64,
                                        c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_void_p]
        L.moe_fp8_quantize_rows.argtypes = [c_int32, c_void_p, c_int64, c_int64, c_int64, c_int32, c_void_p,
                                            c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                            ctypes.c_size_t, c_void_p]
        L.moe_fp8_gather_ws.argtypes = [c_int64, c_int32]
        L.moe_fp8_gather_ws.restype = ctypes.c_size_t
        L.moe_fp8_quantize_cols.argtypes = [c_int32, c_void_p, c_int64, c_int64, c_int64, c_int32, c_void_p,
                                            c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p]
        L.moe_fp8_quantize_blocks.argtypes = [c_int32, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p, c_int64,
                                              c_void_p, c_void_p]
        L.moe_fp8_gemm.argtypes = [c_int64, c_int64, c_int64, c_int32, P(MoeRouting), c_void_p, c_int64, c_void_p,
                                   c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p]
        L.moe_fp8_gemm_dw.argtypes = [c_int64, c_int64, c_int64, c_int32, P(MoeRouting), c_void_p, c_int64, c_void_p,
                                      c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p]
        L.moe_mx_quantize_rows.argtypes = [c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_void_p]
        L.moe_mx_quantize_cols.argtypes = [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p]
        L.moe_get_status.argtypes = [c_void_p, P(c_int32)]
        L.moe_set_spin_limit.argtypes = [c_int64]
        L.moe_selftest_wait_timeout.argtypes = [c_void_p, c_void_p]
        L.moe_profile_enable.argtypes = [c_int32]
        L.moe_profile_enable.restype = c_int32
        L.moe_profile_select.argtypes = [ctypes.c_char_p]
        L.moe_profile_select.restype = c_int32
        L.moe_profile_count.argtypes = []
        L.moe_profile_count.restype = c_int32
        L.moe_profile_read.argtypes = [c_int32, P(ctypes.c_char_p), P(ctypes.c_float)]
        L.moe_profile_read.restype = c_int32
        L.moe_trace_gemm.argtypes = [c_int32, c_void_p, c_int64]
        L.moe_trace_gemm.restype = c_int32
        L.moe_status_str.argtypes = [c_int32]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        for f in ("moe_query_sizes", "moe_route", "moe_token_round", "moe_forward", "moe_backward",
                  "moe_get_status", "moe_set_spin_limit", "moe_selftest_wait_timeout", "moe_backward_ev",
                  "moe_set_sm_budget", "moe_mx_quantize_rows", "moe_mx_quantize_cols", "moe_forward_mxfp8",
                  "moe_route_given", "moe_ep_pack", "moe_ep_combine", "moe_router_backward",
                  "moe_mx_quantize_weights", "moe_forward_mxfp8_q", "moe_sort_sizes", "moe_sort_pairs", "moe_permute",
                  "moe_permute_bwd", "moe_unpermute", "moe_unpermute_bwd", "moe_fp8_quantize_rows",
                  "moe_fp8_quantize_cols", "moe_fp8_quantize_blocks", "moe_fp8_gemm", "moe_fp8_gemm_dw"):
            getattr(L, f).restype = c_int32
        _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().moe_status_str(int(code)).decode()


def last_error() -> str:
    """The CUDA runtime error behind this thread's most recent MOE_ERR_CUDA."""
    return lib().moe_last_error().decode()


def _check(code: int, what: str):
    if code != MOE_OK:
        raise MoEError(code, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def dims_of(T, d, E, n, K) -> MoeDims:
    return MoeDims(int(T), int(d), int(E), int(n), int(K))


def opts_of(round_mode=0, router_grad=1, seed=0) -> MoeOpts:
    return MoeOpts(int(round_mode), int(router_grad), int(seed))


def query_sizes(dims: MoeDims, opts: MoeOpts) -> MoeSizes:
    s = MoeSizes()
    _check(lib().moe_query_sizes(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(s)), "moe_query_sizes")
    return s


@dataclass
class Routing:
    """Device buffers of a moe_routing, allocated with torch."""
    tensors: dict
    struct: MoeRouting
    # the pairs are moe_token_round's: in expert order, some of them not in topk_idx
    rounded: bool = False

    def __getitem__(self, k):
        return self.tensors[k]

    @classmethod
    def allocate(cls, dims: MoeDims, sizes: MoeSizes, device="cuda", with_logits: bool = True,
                 with_pair_ds: bool = False) -> "Routing":
        import torch
        T, E, K = dims.T, dims.E, dims.K
        P, R = sizes.P_max, sizes.R_max
        i32, f32 = torch.int32, torch.float32
        shapes = {"logits": ((T, E), f32), "probs": ((T, E), f32), "topk_idx": ((T, K), i32),
                  "topk_gate": ((T, K), f32), "tok_ptr": ((T + 1,), i32), "pair_expert": ((P,), i32),
                  "pair_gate": ((P,), f32), "pair_row": ((P,), i32), "counts": ((E,), i32),
                  "offsets": ((E + 1,), i32), "row_tok": ((R,), i32), "row_gate": ((R,), f32),
                  "tile_expert": ((R // 128,), i32)}
        t = {}
        for k, (shape, dt) in shapes.items():
            if k == "logits" and not with_logits:
                t[k] = None
                continue
            t[k] = torch.empty(shape, dtype=dt, device=device)
        t["pair_dS"] = torch.empty((P,), dtype=f32, device=device) if with_pair_ds else None
        st = MoeRouting(*[_ptr(t[k]) for k in _ROUTING_PTRS], P, R, _ptr(t["pair_dS"]))
        return cls(t, st)


def moe_route(dims, opts, X, Wr, bias, routing: Routing, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(Wr), _ptr(bias),
                           ctypes.byref(routing.struct), _ptr(ws), ws.numel() * ws.element_size(),
                           _stream(stream)), "moe_route")
    routing.rounded = False


def moe_route_given(dims, opts, routing: Routing, ws, stream=None):
    """Permutation of a caller-given selection (routing['topk_idx'],
    routing['topk_gate'] filled by the caller)."""
    _check(lib().moe_route_given(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(routing.struct), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "moe_route_given")
    routing.rounded = False


def moe_ep_pack(dims, opts, routing: Routing, src, send_rows, send_gate, pair_pos, ws, stream=None):
    _check(lib().moe_ep_pack(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(routing.struct), _ptr(src),
                             _ptr(send_rows), _ptr(send_gate), _ptr(pair_pos), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_ep_pack")


def moe_ep_combine(dims, opts, routing: Routing, pair_pos, rows, out, stream=None):
    _check(lib().moe_ep_combine(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(routing.struct),
                                _ptr(pair_pos), _ptr(rows), _ptr(out), _stream(stream)), "moe_ep_combine")


def moe_router_backward(dims, opts, X, Wr, routing: Routing, dS, pair_pos, dX, dWr, ws, stream=None):
    _check(lib().moe_router_backward(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(Wr),
                                     ctypes.byref(routing.struct), _ptr(dS), _ptr(pair_pos), _ptr(dX), _ptr(dWr),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_router_backward")


def moe_route_noalloc(dims, opts, X, Wr, bias, routing: Routing, stream=None):
    """moe_route without a workspace, for callers that cannot allocate device
    memory; its scratch is a 16 MiB static array in the library (see moe.h)."""
    _check(lib().moe_route_noalloc(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(Wr), _ptr(bias),
                                   ctypes.byref(routing.struct), _stream(stream)), "moe_route_noalloc")
    routing.rounded = False


def moe_token_round(dims, opts, routing: Routing, ws, stream=None):
    _check(lib().moe_token_round(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(routing.struct), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "moe_token_round")
    routing.rounded = True


def moe_forward(dims, opts, X, W1, W2, routing: Routing, O, H, ws, stream=None):
    _check(lib().moe_forward(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(W1), _ptr(W2),
                             ctypes.byref(routing.struct), _ptr(O), _ptr(H), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_forward")


def moe_forward_mxfp8(dims, opts, X, W1, W2, routing: Routing, O, H, ws, stream=None):
    _check(lib().moe_forward_mxfp8(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(W1), _ptr(W2),
                                   ctypes.byref(routing.struct), _ptr(O), _ptr(H), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "moe_forward_mxfp8")


def moe_mx_quantize_weights(dims, opts, W1, W2, wq, stream=None):
    _check(lib().moe_mx_quantize_weights(ctypes.byref(dims), ctypes.byref(opts), _ptr(W1), _ptr(W2), _ptr(wq),
                                         wq.numel() * wq.element_size(), _stream(stream)), "moe_mx_quantize_weights")


def moe_forward_mxfp8_q(dims, opts, X, wq, routing: Routing, O, H, ws, stream=None):
    _check(lib().moe_forward_mxfp8_q(ctypes.byref(dims), ctypes.byref(opts), _ptr(X), _ptr(wq),
                                     ctypes.byref(routing.struct), _ptr(O), _ptr(H), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "moe_forward_mxfp8_q")


def moe_backward(dims, opts, dO, X, Wr, W1, W2, routing: Routing, H, dX, dW1, dW2, dWr, ws, stream=None,
                 grad_events=None):
    """grad_events: None, or three torch.cuda.Event (or None) recorded once
    dW2, dW1 and dWr are final."""
    args = (ctypes.byref(dims), ctypes.byref(opts), _ptr(dO), _ptr(X), _ptr(Wr), _ptr(W1), _ptr(W2),
            ctypes.byref(routing.struct), _ptr(H), _ptr(dX), _ptr(dW1), _ptr(dW2), _ptr(dWr), _ptr(ws),
            ws.numel() * ws.element_size())
    if grad_events is None:
        _check(lib().moe_backward(*args, _stream(stream)), "moe_backward")
        return
    for e in grad_events:
        if e is not None and not e.cuda_event:  # torch creates its event on the first record
            e.record()
    evs = (c_void_p * 3)(*[None if e is None else e.cuda_event for e in grad_events])
    _check(lib().moe_backward_ev(*args, evs, _stream(stream)), "moe_backward_ev")


def mx_quantize_rows(x, stream=None):
    """x [rows, K] bf16 (device) -> (codes [rows, K] uint8, scales [rows, K/32]
    uint8): MXFP8 along each row."""
    import torch
    rows, K = x.shape
    codes = torch.empty(rows, K, dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=x.device)
    _check(lib().moe_mx_quantize_rows(_ptr(x), rows, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_mx_quantize_rows")
    return codes, scales


def mx_quantize_cols(w, stream=None):
    """w [E, K, N] bf16 (device) -> (codes [E, N, K] uint8, scales [E, N, K/32]
    uint8): MXFP8 along K for each column, transposed so that K is contiguous."""
    import torch
    E, K, N = w.shape
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device=w.device)
    _check(lib().moe_mx_quantize_cols(_ptr(w), E, K, N, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_mx_quantize_cols")
    return codes, scales


# ----------------------------------------------------------------------------
# Rows sorted by expert and back.  These check their tensors, allocate what the
# caller leaves out, and run on the tensors' device, on `stream` or its current
# stream.

_torch = None
_DTYPES = {}


def _th():
    """torch, imported on first use (an import statement in every one of these
    short calls adds up)."""
    global _torch
    if _torch is None:
        import torch
        _DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e4m3fn: 3})
        _torch = torch
    return _torch


def _dtype_code(t, what: str, most: int = 2) -> int:
    code = _DTYPES.get(t.dtype, 99)
    if code > most:
        raise TypeError(f"{what}: {t.dtype} is not supported")
    return code


def _shape2(t, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected two dimensions")
    return shape


def _matrix(t, name: str, rows: int, cols: int, device, dtype=None) -> int:
    """Check a [rows, cols] tensor with unit column stride; returns its row
    stride.  (Messages are made only for a refusal: these checks run before
    calls of a few microseconds.)"""
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if rows == 0 or cols == 0:
        return cols
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if rows == 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld} for {cols} columns)")
    return ld


def _elsewhere(device, stream) -> bool:
    """Does a call on tensors of `device` have to change the current device or
    stream?  (It then runs with them current, so that what it allocates belongs
    to the stream that uses it.)"""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}: a CUDA device is needed")
    return stream is not None or _torch._C._cuda_getDevice() != device.index


def _there(device, stream, fn, *args):
    """fn(*args) with `device` and `stream` (or the device's current stream) current."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
    with _torch.cuda.device(device):
        if stream is None:
            return fn(*args)
        with _torch.cuda.stream(stream):
            return fn(*args)


def _current(device) -> int:
    """Handle of the (current) device's current stream (without the Python object
    around it: 0.1 instead of 3.4 us)."""
    return _torch._C._cuda_getCurrentRawStream(device.index)


def sort_pairs(topk_idx, topk_gate, E: int, routing: Routing | None = None, ws=None, stream=None) -> Routing:
    """Sort the choices topk_idx [T, K] (int32; outside [0, E): dropped) with
    gates topk_gate [T, K] (fp32) by expert: see moe_sort_pairs in moe.h.  Both
    are read by this call alone.  A Routing of an earlier call with the same T, K
    and E can be given again as `routing`; it is overwritten.  ws: a uint8
    workspace of moe_sort_sizes' bytes (default: allocated); calls that may
    overlap need one each."""
    torch = _th()
    dev = topk_idx.device
    T, K = _shape2(topk_idx, "topk_idx")
    for t, name, dt in ((topk_idx, "topk_idx", torch.int32), (topk_gate, "topk_gate", torch.float32)):
        if _matrix(t, name, T, K, dev, dt) != K:
            raise ValueError(f"{name}: must be contiguous")
    if ws is not None and (ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous()):
        raise ValueError(f"ws: contiguous uint8 on {dev} expected")
    if _elsewhere(dev, stream):
        return _there(dev, stream, sort_pairs, topk_idx, topk_gate, E, routing, ws)
    if routing is None or ws is None:
        P, R, need = c_int64(0), c_int64(0), ctypes.c_size_t(0)
        _check(lib().moe_sort_sizes(T, E, K, ctypes.byref(P), ctypes.byref(R), ctypes.byref(need)), "moe_sort_sizes")
        if ws is None and need.value:
            ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        if routing is None:
            i32, f32 = torch.int32, torch.float32
            sizes = {"tok_ptr": (T + 1, i32), "pair_expert": (P.value, i32), "pair_gate": (P.value, f32),
                     "pair_row": (P.value, i32), "counts": (E, i32), "offsets": (E + 1, i32),
                     "row_tok": (R.value, i32), "row_gate": (R.value, f32), "tile_expert": (R.value // 128, i32),
                     "pair_slot": (P.value, i32)}
            # at least one element each, so that every pointer is one even without tokens
            whole = {k: torch.empty(max(n, 1), dtype=dt, device=dev) for k, (n, dt) in sizes.items()}
            st = MoeRouting(**{k: _ptr(t) for k, t in whole.items()}, P_max=P.value, R_max=R.value)
            routing = Routing({**{k: t[:sizes[k][0]] for k, t in whole.items()}, "logits": None, "probs": None,
                               "pair_dS": None}, st)
    r, st = routing.tensors, routing.struct
    if r.get("logits") is not None or r.get("probs") is not None:
        raise ValueError("routing: not one that sort_pairs made")
    if r["tok_ptr"].shape[0] != T + 1 or r["counts"].shape[0] != E or r["tok_ptr"].device != dev:
        raise ValueError("routing: made for another T, E or device")
    r["topk_idx"], r["topk_gate"] = topk_idx, topk_gate
    st.topk_idx, st.topk_gate = _ptr(topk_idx), _ptr(topk_gate)
    _check(lib().moe_sort_pairs(T, E, K, ctypes.byref(st), _ptr(ws), 0 if ws is None else ws.numel(),
                                _current(dev)), "moe_sort_pairs")
    return routing


def _routed(routing: Routing):
    """(T, E, R_max, device) of a routing."""
    r = routing.tensors
    tok_ptr = r["tok_ptr"]
    return tok_ptr.shape[0] - 1, r["counts"].shape[0], routing.struct.R_max, tok_ptr.device


def permute(routing: Routing, src, rows=None, stream=None):
    """rows [R_max, width]: src [T, width] in expert order, zeros in the padding
    rows.  Rows past the last expert's segment are left as they were (in a
    tensor allocated here: undefined)."""
    _th()
    T, E, R, dev = _routed(routing)
    code = _dtype_code(src, "src", 3)
    width = _shape2(src, "src")[1]
    ld = _matrix(src, "src", T, width, dev)
    if _elsewhere(dev, stream):
        return _there(dev, stream, permute, routing, src, rows)
    ldr = width
    if rows is None:
        rows = src.new_empty((R, width))
    else:
        ldr = _matrix(rows, "rows", R, width, dev, src.dtype)
    _check(lib().moe_permute(T, E, ctypes.byref(routing.struct), code, width, _ptr(src), ld, _ptr(rows), ldr,
                             _current(dev)), "moe_permute")
    return rows


def _sum_rows(fn, what, routing, rows, out, stream):
    _th()
    T, E, R, dev = _routed(routing)
    code = _dtype_code(rows, "rows")
    width = _shape2(rows, "rows")[1]
    ld = _matrix(rows, "rows", R, width, dev)
    if _elsewhere(dev, stream):
        return _there(dev, stream, _sum_rows, fn, what, routing, rows, out, None)
    ldo = width
    if out is None:
        out = rows.new_empty((T, width))
    else:
        ldo = _matrix(out, "out", T, width, dev, rows.dtype)
    _check(fn(T, E, ctypes.byref(routing.struct), code, width, _ptr(rows), ld, _ptr(out), ldo,
              _current(dev)), what)
    return out


def permute_bwd(routing: Routing, drows, dsrc=None, stream=None):
    """Gradient of permute: dsrc [T, width], each token's rows of drows summed."""
    return _sum_rows(lib().moe_permute_bwd, "moe_permute_bwd", routing, drows, dsrc, stream)


def unpermute(routing: Routing, rows, out=None, stream=None):
    """out [T, width]: each token's rows weighted by their gates and summed."""
    return _sum_rows(lib().moe_unpermute, "moe_unpermute", routing, rows, out, stream)


def unpermute_bwd(routing: Routing, dout, rows, drows=None, dgate=None, pairs: bool = False, stream=None):
    """Gradients of unpermute: (drows [R_max, width], dgate).  dgate is [T, K]
    in the places of the choices, 0 for dropped ones; with pairs=True it is
    [P_max] in pair order (for moe_token_round's routings), where entries past
    the pairs in use are left as they were."""
    torch = _th()
    T, E, R, dev = _routed(routing)
    code = _dtype_code(rows, "rows")
    width = _shape2(rows, "rows")[1]
    ld = _matrix(rows, "rows", R, width, dev)
    ldo = _matrix(dout, "dout", T, width, dev, rows.dtype)
    K = routing.tensors["topk_idx"].shape[1]
    if not pairs and (routing.rounded or routing.struct.P_max != T * K):
        raise ValueError("a routing with token rounding has no place per choice: pass pairs=True")
    if drows is not None and drows.data_ptr() == rows.data_ptr() and drows.numel():
        raise ValueError("drows: must not be rows")
    if _elsewhere(dev, stream):
        return _there(dev, stream, unpermute_bwd, routing, dout, rows, drows, dgate, pairs)
    ldd = width
    if drows is None:
        drows = rows.new_empty((R, width))
    else:
        ldd = _matrix(drows, "drows", R, width, dev, rows.dtype)
    shape = (routing.struct.P_max,) if pairs else (T, K)
    if dgate is None:
        dgate = torch.empty(shape, dtype=torch.float32, device=dev)
    elif dgate.dtype != torch.float32:
        raise TypeError(f"dgate: {dgate.dtype}, expected torch.float32")
    elif dgate.shape != shape or dgate.device != dev or not dgate.is_contiguous():
        raise ValueError(f"dgate: contiguous {shape} on {dev} expected")
    _check(lib().moe_unpermute_bwd(T, E, K, ctypes.byref(routing.struct), code, width, _ptr(dout), ldo, _ptr(rows),
                                   ld, _ptr(drows), ldd, _ptr(dgate) if pairs else None,
                                   None if pairs else _ptr(dgate), _current(dev)), "moe_unpermute_bwd")
    return drows, dgate


# ----------------------------------------------------------------------------
# 8-bit products with one fp32 scale per block of 128 (moe_fp8_* in moe.h).
# Codes are float8_e4m3fn tensors whose rows are 16-byte aligned; those
# allocated here have a row stride of the next multiple of 16.


def _new_codes(lead, cols: int, device):
    torch = _th()
    ld = (cols + 15) // 16 * 16
    codes = torch.empty((*lead, ld), dtype=torch.float8_e4m3fn, device=device)
    return codes if ld == cols else codes[..., :cols]


def _codes(t, name: str, rows: int, cols: int, device) -> int:
    ld = _matrix(t, name, rows, cols, device, _torch.float8_e4m3fn)
    if rows <= 1:
        ld = (cols + 15) // 16 * 16
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must be 16-byte aligned (row stride {ld})")
    return ld


def _i32(t, name: str, n: int, device):
    if t is None:
        return None
    if t.dtype != _torch.int32:
        raise TypeError(f"{name}: {t.dtype}, expected torch.int32")
    if t.device != device or t.dim() != 1 or t.shape[0] < n or (t.shape[0] > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: {n} contiguous values on {device} expected")
    return _ptr(t)


def _quantize(cols_form, x, row_src, rows_used, swiglu, codes, scales, stream):
    torch = _th()
    code = _dtype_code(x, "x")
    n_in, width = _shape2(x, "x")
    dev = x.device
    ld = _matrix(x, "x", n_in, width, dev)
    if swiglu and width % 2:
        raise ValueError(f"x: {width} columns, expected gate and up halves")
    cols = width // 2 if swiglu else width
    rows = n_in if row_src is None else row_src.shape[0]
    src = _i32(row_src, "row_src", rows, dev)
    used = _i32(rows_used, "rows_used", 1, dev)
    if _elsewhere(dev, stream):
        return _there(dev, stream, _quantize, cols_form, x, row_src, rows_used, swiglu, codes, scales, None)
    out, blocks = ((cols, rows), -(-rows // 128)) if cols_form else ((rows, cols), -(-cols // 128))
    ldc, lds = (out[1] + 15) // 16 * 16, out[0]
    if codes is None:
        codes = _new_codes(out[:1], out[1], dev)
    else:
        ldc = _codes(codes, "codes", *out, dev)
    if scales is None:
        scales = torch.empty((blocks, lds), dtype=torch.float32, device=dev)
    else:
        lds = _matrix(scales, "scales", blocks, lds, dev, torch.float32)
    if cols_form:
        _check(lib().moe_fp8_quantize_cols(code, _ptr(x), ld, n_in, rows, cols, src, used, _ptr(codes), ldc,
                                           _ptr(scales), lds, _current(dev)), "moe_fp8_quantize_cols")
    else:
        ws, need = None, 0
        # Rows that repeat often are quantized once and their codes copied (us, row by
        # row / once: 32 x 7168 to 32768 rows 57 / 29, 4096 x 7168 to 65280 128 / 94);
        # not with few repeats (4096 x 7168 to 16384: 34 / 38) or little to copy
        # (1 x 2048 to 1024: 2.1 / 3.8, to 8192: 5.1 / 5.4).  The rows in use are
        # not known here; where they are few it still pays, since the blocks of
        # the others are fewer (512 x 2048 to 512 of 33024: 9.5 / 6.7,
        # 64 x 7168 to 1024 of 33024: 31 / 7.9).
        if src is not None and rows >= 6 * n_in > 0 and rows * cols > 1 << 24:
            need = lib().moe_fp8_gather_ws(n_in, cols)
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _check(lib().moe_fp8_quantize_rows(code, _ptr(x), ld, n_in, rows, cols, src, used, 1 if swiglu else 0,
                                           _ptr(codes), ldc, _ptr(scales), lds, _ptr(ws), need, _current(dev)),
               "moe_fp8_quantize_rows")
    return codes, scales


def fp8_quantize_rows(x, row_src=None, rows_used=None, swiglu: bool = False, codes=None, scales=None, stream=None):
    """x [rows, cols] -> (codes [rows, cols], scales [ceil(cols / 128), rows]).
    row_src [R] int32: row r of the result holds x[row_src[r]], zeros where that
    is no row of x (-1).  rows_used: a device int32; rows from there on are left
    as they were.  swiglu: x is [rows, 2 cols] and
    silu(x[:, :cols]) * x[:, cols:] is quantized."""
    return _quantize(False, x, row_src, rows_used, swiglu, codes, scales, stream)


def fp8_quantize_cols(x, row_src=None, rows_used=None, codes=None, scales=None, stream=None):
    """x [rows, cols] -> (codes [cols, rows], scales [ceil(rows / 128), cols]):
    one scale per column and 128 rows, codes transposed.  row_src and rows_used
    as in fp8_quantize_rows.  At most 65535 x 128 rows."""
    return _quantize(True, x, row_src, rows_used, False, codes, scales, stream)


def fp8_quantize_blocks(w, transpose: bool, codes=None, scales=None, stream=None):
    """w [E, K, N] or [K, N] (contiguous) -> codes and one scale per 128 x 128
    block: [.., K, N] and [.., ceil(K/128), ceil(N/128)], or with transpose
    [.., N, K] and [.., ceil(N/128), ceil(K/128)]."""
    torch = _th()
    code = _dtype_code(w, "w")
    if w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError(f"w: a contiguous [E, K, N] or [K, N] expected, got {tuple(w.shape)}")
    dev = w.device
    K, N = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    if _elsewhere(dev, stream):
        return _there(dev, stream, fp8_quantize_blocks, w, transpose, codes, scales)
    a, b = (N, K) if transpose else (K, N)
    lead = w.shape[:-2]
    if codes is None:
        codes = _new_codes((*lead, a), b, dev)
    if scales is None:
        scales = torch.empty(*lead, -(-a // 128), -(-b // 128), dtype=torch.float32, device=dev)
    ldc = _planes(codes, "codes", (*lead, a, b), dev)
    if scales.shape != (*lead, -(-a // 128), -(-b // 128)) or not scales.is_contiguous() or scales.device != dev:
        raise ValueError(f"scales: contiguous {(*lead, -(-a // 128), -(-b // 128))} on {dev} expected")
    if scales.dtype != torch.float32:
        raise TypeError(f"scales: {scales.dtype}, expected torch.float32")
    _check(lib().moe_fp8_quantize_blocks(code, _ptr(w), E, K, N, 1 if transpose else 0, _ptr(codes), ldc, _ptr(scales),
                                         _current(dev)), "moe_fp8_quantize_blocks")
    return codes, scales


def _planes(t, name: str, shape, device) -> int:
    """Check codes [rows, cols] or [E, rows, cols] without gaps between planes;
    returns the row stride."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if len(shape) == 2:
        return _codes(t, name, *shape, device)
    if shape[0] == 0:
        return (shape[2] + 15) // 16 * 16
    ld = _codes(t[0], name, shape[1], shape[2], device)
    if shape[0] > 1 and t.stride(0) != shape[1] * ld:
        raise ValueError(f"{name}: planes must follow one another (stride {t.stride(0)}, expected {shape[1] * ld})")
    return ld


def _out(out, name, shape, device):
    """bf16 result [.., rows, cols], its rows 16-byte aligned; returns (tensor, row stride)."""
    torch = _torch
    if out is None:
        ld = (shape[-1] + 7) // 8 * 8
        out = torch.empty((*shape[:-1], ld), dtype=torch.bfloat16, device=device)
        return out if ld == shape[-1] else out[..., :shape[-1]], ld
    if out.shape != shape:
        raise ValueError(f"{name}: shape {tuple(out.shape)}, expected {tuple(shape)}")
    flat = out if len(shape) == 2 else out[0]
    ld = _matrix(flat, name, shape[-2], shape[-1], device, torch.bfloat16)
    if shape[-2] <= 1:
        ld = (shape[-1] + 7) // 8 * 8
    if ld % 8 or out.data_ptr() % 16:
        raise ValueError(f"{name}: rows must be 16-byte aligned (row stride {ld})")
    if len(shape) == 3 and shape[0] > 1 and out.stride(0) != shape[1] * ld:
        raise ValueError(f"{name}: planes must follow one another")
    return out, ld


def fp8_gemm(a, sa, b, sb, routing: Routing | None = None, out=None, stream=None):
    """out [M, N] bf16 = a [M, K] times b [N, K] transposed, codes with their
    scales sa [ceil(K/128), M] and sb [ceil(N/128), ceil(K/128)].  With a
    routing: a [R_max, K] in expert order, b [E, N, K], sb [E, .., ..]; rows
    past the last segment are left as they were (undefined in a new tensor)."""
    torch = _th()
    dev = a.device
    M, K = _shape2(a, "a")
    lda = _codes(a, "a", M, K, dev)
    if routing is None:
        E, lead = 1, ()
    else:
        _, E, R, rdev = _routed(routing)
        lead = (E,)
        if M != R or rdev != dev:
            raise ValueError(f"a: {M} rows on {dev}, expected the routing's {R} on {rdev}")
    if b.dim() != 2 + len(lead):
        raise ValueError(f"b: shape {tuple(b.shape)}, expected {'[E, N, K]' if lead else '[N, K]'}")
    N = b.shape[-2]
    ldb = _planes(b, "b", (*lead, N, K), dev)
    nb, kb = (N + 127) // 128, (K + 127) // 128
    lds = _matrix(sa, "sa", kb, M, dev, torch.float32)
    if sb.shape != (*lead, nb, kb) or sb.device != dev or not sb.is_contiguous():
        raise ValueError(f"sb: contiguous {(*lead, nb, kb)} on {dev} expected, got {tuple(sb.shape)}")
    if sb.dtype != torch.float32:
        raise TypeError(f"sb: {sb.dtype}, expected torch.float32")
    if _elsewhere(dev, stream):
        return _there(dev, stream, fp8_gemm, a, sa, b, sb, routing, out)
    out, ldo = _out(out, "out", (M, N), dev)
    _check(lib().moe_fp8_gemm(M, N, K, E, None if routing is None else ctypes.byref(routing.struct), _ptr(a), lda,
                              _ptr(sa), lds, _ptr(b), ldb, _ptr(sb), _ptr(out), ldo, _current(dev)),
           "moe_fp8_gemm")
    return out


def fp8_gemm_dw(a, sa, b, sb, routing: Routing | None = None, out=None, stream=None):
    """Weight gradient out [M, N] bf16 = a [M, tokens] times b [N, tokens]
    transposed, both as fp8_quantize_cols leaves them (sa [ceil(tokens/128), M],
    sb [.., N]).  With a routing the tokens are its rows and out is [E, M, N],
    each expert's product over its own rows."""
    torch = _th()
    dev = a.device
    M, K = _shape2(a, "a")
    N = _shape2(b, "b")[0]
    lda, ldb = _codes(a, "a", M, K, dev), _codes(b, "b", N, K, dev)
    kb = (K + 127) // 128
    ldsa = _matrix(sa, "sa", kb, M, dev, torch.float32)
    ldsb = _matrix(sb, "sb", kb, N, dev, torch.float32)
    if routing is None:
        E, lead = 1, ()
    else:
        _, E, R, rdev = _routed(routing)
        lead = (E,)
        if K != R or rdev != dev:
            raise ValueError(f"a: {K} tokens on {dev}, expected the routing's {R} rows on {rdev}")
    if _elsewhere(dev, stream):
        return _there(dev, stream, fp8_gemm_dw, a, sa, b, sb, routing, out)
    out, ldo = _out(out, "out", (*lead, M, N), dev)
    _check(lib().moe_fp8_gemm_dw(M, N, K, E, None if routing is None else ctypes.byref(routing.struct), _ptr(a), lda,
                                 _ptr(sa), ldsa, _ptr(b), ldb, _ptr(sb), ldsb, _ptr(out), ldo, _current(dev)),
           "moe_fp8_gemm_dw")
    return out


def moe_set_sm_budget(sms: int):
    """At most `sms` CTAs per persistent GEMM (0: one per SM)."""
    _check(lib().moe_set_sm_budget(int(sms)), "moe_set_sm_budget")


def moe_get_status(stream=None) -> tuple[int, int]:
    where = c_int32(0)
    code = lib().moe_get_status(_stream(stream), ctypes.byref(where))
    return int(code), int(where.value)


def moe_set_spin_limit(cycles: int):
    _check(lib().moe_set_spin_limit(int(cycles)), "moe_set_spin_limit")


def moe_selftest_wait_timeout(flag, stream=None):
    _check(lib().moe_selftest_wait_timeout(_ptr(flag), _stream(stream)), "moe_selftest_wait_timeout")


def moe_profile_enable(on: bool):
    _check(lib().moe_profile_enable(1 if on else 0), "moe_profile_enable")


def moe_profile_select(name: str | None):
    """Record only launches of `name` (None: record every launch)."""
    _check(lib().moe_profile_select(None if name is None else name.encode()), "moe_profile_select")


def moe_profile_records() -> list[tuple[str, float]]:
    """(kernel name, ms) of every launch recorded since moe_profile_enable(True);
    the streams must have completed."""
    L = lib()
    out = []
    name = ctypes.c_char_p()
    ms = ctypes.c_float()
    for i in range(L.moe_profile_count()):
        _check(L.moe_profile_read(i, ctypes.byref(name), ctypes.byref(ms)), "moe_profile_read")
        out.append((name.value.decode(), float(ms.value)))
    return out


GEMM_KINDS = {"up_proj_gemm": 0, "down_proj_gemm": 1, "dh_gemm": 2, "dxt_gemm": 3, "dw1_gemm": 4, "dw2_gemm": 5,
              "router_logits_gemm": 6, "router_dwr_gemm": 7, "up_proj_gemm_mx": 8, "down_proj_gemm_mx": 9}


class GemmTrace:
    """Role timeline of one grouped-GEMM kind (moe_trace_gemm): start() before
    the launches to trace, stop() after them, then records() gives one numpy
    structured array per (CTA, role) with fields ns, clk, tile, event."""

    ROLES = ("producer", "mma", "epilogue", "gather")

    def __init__(self, kernel: str, records_per_role: int = 4096, device="cuda"):
        import torch
        self.kind = GEMM_KINDS[kernel]
        self.cap = int(records_per_role)
        sms = torch.cuda.get_device_properties(torch.device(device)).multi_processor_count
        self.ctas = sms
        self.buf = torch.zeros(self.ctas * 4 * self.cap * 16, dtype=torch.uint8, device=device)

    def start(self):
        self.buf.zero_()
        _check(lib().moe_trace_gemm(self.kind, _ptr(self.buf), self.cap), "moe_trace_gemm")

    def stop(self):
        _check(lib().moe_trace_gemm(-1, None, 0), "moe_trace_gemm")

    def records(self):
        import numpy as np
        raw = self.buf.cpu().numpy()
        dt = np.dtype([("ns", "<u8"), ("clk", "<u4"), ("info", "<u4")])
        rec = raw.view(dt).reshape(self.ctas, 4, self.cap)
        out = {}
        for c in range(self.ctas):
            for r in range(4):
                x = rec[c, r]
                x = x[x["ns"] != 0]
                out[(c, self.ROLES[r])] = {"ns": x["ns"].astype(np.int64), "clk": x["clk"].astype(np.int64),
                                           "tile": (x["info"] >> 8).astype(np.int64),
                                           "event": (x["info"] & 0xFF).astype(np.int64)}
        return out


class MoELayer:
    """All device buffers of one layer shape, allocated once with torch; each
    method is one library call."""

    def __init__(self, T, d, E, n, K, round_mode=0, router_grad=1, seed=0, device="cuda"):
        import torch
        self.dims = dims_of(T, d, E, n, K)
        self.opts = opts_of(round_mode, router_grad, seed)
        self.sizes = query_sizes(self.dims, self.opts)
        self.device = device
        self.routing = Routing.allocate(self.dims, self.sizes, device)
        u8, bf = torch.uint8, torch.bfloat16
        self.ws_route = torch.empty(self.sizes.route_ws, dtype=u8, device=device)
        self.ws_fwd = torch.empty(self.sizes.fwd_ws, dtype=u8, device=device)
        self.ws_bwd = torch.empty(self.sizes.bwd_ws, dtype=u8, device=device)
        self.ws_fwd_mx = None   # MXFP8 forward workspace, allocated on first use
        self.ws_fp8 = None      # buffers of forward_fp8, allocated on first use
        self.mxfp8 = False      # default precision of forward(): MXFP8 GEMM operands when True
        self.H = torch.empty(self.sizes.R_max, 2 * n, dtype=bf, device=device)
        self.O = torch.empty(T, d, dtype=bf, device=device)
        self.dX = torch.empty(T, d, dtype=bf, device=device)
        self.dW1 = torch.empty(E, d, 2 * n, dtype=bf, device=device)
        self.dW2 = torch.empty(E, n, d, dtype=bf, device=device)
        self.dWr = torch.empty(d, E, dtype=torch.float32, device=device)

    def _bytes(self, n, stream):
        """Memory that belongs to the stream that uses it (None: the current one)."""
        torch = _th()
        with torch.cuda.stream(stream):
            return torch.empty(n, dtype=torch.uint8, device=self.device)

    def route(self, X, Wr, bias=None, stream=None):
        moe_route(self.dims, self.opts, X, Wr, bias, self.routing, self.ws_route, stream)
        if self.opts.round_mode:
            moe_token_round(self.dims, self.opts, self.routing, self.ws_route, stream)

    def forward(self, X, W1, W2, stream=None, O=None, mxfp8=None):
        O = self.O if O is None else O
        if self.mxfp8 if mxfp8 is None else mxfp8:
            if self.ws_fwd_mx is None:
                if self.sizes.fwd_mx_ws == 0:
                    raise MoEError(2, "moe_forward_mxfp8 (needs n % 128 == 0)")
                self.ws_fwd_mx = self._bytes(self.sizes.fwd_mx_ws, stream)
            moe_forward_mxfp8(self.dims, self.opts, X, W1, W2, self.routing, O, self.H, self.ws_fwd_mx, stream)
        else:
            moe_forward(self.dims, self.opts, X, W1, W2, self.routing, O, self.H, self.ws_fwd, stream)
        return O

    def quantize_weights_mxfp8(self, W1, W2, stream=None):
        """MXFP8 copy of W1, W2 for forward_mxfp8_q (weights that stay fixed)."""
        if self.sizes.mx_weights_bytes == 0:
            raise MoEError(2, "moe_mx_quantize_weights (needs n % 128 == 0)")
        wq = self._bytes(self.sizes.mx_weights_bytes, stream)
        moe_mx_quantize_weights(self.dims, self.opts, W1, W2, wq, stream)
        return wq

    def forward_mxfp8_q(self, X, wq, stream=None, O=None):
        """The MXFP8 forward on weights quantized once by quantize_weights_mxfp8."""
        O = self.O if O is None else O
        if self.ws_fwd_mx is None:
            self.ws_fwd_mx = self._bytes(self.sizes.fwd_mx_ws, stream)
        moe_forward_mxfp8_q(self.dims, self.opts, X, wq, self.routing, O, self.H, self.ws_fwd_mx, stream)
        return O

    def quantize_weights_fp8(self, W1, W2, stream=None):
        """E4M3 copy of W1, W2 with a scale per 128 x 128 block, for forward_fp8."""
        return (*fp8_quantize_blocks(W1, transpose=True, stream=stream),
                *fp8_quantize_blocks(W2, transpose=True, stream=stream))

    def forward_fp8(self, X, wq, stream=None, O=None):
        """The forward with 8-bit products on the weights of quantize_weights_fp8:
        X is quantized into expert order and A = SwiGLU(H) per row, with an fp32
        scale per 128 values.  O and the saved H (bf16) as forward leaves them, so
        that backward follows unchanged."""
        torch = _th()
        if _elsewhere(X.device, stream):
            return _there(X.device, stream, self.forward_fp8, X, wq, None, O)
        rt, (w1, s1, w2, s2) = self.routing, wq
        O = self.O if O is None else O
        d, n, R = self.dims.d, self.dims.n, self.sizes.R_max
        if self.ws_fp8 is None:
            dev = X.device
            self.ws_fp8 = {
                "x": _new_codes((R,), d, dev), "sx": torch.empty(-(-d // 128), R, dtype=torch.float32, device=dev),
                "a": _new_codes((R,), n, dev), "sa": torch.empty(-(-n // 128), R, dtype=torch.float32, device=dev),
                "Y": torch.empty(R, d, dtype=torch.bfloat16, device=dev)}
        b, used = self.ws_fp8, rt["offsets"][self.dims.E:]
        fp8_quantize_rows(X, row_src=rt["row_tok"], rows_used=used, codes=b["x"], scales=b["sx"])
        fp8_gemm(b["x"], b["sx"], w1, s1, routing=rt, out=self.H)
        fp8_quantize_rows(self.H, rows_used=used, swiglu=True, codes=b["a"], scales=b["sa"])
        fp8_gemm(b["a"], b["sa"], w2, s2, routing=rt, out=b["Y"])
        return unpermute(rt, b["Y"], out=O)

    def backward(self, dO, X, Wr, W1, W2, stream=None, grad_events=None, dX=None):
        """dX: output buffer [T, d] bf16 (default: self.dX)."""
        dX = self.dX if dX is None else dX
        moe_backward(self.dims, self.opts, dO, X, Wr, W1, W2, self.routing, self.H, dX, self.dW1, self.dW2,
                     self.dWr if self.opts.router_grad else None, self.ws_bwd, stream, grad_events)
        return dX, self.dW1, self.dW2, self.dWr

    def step(self, X, Wr, bias, W1, W2, dO, stream=None, grad_events=None):
        """One pass of the whole path: route (+ rounding), forward, backward."""
        self.route(X, Wr, bias, stream)
        self.forward(X, W1, W2, stream)
        return self.backward(dO, X, Wr, W1, W2, stream, grad_events)


class CudaStreamHooks:
    """Stream and event plumbing of OverlappedGradReduce on a CUDA device:
    three events the backward records (dW2, dW1, dWr written), and a
    communication stream that waits on each before its all-reduce."""

    def __init__(self):
        import torch
        self.comm = torch.cuda.Stream()
        self.events = [torch.cuda.Event() for _ in range(3)]

    def on_comm(self):
        import torch
        return torch.cuda.stream(self.comm)

    def wait(self, ev):
        self.comm.wait_event(ev)

    def join(self):
        import torch
        torch.cuda.current_stream().wait_stream(self.comm)


class OverlappedGradReduce:
    """Data-parallel steps whose weight-gradient sums over `group` overlap the
    backward.  The backward records an event as soon as dW2, then dW1, then dWr
    are written (moe_backward_ev computes dW2 and dW1 before dX~); each
    all-reduce waits on its event on a separate stream, so the reductions of
    dW2 and dW1 run while the dX~ GEMM and the dX aggregation do.  The current
    stream waits for the reductions at the end of the step, before the next
    step can overwrite the gradients.

    `hooks` supplies the streams and events (CudaStreamHooks by default); the
    CPU tests pass host stand-ins so that the ordering logic runs on gloo
    ranks."""

    def __init__(self, layer, group=None, hooks=None):
        self.layer = layer
        self.group = group
        self.hooks = hooks if hooks is not None else CudaStreamHooks()

    def step(self, X, Wr, bias, W1, W2, dO):
        import torch.distributed as dist
        L = self.layer
        h = self.hooks
        L.step(X, Wr, bias, W1, W2, dO, grad_events=h.events)
        grads = (L.dW2, L.dW1, L.dWr if L.opts.router_grad else None)
        with h.on_comm():
            for ev, g in zip(h.events, grads):
                if g is None:
                    continue
                h.wait(ev)
                dist.all_reduce(g, group=self.group)
        h.join()
        return L.dX, L.dW1, L.dW2, L.dWr


class HostFedRunner:
    """Whole steps (route, forward, backward) on batches held in pinned host
    memory.  Each step's inputs X and dO are copied to the device on a copy
    stream; its per-token outputs O and dX are copied back on a second copy
    stream, O as soon as the forward is done and dX after the backward, so the
    copies of consecutive steps overlap with the kernels.  Device input and
    output buffers alternate between two sets; events keep a buffer from being
    overwritten while a step or a copy still uses it.  Weight gradients stay
    on the device (layer.dW1, layer.dW2, layer.dWr)."""

    def __init__(self, layer: MoELayer):
        import torch
        T, d = layer.dims.T, layer.dims.d
        dev = layer.device
        bf = torch.bfloat16
        self.layer = layer
        self.X = [torch.empty(T, d, dtype=bf, device=dev) for _ in range(2)]
        self.dO = [torch.empty(T, d, dtype=bf, device=dev) for _ in range(2)]
        self.O = [torch.empty(T, d, dtype=bf, device=dev) for _ in range(2)]
        self.dX = [torch.empty(T, d, dtype=bf, device=dev) for _ in range(2)]
        self.h2d = torch.cuda.Stream(device=dev)
        self.d2h = torch.cuda.Stream(device=dev)
        ev = torch.cuda.Event
        self.inputs_ready = [ev(), ev()]
        self.inputs_free = [ev(), ev()]
        self.fwd_done = [ev(), ev()]
        self.bwd_done = [ev(), ev()]
        self.out_free = [ev(), ev()]
        self.i = 0

    def step(self, Xh, dOh, Oh, Wr, bias, W1, W2, dXh=None):
        """Enqueue one step; Xh, dOh, Oh (and dXh, if given) are pinned host
        tensors [T, d] bf16.  Returns immediately; call finish() before
        reading Oh or dXh.  Without dXh the step's dX stays on the device
        (the buffer of this step's set, self.dX[step % 2])."""
        import torch
        j = self.i & 1
        compute = torch.cuda.current_stream()
        L = self.layer
        with torch.cuda.stream(self.h2d):
            self.h2d.wait_event(self.inputs_free[j])
            self.X[j].copy_(Xh, non_blocking=True)
            self.dO[j].copy_(dOh, non_blocking=True)
            self.inputs_ready[j].record(self.h2d)
        compute.wait_event(self.inputs_ready[j])
        compute.wait_event(self.out_free[j])
        L.route(self.X[j], Wr, bias)
        L.forward(self.X[j], W1, W2, O=self.O[j])
        self.fwd_done[j].record(compute)
        with torch.cuda.stream(self.d2h):
            self.d2h.wait_event(self.fwd_done[j])
            Oh.copy_(self.O[j], non_blocking=True)
        L.backward(self.dO[j], self.X[j], Wr, W1, W2, dX=self.dX[j])
        self.inputs_free[j].record(compute)
        self.bwd_done[j].record(compute)
        with torch.cuda.stream(self.d2h):
            if dXh is not None:
                self.d2h.wait_event(self.bwd_done[j])
                dXh.copy_(self.dX[j], non_blocking=True)
            self.out_free[j].record(self.d2h)
        self.i += 1

    def finish(self):
        """Make the current stream wait for every copy enqueued so far."""
        import torch
        compute = torch.cuda.current_stream()
        compute.wait_stream(self.h2d)
        compute.wait_stream(self.d2h)
