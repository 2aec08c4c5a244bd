"""Python binding of libmoe_b200.so, the sm_100a hard-routed sparse MoE
layer forward.

Argument marshalling only: every function here checks shapes and dtypes,
allocates outputs with PyTorch on the inputs' device, passes raw device
pointers and the current CUDA stream to the C ABI (``include/moe.h``), and
raises on a non-OK status. `stream=` makes a call as under
``torch.cuda.stream(stream)``; the caller orders its own reads after that
stream's work. All arithmetic runs in the library's CUDA
kernels; there is no CPU path. Importing this module fails loudly if the
library is missing or cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_RANGE = range(7)
F32, BF16, F16 = 0, 1, 2
W_F32, W_BF16, W_Q4G64 = 0, 1, 2
REGIME_AUTO, REGIME_GEMV, REGIME_TC = 0, 1, 2

EXPORTS = ("moe_route", "moe_topk", "moe_sort_rows_workspace", "moe_sort_rows",
           "moe_sort_rows_noalloc", "moe_sort_block_m",
           "moe_grouped_swiglu_workspace", "moe_grouped_swiglu", "moe_grouped_down",
           "moe_combine", "moe_forward_workspace", "moe_pack_gate_up",
           "moe_forward", "moe_forward_layout", "moe_device_status", "moe_status_str",
           "moe_version", "moe_set_wait_cycles", "moe_selftest_wait_timeout",
           "moe_quantize_fp8", "moe_fp8_matmul", "moe_grouped_swiglu_fp8",
           "moe_grouped_down_fp8", "moe_balance_loss_workspace", "moe_balance_loss",
           "moe_balance_loss_backward")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} (status {status})")
        self.status = status


class Experts(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("E", ctypes.c_int32), ("d", ctypes.c_int32),
                ("F", ctypes.c_int32), ("w_gu", ctypes.c_void_p), ("s_gu", ctypes.c_void_p),
                ("b_gu", ctypes.c_void_p), ("w_dn", ctypes.c_void_p), ("s_dn", ctypes.c_void_p),
                ("b_dn", ctypes.c_void_p), ("act", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("logits", "topk_idx", "topk_w", "order", "inv_order", "row_map", "counts",
                 "row_off", "tile_off", "sort_ws", "h", "ys", "x16", "total")] + \
               [("regime", ctypes.c_int32), ("BM", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python sparse_mixture_experts_top_b200/build.py` (needs nvcc)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.moe_route.argtypes = [P, I, P, P, I, I, I, I, P, P, P, P]
    L.moe_topk.argtypes = [P, I, I, I, P, P, P]
    L.moe_sort_rows_workspace.argtypes = [I, I, I]
    L.moe_sort_rows_workspace.restype = S
    L.moe_sort_rows.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, S, P]
    L.moe_grouped_swiglu_workspace.argtypes = [I, I, I, I]
    L.moe_grouped_swiglu_workspace.restype = S
    L.moe_grouped_swiglu.argtypes = [P, I, P, P, P, I, I, I, ctypes.POINTER(Experts), P, P, S, I,
                                     P]
    L.moe_grouped_down.argtypes = [P, I, P, P, I, I, I, ctypes.POINTER(Experts), P, I, P]
    L.moe_combine.argtypes = [P, P, P, I, I, I, I, P, P]
    L.moe_forward_workspace.argtypes = [I, I, I, I, I, I, I, I]
    L.moe_forward_workspace.restype = S
    L.moe_forward.argtypes = [P, I, P, P, ctypes.POINTER(Experts), I, I, P, P, S, I, P]
    L.moe_forward_layout.argtypes = [I, I, I, I, I, I, I, I, ctypes.POINTER(WsLayout)]
    L.moe_sort_block_m.argtypes = []
    L.moe_sort_block_m.restype = ctypes.c_int
    L.moe_sort_rows_noalloc.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P]
    L.moe_pack_gate_up.argtypes = [I, I, I, I, P, P, P, P, P, P, P, P, P, P]
    L.moe_pack_gate_up.restype = ctypes.c_int
    L.moe_device_status.argtypes = []
    L.moe_set_wait_cycles.argtypes = [ctypes.c_longlong]
    L.moe_set_wait_cycles.restype = ctypes.c_int
    L.moe_selftest_wait_timeout.argtypes = [I, ctypes.c_longlong, P, P]
    L.moe_selftest_wait_timeout.restype = ctypes.c_int
    L.moe_status_str.argtypes = [I]
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_version.restype = ctypes.c_char_p
    f32 = ctypes.c_float
    L.moe_quantize_fp8.argtypes = [P, I, I, I, I, P, P, P]
    L.moe_fp8_matmul.argtypes = [P, P, P, P, I, I, I, I, P, P]
    L.moe_grouped_swiglu_fp8.argtypes = [P, P, P, P, P, I, I, I, ctypes.POINTER(Experts), P, P, I,
                                         P]
    L.moe_grouped_down_fp8.argtypes = [P, P, P, P, I, I, I, ctypes.POINTER(Experts), P, I, P]
    L.moe_balance_loss_workspace.argtypes = [I, I, I]
    L.moe_balance_loss_workspace.restype = S
    L.moe_balance_loss.argtypes = [P, P, P, P, I, I, I, I, f32, P, P, P, P, P, S, P]
    L.moe_balance_loss_backward.argtypes = [P, P, P, I, I, I, I, f32, P, P, P, P, P]
    for name in ("moe_quantize_fp8", "moe_fp8_matmul", "moe_grouped_swiglu_fp8",
                 "moe_grouped_down_fp8", "moe_balance_loss", "moe_balance_loss_backward"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("moe_route", "moe_topk", "moe_sort_rows", "moe_sort_rows_noalloc",
                 "moe_grouped_swiglu",
                 "moe_grouped_down", "moe_combine", "moe_forward", "moe_forward_layout",
                 "moe_device_status"):
        getattr(L, name).restype = ctypes.c_int
    return L


lib = _load()


def status_str(s: int) -> str:
    return lib.moe_status_str(s).decode()


def version() -> str:
    return lib.moe_version().decode()


def _check(st: int, what: str):
    if st != OK:
        raise MoeError(st, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _under(stream, call, *args, **kw):
    """`stream=` of a call: the call as made under torch.cuda.stream(stream), so
    that the allocator hands out, and takes back, on that stream what the call
    writes there. (A block of the current stream's pool may still be in use by
    that stream's pending kernels, a call's scratch above all.) The outputs are
    recorded for the caller's stream too: one that is read there, and dropped, is
    not handed out again before that read."""
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    if caller != stream:
        outs = (out,) if torch.is_tensor(out) else out if type(out) is tuple else vars(out).values()
        for t in outs:
            if torch.is_tensor(t):
                t.record_stream(caller)
    return out


_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _dt_of(dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"activations must be bfloat16, float16 or float32, got {dtype}")
    return _DT[dtype]


def _dt(t: torch.Tensor) -> int:
    return _dt_of(t.dtype)


def _dev(*ts):
    for t in ts:
        if t is not None and (t.device.type != "cuda" or not t.is_contiguous()):
            raise ValueError("inputs must be contiguous CUDA tensors")


W_Q4G32, W_Q4G128, W_Q8G64, W_F8 = 3, 4, 5, 6
_FMT = {"f32": W_F32, "bf16": W_BF16, "q4": W_Q4G64, "q4g32": W_Q4G32, "q4g128": W_Q4G128,
        "q8": W_Q8G64, "f8": W_F8}
ACT_SWIGLU, ACT_GEGLU_TANH = 0, 1
_ACT = {"swiglu": ACT_SWIGLU, "geglu": ACT_GEGLU_TANH}


def experts_struct(ex) -> Experts:
    """C view of an expert-weight set (any object with fmt, E, d, F, w_gu,
    s_gu, b_gu, w_dn, s_dn, b_dn, tensors on the device; act, "swiglu" or
    "geglu", defaults to "swiglu")."""
    _dev(ex.w_gu, ex.w_dn, ex.s_gu, ex.b_gu, ex.s_dn, ex.b_dn)
    fmt = _FMT[ex.fmt] if isinstance(ex.fmt, str) else int(ex.fmt)
    act = getattr(ex, "act", "swiglu")
    act = _ACT[act] if isinstance(act, str) else int(act)
    return Experts(fmt, ex.E, ex.d, ex.F, _ptr(ex.w_gu), _ptr(ex.s_gu), _ptr(ex.b_gu),
                   _ptr(ex.w_dn), _ptr(ex.s_dn), _ptr(ex.b_dn), act)


# ------------------------------------------------------------------ stages

def route(x, w_router, router_bias, k, stream=None):
    """-> (logits fp32 [T,E], topk_idx int32 [T,k], topk_w fp32 [T,k])"""
    if stream is not None:
        return _under(stream, route, x, w_router, router_bias, k)
    _dev(x, w_router, router_bias)
    T, d = x.shape
    E = w_router.shape[0]
    dev = x.device
    logits = torch.empty(T, E, dtype=torch.float32, device=dev)
    idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    _check(lib.moe_route(_ptr(x), _dt(x), _ptr(w_router), _ptr(router_bias), T, d, E, k,
                         _ptr(logits), _ptr(idx), _ptr(w), _stream()), "moe_route")
    return logits, idx, w


def topk(logits, k, stream=None):
    """-> (topk_idx int32 [T,k], topk_w fp32 [T,k]) from fp32 logits [T,E]"""
    if stream is not None:
        return _under(stream, topk, logits, k)
    _dev(logits)
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _check(lib.moe_topk(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream()), "moe_topk")
    return idx, w


@dataclass
class SortTables:
    order: torch.Tensor
    inv_order: torch.Tensor
    row_map: torch.Tensor
    counts: torch.Tensor
    row_off: torch.Tensor
    tile_off: torch.Tensor
    BM: int


def sort_rows(topk_idx, E, BM, stream=None) -> SortTables:
    if stream is not None:
        return _under(stream, sort_rows, topk_idx, E, BM)
    _dev(topk_idx)
    T, k = topk_idx.shape
    R = T * k
    dev = topk_idx.device
    u32 = lambda n: torch.empty(n, dtype=torch.uint32, device=dev)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
    order, inv, rmap = u32(R), u32(R), u32(R)
    counts, roff, toff = i32(E), i32(E + 1), i32(E + 1)
    nws = lib.moe_sort_rows_workspace(T, k, E)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev)
    _check(lib.moe_sort_rows(_ptr(topk_idx), T, k, E, BM, _ptr(order), _ptr(inv), _ptr(rmap),
                             _ptr(counts), _ptr(roff), _ptr(toff), _ptr(ws), nws,
                             _stream()), "moe_sort_rows")
    return SortTables(order, inv, rmap, counts, roff, toff, BM)


def grouped_swiglu(x, tables: SortTables, k, experts, regime=REGIME_AUTO, ws=None, stream=None):
    """-> h [T*k, F]: fp16 for bf16 or fp16 x, fp32 for fp32 x"""
    if stream is not None:
        return _under(stream, grouped_swiglu, x, tables, k, experts, regime, ws)
    _dev(x)
    T = x.shape[0]
    ex = experts_struct(experts)
    hdt = torch.float32 if x.dtype == torch.float32 else torch.float16
    h = torch.empty(T * k, experts.F, dtype=hdt, device=x.device)
    nws = lib.moe_grouped_swiglu_workspace(T, k, experts.d, _dt(x))
    if ws is None:
        ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=x.device)
    _check(lib.moe_grouped_swiglu(_ptr(x), _dt(x), _ptr(tables.row_map), _ptr(tables.row_off),
                                  _ptr(tables.tile_off), tables.BM, T, k, ctypes.byref(ex),
                                  _ptr(h), _ptr(ws), ws.numel(), regime, _stream()),
           "moe_grouped_swiglu")
    return h


def grouped_down(h, tables: SortTables, T, k, experts, regime=REGIME_AUTO, stream=None,
                 dtype=None):
    """-> ys [T*k, d]: fp16 for 16-bit activations (fp16 h), fp32 for fp32.
    `dtype` is the layer's activation type (torch.bfloat16, torch.float16 or
    torch.float32); it may be left out for fp32 h, which only fp32
    activations produce."""
    if stream is not None:
        return _under(stream, grouped_down, h, tables, T, k, experts, regime, dtype=dtype)
    _dev(h)
    ex = experts_struct(experts)
    if dtype is None:
        if h.dtype != torch.float32:
            raise TypeError("grouped_down: pass dtype, the activation type (bf16 or fp16) "
                            "the fp16 h was computed from")
        dtype = torch.float32
    adt = _dt_of(dtype)
    want = torch.float32 if adt == F32 else torch.float16
    if h.dtype != want:
        raise TypeError(f"h must be {want} for {dtype} activations")
    ys = torch.empty(T * k, experts.d, dtype=h.dtype, device=h.device)
    _check(lib.moe_grouped_down(_ptr(h), adt, _ptr(tables.row_off), _ptr(tables.tile_off),
                                tables.BM, T, k, ctypes.byref(ex), _ptr(ys), regime,
                                _stream()), "moe_grouped_down")
    return ys


def combine(ys, inv_order, topk_w, T, k, dtype=torch.bfloat16, stream=None):
    """-> y [T, d] in `dtype` from ys [T*k, d] (fp16 for 16-bit `dtype`, fp32 for fp32)"""
    if stream is not None:
        return _under(stream, combine, ys, inv_order, topk_w, T, k, dtype)
    _dev(ys, inv_order, topk_w)
    want = torch.float32 if dtype == torch.float32 else torch.float16
    if ys.dtype != want:
        raise TypeError(f"ys must be {want} for {dtype} outputs")
    d = ys.shape[1]
    y = torch.empty(T, d, dtype=dtype, device=ys.device)
    _check(lib.moe_combine(_ptr(ys), _ptr(inv_order), _ptr(topk_w), T, k, d,
                           _dt_of(dtype), _ptr(y), _stream()), "moe_combine")
    return y


# ------------------------------------------------------------------ 8-bit floating point

F8 = torch.float8_e4m3fn
FP8_BLOCK = 128
_F32, _U8, _I32 = torch.float32, torch.uint8, torch.int32
_ROWS = (torch.uint32, torch.int32)          # row numbers: below 2^31 either way
_empty = torch.empty
# the current device and its current stream's handle, by torch's own shortcuts
# where it has them (the public calls take about a microsecond more)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _on(*ts):
    """Contiguous tensors of the current device, where the launches go; the
    raw handle of its current stream."""
    dev = -1
    for t in ts:
        if t is not None:
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("inputs must be contiguous CUDA tensors")
            if t.get_device() != dev:
                if dev >= 0 or t.get_device() != _device():
                    raise ValueError(f"a tensor is on {t.device}, the call is for the current "
                                     f"device, cuda:{_device()}")
                dev = t.get_device()
    return _raw_stream(dev)


def _is(t, dtype, shape, what):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


def _codes(t, dims, what):
    dt = t.dtype
    if dt != F8 and dt != _U8:
        raise TypeError(f"{what} must be e4m3 codes (float8_e4m3fn or uint8), got {dt}")
    if t.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions, got {list(t.shape)}")


def _sizes(*ns):
    """The library's size limit, which a larger Python int would slip past as a C int."""
    if max(ns) > 1 << 30:
        raise ValueError(f"sizes {list(ns)} are limited to 2^30 each")


def _at(t):
    return None if t is None else t.data_ptr()


def quantize_fp8(x, block=1, stream=None):
    """e4m3 codes (x's shape) and fp32 scales of x [rows, K]: a scale per row and
    128 columns (block=1: [rows, ceil(K/128)], for activations) or per 128 x 128
    elements (block=128: [ceil(rows/128), ceil(K/128)], for weights). A stack of
    weights x [E, rows, K] (rows a multiple of 128 for block=128) gives a stack
    of scales."""
    if stream is not None:
        return _under(stream, quantize_fp8, x, block)
    raw = _on(x)
    shape = x.shape
    if len(shape) < 2:
        raise ValueError(f"x must be [rows, K] or a stack of such, got {list(shape)}")
    rows, K = shape[-2:]
    if block != 1 and block != FP8_BLOCK:
        raise ValueError(f"block must be 1 or {FP8_BLOCK}, got {block}")
    n, groups = rows, (rows if block == 1 else -(-rows // FP8_BLOCK))
    if len(shape) > 2:
        n = x.numel() // K if K else 0
    _sizes(n, K)
    q = torch.empty_like(x, dtype=F8)
    if len(shape) == 2:
        s = _empty(groups, -(-K // FP8_BLOCK), dtype=_F32, device=x.device)
    else:
        if block != 1 and rows % FP8_BLOCK:
            raise ValueError("a stack of weights needs rows in multiples of 128 (a block of "
                             "scales may not straddle two of them)")
        s = _empty(*shape[:-2], groups, -(-K // FP8_BLOCK), dtype=_F32, device=x.device)
    st = lib.moe_quantize_fp8(x.data_ptr(), _dt(x), n, K, block, q.data_ptr(), s.data_ptr(), raw)
    if st:
        _check(st, "moe_quantize_fp8")
    return q, s


def fp8_matmul(a, sa, b, sb, dtype=torch.bfloat16, out=None, stream=None):
    """y [M, N] = a . b^T in `dtype` from e4m3 codes a [M, K], b [N, K] and fp32
    scales sa [M, ceil(K/128)], sb [ceil(N/128), ceil(K/128)]."""
    if stream is not None:
        return _under(stream, fp8_matmul, a, sa, b, sb, dtype, out)
    raw = _on(a, sa, b, sb, out)
    _codes(a, 2, "a")
    _codes(b, 2, "b")
    M, K = a.shape
    N, Kb = b.shape
    if Kb != K:
        raise ValueError(f"a is [{M}, {K}] and b [{N}, {Kb}]: K differs")
    _sizes(M, N, K)
    KB = -(-K // FP8_BLOCK)
    _is(sa, _F32, (M, KB), "sa")
    _is(sb, _F32, (-(-N // FP8_BLOCK), KB), "sb")
    dt = _dt_of(dtype)
    if out is None:
        out = _empty(M, N, dtype=dtype, device=a.device)
    else:
        _is(out, dtype, (M, N), "out")
    st = lib.moe_fp8_matmul(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), M, N, K, dt,
                            out.data_ptr(), raw)
    if st:
        _check(st, "moe_fp8_matmul")
    return out


def _f8_experts(ex) -> Experts:
    """C view of f8 experts, whose shapes and types the kernels rely on; experts
    of another format as experts_struct has them (the fp8 stage calls of the
    library refuse them)."""
    fmt = ex.fmt
    if fmt != "f8" and fmt != W_F8:
        return experts_struct(ex)
    w_gu, s_gu, w_dn, s_dn, act = ex.w_gu, ex.s_gu, ex.w_dn, ex.s_dn, getattr(ex, "act", "swiglu")
    E, d, F, B = ex.E, ex.d, ex.F, FP8_BLOCK
    if w_gu.shape != (E, 2 * F, d) or w_dn.shape != (E, d, F):
        raise ValueError("f8 experts: w_gu must be [E, 2F, d] and w_dn [E, d, F]")
    _codes(w_gu, 3, "w_gu")
    _codes(w_dn, 3, "w_dn")
    _is(s_gu, _F32, (E, 2 * F // B, d // B), "s_gu")
    _is(s_dn, _F32, (E, d // B, F // B), "s_dn")
    _on(w_gu, s_gu, w_dn, s_dn)
    return Experts(W_F8, E, d, F, w_gu.data_ptr(), s_gu.data_ptr(), None, w_dn.data_ptr(),
                   s_dn.data_ptr(), None, _ACT[act] if isinstance(act, str) else int(act))


def _tables_of(t: SortTables, R, E):
    """sort_rows' tables of R rows and E experts: the kernels index by them."""
    rows, roff, toff = t.row_map, t.row_off, t.tile_off
    if rows.numel() != R or roff.numel() != E + 1 or toff.numel() != E + 1:
        raise ValueError(f"the tables are of {rows.numel()} rows and {roff.numel() - 1} experts, "
                         f"not {R} rows and {E}")
    if roff.dtype != _I32 or toff.dtype != _I32:
        raise ValueError(f"row_off and tile_off must be int32, got {roff.dtype} and {toff.dtype}")


def grouped_swiglu_fp8(xq, xs, tables: SortTables, k, experts, regime=REGIME_AUTO, stream=None):
    """-> (hq e4m3 [T*k, F], hs fp32 [T*k, F/128]): gate|up and GLU of f8 experts
    from quantised token rows xq [T, d], xs [T, d/128] (quantize_fp8)."""
    if stream is not None:
        return _under(stream, grouped_swiglu_fp8, xq, xs, tables, k, experts, regime)
    rmap, roff, toff = tables.row_map, tables.row_off, tables.tile_off
    raw = _on(xq, xs, rmap, roff, toff)
    _codes(xq, 2, "xq")
    T, d = xq.shape
    if d != experts.d:
        raise ValueError(f"xq is {list(xq.shape)}, the experts' d is {experts.d}")
    _is(xs, _F32, (T, -(-d // FP8_BLOCK)), "xs")
    R, F, E = T * k, experts.F, experts.E
    _tables_of(tables, R, E)
    if rmap.dtype not in _ROWS:
        raise ValueError(f"row_map must be uint32 or int32, got {rmap.dtype}")
    ex = _f8_experts(experts)
    dev = xq.device
    hq = _empty(R, F, dtype=F8, device=dev)
    hs = _empty(R, -(-F // FP8_BLOCK), dtype=_F32, device=dev)
    st = lib.moe_grouped_swiglu_fp8(xq.data_ptr(), xs.data_ptr(), rmap.data_ptr(), roff.data_ptr(),
                                    toff.data_ptr(), tables.BM, T, k, ctypes.byref(ex),
                                    hq.data_ptr(), hs.data_ptr(), regime, raw)
    if st:
        _check(st, "moe_grouped_swiglu_fp8")
    return hq, hs


def grouped_down_fp8(hq, hs, tables: SortTables, T, k, experts, regime=REGIME_AUTO, stream=None):
    """-> ys fp16 [T*k, d] from quantised rows hq [T*k, F], hs [T*k, F/128]
    (grouped_swiglu_fp8)."""
    if stream is not None:
        return _under(stream, grouped_down_fp8, hq, hs, tables, T, k, experts, regime)
    roff, toff = tables.row_off, tables.tile_off
    raw = _on(hq, hs, roff, toff)
    _codes(hq, 2, "hq")
    R, F, E = T * k, experts.F, experts.E
    if hq.shape != (R, F):
        raise ValueError(f"hq is {list(hq.shape)}, not [{T} x {k}, {F}]")
    _is(hs, _F32, (R, -(-F // FP8_BLOCK)), "hs")
    _tables_of(tables, R, E)
    ex = _f8_experts(experts)
    ys = _empty(R, experts.d, dtype=torch.float16, device=hq.device)
    st = lib.moe_grouped_down_fp8(hq.data_ptr(), hs.data_ptr(), roff.data_ptr(), toff.data_ptr(),
                                  tables.BM, T, k, ctypes.byref(ex), ys.data_ptr(), regime, raw)
    if st:
        _check(st, "moe_grouped_down_fp8")
    return ys


# ------------------------------------------------------------------ router training

@dataclass
class BalanceStats:
    loss: torch.Tensor      # fp32 []
    counts: torch.Tensor    # int32 [sequences, E]
    probs: torch.Tensor     # fp32 [sequences, E]
    tokens: torch.Tensor    # int32 [sequences]


def _balance_sizes(logits, mask, seq_off):
    if logits.dtype != _F32 or logits.dim() != 2:
        raise ValueError(f"logits must be fp32 [T, E], got {logits.dtype} {list(logits.shape)}")
    T, E = logits.shape
    _sizes(T, E)
    if mask is not None and (mask.dtype not in (torch.bool, _U8) or mask.shape != (T,)):
        raise ValueError(f"mask must be bool or uint8 [{T}], got {mask.dtype} {list(mask.shape)}")
    if seq_off is None:
        return T, E, 1
    if seq_off.dtype != _I32 or seq_off.dim() != 1 or seq_off.numel() < 2:
        raise ValueError("seq_off must be int32 [sequences + 1]")
    _sizes(seq_off.numel())
    return T, E, seq_off.numel() - 1


def balance_loss(logits, topk_idx, coef, mask=None, seq_off=None, ws=None,
                 stream=None) -> BalanceStats:
    """The router's balance loss with its per-expert counts and mean
    probabilities, per sequence (seq_off int32 [sequences + 1]; all tokens are
    one where it is left out), from fp32 logits [T, E] and topk_idx int32 [T, k].
    mask [T]: tokens that are False take no part. ws: a uint8 tensor of
    moe_balance_loss_workspace bytes to reuse.

    Logits that require a gradient give a loss that has one, by
    balance_loss_backward. The counts are constants of it; a gradient that arrives
    at probs, and a second derivative, are refused."""
    if stream is not None:
        return _under(stream, balance_loss, logits, topk_idx, coef, mask, seq_off, ws)
    if logits.requires_grad and torch.is_grad_enabled():
        return BalanceStats(*_BalanceLoss.apply(logits, topk_idx, coef, mask, seq_off, ws))
    raw = _on(logits, topk_idx, mask, seq_off, ws)
    T, E, B = _balance_sizes(logits, mask, seq_off)
    if topk_idx.dtype != _I32 or topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError(f"topk_idx must be int32 [{T}, k], got {topk_idx.dtype} "
                         f"{list(topk_idx.shape)}")
    k = topk_idx.shape[1]
    _sizes(k)
    dev = logits.device
    loss = torch.empty((), dtype=_F32, device=dev)
    probs = _empty(B, E, dtype=_F32, device=dev)
    counts = _empty(B, E, dtype=_I32, device=dev)
    tokens = _empty(B, dtype=_I32, device=dev)
    if ws is None:
        need = lib.moe_balance_loss_workspace(T, E, B)
        if need:
            ws = _empty(need, dtype=_U8, device=dev)
    st = lib.moe_balance_loss(logits.data_ptr(), topk_idx.data_ptr(), _at(mask), _at(seq_off), T, E,
                              k, B, coef, loss.data_ptr(), counts.data_ptr(), probs.data_ptr(),
                              tokens.data_ptr(), _at(ws), 0 if ws is None else ws.nbytes, raw)
    if st:
        _check(st, "moe_balance_loss")
    return BalanceStats(loss, counts, probs, tokens)


def balance_loss_backward(logits, stats: BalanceStats, k, coef, mask=None, seq_off=None,
                          dloss=None, stream=None):
    """-> dlogits fp32 [T, E], the gradient of balance_loss(logits, ..., coef, mask,
    seq_off) times dloss (an fp32 tensor of one value; 1 where it is left out)."""
    if stream is not None:
        return _under(stream, balance_loss_backward, logits, stats, k, coef, mask, seq_off, dloss)
    counts, tokens = stats.counts, stats.tokens
    raw = _on(logits, counts, tokens, mask, seq_off, dloss)
    T, E, B = _balance_sizes(logits, mask, seq_off)
    _sizes(k)
    _is(counts, _I32, (B, E), "stats.counts")
    _is(tokens, _I32, (B,), "stats.tokens")
    if dloss is not None and (dloss.dtype != _F32 or dloss.numel() != 1):
        raise ValueError("dloss must be one fp32 value")
    d = torch.empty_like(logits)
    st = lib.moe_balance_loss_backward(logits.data_ptr(), _at(mask), _at(seq_off), T, E, k, B, coef,
                                       counts.data_ptr(), tokens.data_ptr(), _at(dloss),
                                       d.data_ptr(), raw)
    if st:
        _check(st, "moe_balance_loss_backward")
    return d


class _BalanceLoss(torch.autograd.Function):
    """balance_loss as a node of torch's graph (grad mode is off inside)."""

    @staticmethod
    def forward(ctx, logits, topk_idx, coef, mask, seq_off, ws):
        s = balance_loss(logits, topk_idx, coef, mask, seq_off, ws)
        ctx.k, ctx.coef = topk_idx.shape[1], coef
        ctx.save_for_backward(logits, s.counts, s.tokens, mask, seq_off)
        ctx.mark_non_differentiable(s.counts, s.tokens)
        ctx.set_materialize_grads(False)
        return s.loss, s.counts, s.probs, s.tokens

    @staticmethod
    def backward(ctx, dloss, dcounts, dprobs, dtokens):
        if torch.is_grad_enabled():
            raise RuntimeError("balance_loss is once differentiable (create_graph is not for it)")
        if dprobs is not None:
            raise RuntimeError("balance_loss: probs is a statistic without a gradient of its own "
                               "(detach it)")
        if dloss is None:
            return (None,) * 6
        logits, counts, tokens, mask, seq_off = ctx.saved_tensors
        d = balance_loss_backward(logits, BalanceStats(None, counts, None, tokens), ctx.k, ctx.coef,
                                  mask, seq_off, dloss)
        return (d,) + (None,) * 5


# ------------------------------------------------------------------ forward

def _fmt_code(fmt) -> int:
    return _FMT[fmt] if isinstance(fmt, str) else int(fmt)


def forward_layout(T, d, E, k, F, dtype, wfmt, regime=REGIME_AUTO) -> WsLayout:
    """moe_forward's workspace layout for experts of weight format `wfmt`
    (a name such as "q4", or a moe_wfmt code)."""
    L = WsLayout()
    dt = _dt_of(dtype)
    _check(lib.moe_forward_layout(T, d, E, k, F, dt, _fmt_code(wfmt), regime, ctypes.byref(L)),
           "moe_forward_layout")
    return L


def sort_block_m() -> int:
    """BM of the tensor-core regime (moe_sort_block_m)."""
    return lib.moe_sort_block_m()


def forward_workspace(x, experts, k, regime=REGIME_AUTO):
    """A workspace tensor large enough for moe_forward on these shapes."""
    L = forward_layout(x.shape[0], experts.d, experts.E, k, experts.F, x.dtype, experts.fmt,
                       regime)
    return torch.empty(max(L.total, 256), dtype=torch.uint8, device=x.device)


def forward(x, w_router, router_bias, experts, k, regime=REGIME_AUTO, ws=None, out=None,
            stream=None):
    """The whole layer: y [T, d] in x's dtype."""
    if stream is not None:
        return _under(stream, forward, x, w_router, router_bias, experts, k, regime, ws, out)
    _dev(x, w_router, router_bias)
    T = x.shape[0]
    if x.shape != (T, experts.d) or w_router.shape != (experts.E, experts.d):
        raise ValueError(f"x is {list(x.shape)} and w_router {list(w_router.shape)}, not "
                         f"[T, {experts.d}] and [{experts.E}, {experts.d}]")
    ex = _f8_experts(experts)
    if ws is None:
        ws = forward_workspace(x, experts, k, regime)
    y = out if out is not None else torch.empty(T, experts.d, dtype=x.dtype, device=x.device)
    _check(lib.moe_forward(_ptr(x), _dt(x), _ptr(w_router), _ptr(router_bias), ctypes.byref(ex),
                           T, k, _ptr(y), _ptr(ws), ws.numel(), regime, _stream()),
           "moe_forward")
    return y


def pack_gate_up(fmt, w_g, w_u, s_g=None, b_g=None, s_u=None, b_u=None, stream=None):
    """Fused [gate|up] tensors (w_gu, s_gu, b_gu) from separate gate and up
    projections [E][F][...] on the device; s_gu, b_gu are None unless q4 or q8
    (f8 has s_gu alone)."""
    if stream is not None:
        return _under(stream, pack_gate_up, fmt, w_g, w_u, s_g, b_g, s_u, b_u)
    _dev(w_g, w_u, s_g, b_g, s_u, b_u)
    E, F = w_g.shape[0], w_g.shape[1]
    fmt_c = _FMT[fmt] if isinstance(fmt, str) else int(fmt)
    per_word = {W_Q4G64: 8, W_Q4G32: 8, W_Q4G128: 8, W_Q8G64: 4}.get(fmt_c, 1)
    d = w_g.shape[2] * per_word
    if w_u.shape != w_g.shape or w_u.element_size() != w_g.element_size():
        raise ValueError(f"w_u must be {w_g.dtype} {list(w_g.shape)} as w_g is, got {w_u.dtype} "
                         f"{list(w_u.shape)}")
    group = {W_Q4G64: 64, W_Q4G32: 32, W_Q4G128: 128, W_Q8G64: 64}.get(fmt_c, 0)
    w_gu = torch.empty((E, 2 * F) + tuple(w_g.shape[2:]), dtype=w_g.dtype, device=w_g.device)
    s_gu = b_gu = None
    if group:
        s_gu = torch.empty((E, 2 * F, d // group), dtype=s_g.dtype, device=s_g.device)
        b_gu = torch.empty_like(s_gu)
    elif fmt_c == W_F8:
        _codes(w_g, 3, "w_g")
        _codes(w_u, 3, "w_u")
        for s, what in ((s_g, "s_g"), (s_u, "s_u")):
            if s is None:
                raise ValueError(f"f8 weights need {what}")
            _is(s, _F32, (E, F // FP8_BLOCK, d // FP8_BLOCK), what)
        s_gu = torch.empty((E, 2 * (F // FP8_BLOCK), d // FP8_BLOCK), dtype=_F32,
                           device=s_g.device)
    _check(lib.moe_pack_gate_up(fmt_c, E, d, F, _ptr(w_g), _ptr(s_g), _ptr(b_g), _ptr(w_u),
                                _ptr(s_u), _ptr(b_u), _ptr(w_gu), _ptr(s_gu), _ptr(b_gu),
                                _stream()), "moe_pack_gate_up")
    return w_gu, s_gu, b_gu


def device_status() -> int:
    """Status word of device-side errors since the last read (resets it)."""
    return lib.moe_device_status()


def set_wait_cycles(cycles: int):
    """Bound of every device-side wait, in SM cycles (0: the default, ~1 s)."""
    _check(lib.moe_set_wait_cycles(int(cycles)), "moe_set_wait_cycles")
