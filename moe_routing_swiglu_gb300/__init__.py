"""Python binding of the GB300 local MoE forward chain.

Thin ctypes layer over the C ABI in ``include/moe.h`` (``libmoe_gb300.so``,
built in-tree by ``_build.build``). The functions carry the C names and only
marshal arguments: PyTorch supplies device memory and the current stream;
every step of the chain runs in the library's CUDA kernels. There is no
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
from array import array
from collections import namedtuple
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmoe_gb300.so"

MOE_F32, MOE_F16, MOE_BF16 = 0, 1, 2
_DTYPE = {torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}

STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_DTYPE", 4: "MOE_ERR_TOP_K",
    5: "MOE_ERR_ALIGNMENT", 6: "MOE_ERR_WORKSPACE", 7: "MOE_ERR_UNSUPPORTED", 8: "MOE_ERR_CUDA",
    9: "MOE_ERR_DEVICE_CHECK",
}


class GroupRoutingOptions(ctypes.Structure):
    """moe_group_routing_options (GroupRoutingOptions of the grouped sigmoid
    routing): top_k, groups, selected_groups, group_top_two, renormalize, scale."""
    _fields_ = [("top_k", ctypes.c_int32), ("groups", ctypes.c_int32), ("selected_groups", ctypes.c_int32),
                ("group_top_two", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, top_k, groups, selected_groups, group_top_two=False, renormalize=True, scale=1.0):
        super().__init__(int(top_k), int(groups), int(selected_groups), int(bool(group_top_two)),
                         int(bool(renormalize)), float(scale))


class RouterWeightOptions(ctypes.Structure):
    """moe_router_weight_options (RouterWeightOptions of first-order training):
    scoring ("softmax" or "sigmoid"), renormalize, scale."""
    _fields_ = [("scoring", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, scoring="softmax", renormalize=True, scale=1.0):
        code = {"softmax": 0, "sigmoid": 1}[scoring] if isinstance(scoring, str) else int(scoring)
        super().__init__(code, int(bool(renormalize)), float(scale))


class GradTensor(ctypes.Structure):
    """moe_grad_tensor: one dense gradient (src, dst, numel, dtype code)."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


_INDEX = {torch.int32: 1, torch.int64: 2}
if hasattr(torch, "uint32"):
    _INDEX[torch.uint32] = 0


# Every entry point declared in include/moe.h: name -> (restype, argtypes).
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_OPT = ctypes.POINTER(GroupRoutingOptions)
_ROPT = ctypes.POINTER(RouterWeightOptions)
_FP = ctypes.c_void_p
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (ctypes.c_int, []),
    "moe_route": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I32, _I32, _P, _P, _P, _P]),
    "moe_dispatch_workspace_size": (_SZ, [_I64, _I64, _I32]),
    "moe_dispatch": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, ctypes.c_int, _I64, _P, _P, _P, _P, _P,
                                    _P, _SZ, _P]),
    "moe_dispatch_noalloc": (ctypes.c_int, [_P, _I64, _I64, _I32, _P, ctypes.c_int, _I64, _P, _P, _P, _P, _P,
                                            _P]),
    "moe_route_dispatch_workspace_size": (_SZ, [_I64, _I64]),
    "moe_route_dispatch": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I32, _I32, _P, _P, _P, _P, ctypes.c_int,
                                          _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_permute_rows": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, _I64, _I32, _P]),
    "moe_experts_create": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _I64, _I64,
                                          ctypes.POINTER(ctypes.c_void_p)]),
    "moe_experts_destroy": (None, [_P]),
    "moe_experts_forward_dispatched_workspace_size": (_SZ, [_P, _I64]),
    "moe_experts_forward_dispatched": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "moe_experts_forward_combine_workspace_size": (_SZ, [_P, _I64, _I32]),
    "moe_experts_forward_combine": (ctypes.c_int, [_P, _P, _P, _P, _P, ctypes.c_int, _I64, _I32, _P, _P, _SZ,
                                                   _P]),
    "moe_experts_gate_up": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "moe_experts_down": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "moe_experts_gate_up_gather": (ctypes.c_int, [_P, _P, _I64, _P, _I32, _P, _I64, _P, _P, _SZ, _P]),
    "moe_combine": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, ctypes.c_int, _I64, _I32, _I64, _P, _P]),
    "moe_forward_workspace_size": (_SZ, [_P, _I64, _I32]),
    "moe_forward": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_host_workspace_size": (ctypes.c_size_t, [_P, _I64, _I32, ctypes.c_int]),
    "moe_forward_host": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_sigmoid_grouped": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _OPT, _P, _P, _P, _P]),
    "moe_route_sigmoid_grouped_dispatch": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _OPT, _P, _P, _P, _P,
                                                          ctypes.c_int, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_sigmoid_grouped": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, _I64, _P, _OPT, _P, _P, _P, _P,
                                                   _SZ, _P]),
    "moe_router_weights": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, ctypes.c_int, _I32, _ROPT, _P, _P]),
    "moe_router_backward": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, ctypes.c_int, _I32, _ROPT, _P, _P,
                                           _P]),
    "moe_experts_forward_training_workspace_size": (_SZ, [_P]),
    "moe_experts_forward_training": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_combine_backward": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, ctypes.c_int, _P, _I64, _I32, _I64, _P,
                                            _P, _P]),
    "moe_experts_backward_workspace_size": (_SZ, [_P, _I64]),
    "moe_experts_backward": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_dispatch_backward": (ctypes.c_int, [_P, ctypes.c_int, _P, _I64, _I32, _I64, _P, _P]),
    "moe_mxfp4_scale_pitch": (_I64, [_I64]),
    "moe_mxfp4_quantize": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _I32, _P, _P, _P]),
    "moe_mxfp4_dequantize": (ctypes.c_int, [_P, _P, _I64, _I64, _P, ctypes.c_int, _P]),
    "moe_experts_mxfp4_storage_size": (_SZ, [_I64, _I64, _I64]),
    "moe_experts_mxfp4_create": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P,
                                                ctypes.POINTER(ctypes.c_void_p)]),
    "moe_experts_mxfp4_destroy": (None, [_P]),
    "moe_experts_mxfp4_gate_up": (ctypes.c_int, [_P, _P, _P, _P, _I64, ctypes.c_int, _P, _P, _P, _P]),
    "moe_experts_mxfp4_down": (ctypes.c_int, [_P, _P, _P, _P, _I64, ctypes.c_int, _P, _P]),
    "moe_experts_mxfp4_forward_dispatched_workspace_size": (_SZ, [_P, _I64]),
    "moe_experts_mxfp4_forward_dispatched": (ctypes.c_int, [_P, _P, _P, _P, _I64, ctypes.c_int, _P, _P, _SZ, _P]),
    "moe_forward_mxfp4_workspace_size": (_SZ, [_P, _I64, _I32, ctypes.c_int]),
    "moe_forward_mxfp4": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, ctypes.c_int, _I64, _I32, _I32, _P, _P, _P, _P,
                                         _SZ, _P]),
    "moe_grad_norm_workspace_size": (_SZ, [_I64]),
    "moe_grad_norm": (ctypes.c_int, [_P, _I64, _P, _P, _SZ, _P]),
    "moe_grad_clip": (ctypes.c_int, [_P, _I64, _P, ctypes.c_float, _P]),
    "moe_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _I32]),
    "moe_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_uint32, _P]),
}

_lib = None


class MoeError(RuntimeError):
    """A nonzero moe_status from the library (the MoeError of the pages)."""

    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, f"status {status}")
        super().__init__(f"{self.name}: {message}")


def load_library(path: str | Path | None = None):
    """Load libmoe_gb300.so (once) and declare every entry point. Raises if it
    is missing: there is no CPU or eager fallback."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path is not None else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build it with __graft_entry__.build() "
                           "(nvcc, sm_103a); there is no fallback path")
    lib = ctypes.CDLL(str(p))
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise MoeError(status, load_library().moe_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev_tensor(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPE:
        raise MoeError(3, f"unsupported dtype {t.dtype}")
    return _DTYPE[t.dtype]


def _workspace(nbytes: int, device, ws: torch.Tensor | None) -> torch.Tensor:
    if ws is not None:
        return ws
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool, *, indices=None, weights=None,
              weights_fp32=False, stream=None):
    """RoutingPlan: returns (indices [T,k] uint32 as int32 view, weights [T,k] in
    the logits dtype[, FP32 weights before the cast])."""
    lib = load_library()
    _dev_tensor(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    if indices is None:
        indices = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, top_k, dtype=logits.dtype, device=dev)
    w32 = torch.empty(T, top_k, dtype=torch.float32, device=dev) if weights_fp32 is True else (
        weights_fp32 if isinstance(weights_fp32, torch.Tensor) else None)
    _check(lib.moe_route(_ptr(logits), _dt(logits), T, E, top_k, int(bool(renormalize)), _ptr(indices),
                         _ptr(weights), _ptr(w32), _stream(stream)))
    return (indices, weights, w32) if w32 is not None else (indices, weights)


DispatchedTokens = namedtuple("DispatchedTokens", "counts offsets row_src inv x_dispatched")


def moe_dispatch(indices: torch.Tensor, num_experts: int, x: torch.Tensor | None = None,
                 workspace=None, stream=None) -> DispatchedTokens:
    """RoutingPlan::dispatch: per-expert counts/offsets, row_src, inv and (if x
    is given) x_dispatched [T*k, H]."""
    lib = load_library()
    _dev_tensor(indices, "indices")
    T, k = indices.shape
    dev = indices.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    row_src = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    xd = None
    H, xdt = 0, MOE_F32
    if x is not None:
        _dev_tensor(x, "x")
        H, xdt = x.shape[1], _dt(x)
        xd = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    need = lib.moe_dispatch_workspace_size(T, num_experts, k)
    ws = _workspace(need, dev, workspace)
    _check(lib.moe_dispatch(_ptr(indices), T, num_experts, k, _ptr(x), xdt, H, _ptr(counts),
                            _ptr(offsets), _ptr(row_src), _ptr(inv), _ptr(xd), _ptr(ws),
                            ws.numel(), _stream(stream)))
    return DispatchedTokens(counts, offsets, row_src, inv, xd)


def moe_route_dispatch(logits: torch.Tensor, top_k: int, renormalize: bool, x: torch.Tensor | None = None,
                       *, weights_fp32=False, workspace=None, stream=None):
    """moe_route then moe_dispatch as one launch (the same outputs, bit for
    bit): returns (indices, weights[, FP32 weights], DispatchedTokens)."""
    lib = load_library()
    _dev_tensor(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    indices = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    weights = torch.empty(T, top_k, dtype=logits.dtype, device=dev)
    w32 = torch.empty(T, top_k, dtype=torch.float32, device=dev) if weights_fp32 else None
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_src = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    xd = None
    H, xdt = 0, MOE_F32
    if x is not None:
        _dev_tensor(x, "x")
        H, xdt = x.shape[1], _dt(x)
        xd = torch.empty(T * top_k, H, dtype=x.dtype, device=dev)
    need = lib.moe_route_dispatch_workspace_size(T, E)
    ws = _workspace(need, dev, workspace)
    _check(lib.moe_route_dispatch(_ptr(logits), _dt(logits), T, E, top_k, int(bool(renormalize)), _ptr(indices),
                                  _ptr(weights), _ptr(w32), _ptr(x), xdt, H, _ptr(counts), _ptr(offsets),
                                  _ptr(row_src), _ptr(inv), _ptr(xd), _ptr(ws), ws.numel(), _stream(stream)))
    disp = DispatchedTokens(counts, offsets, row_src, inv, xd)
    return (indices, weights, w32, disp) if w32 is not None else (indices, weights, disp)


def moe_permute_rows(src: torch.Tensor, index: torch.Tensor, *, scatter: bool = False, out=None,
                     out_rows: int | None = None, stream=None) -> torch.Tensor:
    """Row moves by an int64 index on the device: gather out[r] = src[index[r]]
    (out has index.numel() rows), or with scatter out[index[r]] = src[r] (out
    has out_rows rows, default src's)."""
    lib = load_library()
    _dev_tensor(src, "src")
    _dev_tensor(index, "index")
    if index.dtype != torch.int64:
        raise MoeError(3, "index must be int64")
    rows = index.numel()
    row_shape = tuple(src.shape[1:])
    if out is None:
        n_out = (out_rows if out_rows is not None else src.shape[0]) if scatter else rows
        out = torch.empty((n_out,) + row_shape, dtype=src.dtype, device=src.device)
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] else 1
    _check(lib.moe_permute_rows(_ptr(src), src.shape[0], _ptr(out), out.shape[0], _ptr(index), rows, row_bytes,
                                int(bool(scatter)), _stream(stream)))
    return out


def moe_dispatch_noalloc(indices: torch.Tensor, num_experts: int, x: torch.Tensor | None = None,
                         stream=None) -> DispatchedTokens:
    """moe_dispatch with the library's fixed 1 MiB scratch instead of a
    workspace, for callers that cannot allocate device memory when they
    dispatch (the output tensors here are still allocated by torch)."""
    lib = load_library()
    _dev_tensor(indices, "indices")
    T, k = indices.shape
    dev = indices.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    row_src = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    xd = None
    H, xdt = 0, MOE_F32
    if x is not None:
        _dev_tensor(x, "x")
        H, xdt = x.shape[1], _dt(x)
        xd = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    _check(lib.moe_dispatch_noalloc(_ptr(indices), T, num_experts, k, _ptr(x), xdt, H, _ptr(counts),
                                    _ptr(offsets), _ptr(row_src), _ptr(inv), _ptr(xd), _stream(stream)))
    return DispatchedTokens(counts, offsets, row_src, inv, xd)


class Experts:
    """SwiGluExperts: a handle over gate/up [E,I,H] and down [E,H,I] (kept alive here)."""

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor):
        lib = load_library()
        for name, t in (("gate", gate), ("up", up), ("down", down)):
            _dev_tensor(t, name)
        E, I, H = gate.shape
        self.gate, self.up, self.down = gate, up, down
        self.E, self.H, self.I = E, H, I
        self.dtype = gate.dtype
        handle = ctypes.c_void_p()
        _check(lib.moe_experts_create(_ptr(gate), _ptr(up), _ptr(down), _dt(gate), E, H, I,
                                      ctypes.byref(handle)))
        self.handle = handle

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_experts_destroy(self.handle)
            self.handle = None


def moe_experts_create(gate, up, down) -> Experts:
    return Experts(gate, up, down)


def moe_experts_forward_dispatched(experts: Experts, x_dispatched: torch.Tensor,
                                   offsets: torch.Tensor, out=None, workspace=None, stream=None):
    """SwiGluExperts::forward_dispatched: y_dispatched [rows, H] in the experts' dtype."""
    lib = load_library()
    _dev_tensor(x_dispatched, "x_dispatched")
    rows = x_dispatched.shape[0]
    y = out if out is not None else torch.empty(rows, experts.H, dtype=experts.dtype,
                                                device=x_dispatched.device)
    need = lib.moe_experts_forward_dispatched_workspace_size(experts.handle, rows)
    ws = _workspace(need, x_dispatched.device, workspace)
    _check(lib.moe_experts_forward_dispatched(experts.handle, _ptr(x_dispatched), _ptr(offsets), rows,
                                              _ptr(y), _ptr(ws), ws.numel(), _stream(stream)))
    return y


def moe_experts_forward_combine(experts: Experts, x_dispatched: torch.Tensor, offsets: torch.Tensor,
                                inv: torch.Tensor, weights: torch.Tensor, out=None, workspace=None, stream=None):
    """forward_dispatched and combine in one launch: out [T, H] = sum over
    slots j (in order) of w[t, j] * y[inv[t * top_k + j]] (inv from
    moe_dispatch, weights [T, top_k] from moe_route)."""
    lib = load_library()
    _dev_tensor(x_dispatched, "x_dispatched")
    T, top_k = weights.shape
    y = out if out is not None else torch.empty(T, experts.H, dtype=experts.dtype, device=x_dispatched.device)
    need = lib.moe_experts_forward_combine_workspace_size(experts.handle, T, top_k)
    ws = _workspace(need, x_dispatched.device, workspace)
    _check(lib.moe_experts_forward_combine(experts.handle, _ptr(x_dispatched), _ptr(offsets), _ptr(inv),
                                           _ptr(weights), _dt(weights), T, top_k, _ptr(y), _ptr(ws), ws.numel(),
                                           _stream(stream)))
    return y


STAGE_WORKSPACE_BYTES = 256


def moe_experts_gate_up(experts: Experts, x_dispatched: torch.Tensor, offsets: torch.Tensor, out=None,
                        workspace=None, stream=None):
    """First GEMM stage: h [rows, I] = SiLU(x W_gate^T) * (x W_up^T) per expert."""
    lib = load_library()
    _dev_tensor(x_dispatched, "x_dispatched")
    rows = x_dispatched.shape[0]
    h = out if out is not None else torch.empty(rows, experts.I, dtype=experts.dtype,
                                                device=x_dispatched.device)
    ws = _workspace(STAGE_WORKSPACE_BYTES, x_dispatched.device, workspace)
    _check(lib.moe_experts_gate_up(experts.handle, _ptr(x_dispatched), _ptr(offsets), rows, _ptr(h),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return h


def moe_experts_gate_up_gather(experts: Experts, x: torch.Tensor, row_src: torch.Tensor, top_k: int,
                               offsets: torch.Tensor, rows: int | None = None, out=None, workspace=None,
                               stream=None):
    """Gate/up stage reading dispatched row r from x[row_src[r] // top_k]:
    h [rows, I] without an x_dispatched copy (rows defaults to row_src's length)."""
    lib = load_library()
    _dev_tensor(x, "x")
    _dev_tensor(row_src, "row_src")
    T = x.shape[0]
    rows = row_src.shape[0] if rows is None else rows
    h = out if out is not None else torch.empty(rows, experts.I, dtype=experts.dtype, device=x.device)
    ws = _workspace(STAGE_WORKSPACE_BYTES, x.device, workspace)
    _check(lib.moe_experts_gate_up_gather(experts.handle, _ptr(x), T, _ptr(row_src), top_k, _ptr(offsets), rows,
                                          _ptr(h), _ptr(ws), ws.numel(), _stream(stream)))
    return h


def moe_experts_down(experts: Experts, h: torch.Tensor, offsets: torch.Tensor, out=None, workspace=None,
                     stream=None):
    """Second GEMM stage: y [rows, H] = h W_down^T per expert."""
    lib = load_library()
    _dev_tensor(h, "h")
    rows = h.shape[0]
    y = out if out is not None else torch.empty(rows, experts.H, dtype=experts.dtype, device=h.device)
    ws = _workspace(STAGE_WORKSPACE_BYTES, h.device, workspace)
    _check(lib.moe_experts_down(experts.handle, _ptr(h), _ptr(offsets), rows, _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)))
    return y


def moe_combine(y_dispatched: torch.Tensor, inv: torch.Tensor, weights: torch.Tensor, out=None,
                stream=None):
    """DispatchedTokens::combine: out [T, H] in y's dtype."""
    lib = load_library()
    _dev_tensor(y_dispatched, "y_dispatched")
    T, k = weights.shape
    H = y_dispatched.shape[1]
    o = out if out is not None else torch.empty(T, H, dtype=y_dispatched.dtype, device=y_dispatched.device)
    _check(lib.moe_combine(_ptr(y_dispatched), _dt(y_dispatched), _ptr(inv), _ptr(weights), _dt(weights),
                           T, k, H, _ptr(o), _stream(stream)))
    return o


def moe_forward_workspace_size(experts: Experts, T: int, top_k: int) -> int:
    return int(load_library().moe_forward_workspace_size(experts.handle, T, top_k))


def moe_forward(experts: Experts, x: torch.Tensor, logits: torch.Tensor, top_k: int,
                renormalize: bool, *, out=None, indices=None, weights=None, workspace=None,
                stream=None):
    """SwiGluExperts::forward: the whole chain, out [T, H]."""
    lib = load_library()
    _dev_tensor(x, "x")
    _dev_tensor(logits, "logits")
    T = x.shape[0]
    o = out if out is not None else torch.empty(T, experts.H, dtype=experts.dtype, device=x.device)
    ws = _workspace(lib.moe_forward_workspace_size(experts.handle, T, top_k), x.device, workspace)
    _check(lib.moe_forward(experts.handle, _ptr(x), _ptr(logits), _dt(logits), T, top_k,
                           int(bool(renormalize)), _ptr(o), _ptr(indices), _ptr(weights), _ptr(ws),
                           ws.numel(), _stream(stream)))
    return o


def moe_forward_host(experts: Experts, x: torch.Tensor, logits: torch.Tensor, top_k: int, renormalize: bool, *,
                     out=None, indices=None, weights=None, workspace=None, stream=None):
    """moe_forward on host (CPU) tensors: x [T, H] and logits [T, E] are
    copied to the device, the chain runs and out [T, H] is copied back, all
    enqueued on the stream. Pin the host tensors (`pin_memory()`) for
    asynchronous copies; the result is in `out` once the stream has passed
    the call's work."""
    lib = load_library()
    for t, name in ((x, "x"), (logits, "logits")):
        if t.is_cuda or not t.is_contiguous():
            raise MoeError(2, f"{name} must be a contiguous host tensor")
    T = x.shape[0]
    o = out if out is not None else torch.empty(T, experts.H, dtype=experts.dtype).pin_memory()
    if o.is_cuda or not o.is_contiguous():
        raise MoeError(2, "out must be a contiguous host tensor")
    dev = torch.device("cuda", torch.cuda.current_device())
    ws = _workspace(lib.moe_forward_host_workspace_size(experts.handle, T, top_k, _dt(logits)), dev, workspace)
    _check(lib.moe_forward_host(experts.handle, _ptr(x), _ptr(logits), _dt(logits), T, top_k, int(bool(renormalize)),
                                _ptr(o), _ptr(indices), _ptr(weights), _ptr(ws), ws.numel(), _stream(stream)))
    return o


def _options(options) -> GroupRoutingOptions:
    if isinstance(options, GroupRoutingOptions):
        return options
    return GroupRoutingOptions(options.top_k, options.groups, options.selected_groups, options.group_top_two,
                               options.renormalize, options.scale)


def moe_route_sigmoid_grouped(logits: torch.Tensor, bias: torch.Tensor | None, options, *, indices=None,
                              weights=None, weights_fp32=False, stream=None):
    """route_sigmoid_grouped: (indices [T,k], weights [T,k] in the logits
    dtype[, FP32 weights before the cast]). `options` is a
    GroupRoutingOptions (or any object with the same fields); `bias` is an
    FP32 [E] device tensor or None."""
    lib = load_library()
    _dev_tensor(logits, "logits")
    if bias is not None:
        _dev_tensor(bias, "bias")
        if bias.dtype != torch.float32:
            raise MoeError(3, "bias must be float32")
    o = _options(options)
    T, E = logits.shape
    k = o.top_k
    dev = logits.device
    if indices is None:
        indices = torch.empty(T, k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, k, dtype=logits.dtype, device=dev)
    w32 = torch.empty(T, k, dtype=torch.float32, device=dev) if weights_fp32 is True else (
        weights_fp32 if isinstance(weights_fp32, torch.Tensor) else None)
    _check(lib.moe_route_sigmoid_grouped(_ptr(logits), _dt(logits), T, E, _ptr(bias), ctypes.byref(o),
                                         _ptr(indices), _ptr(weights), _ptr(w32), _stream(stream)))
    return (indices, weights, w32) if w32 is not None else (indices, weights)


def moe_route_sigmoid_grouped_dispatch(logits: torch.Tensor, bias: torch.Tensor | None, options,
                                       x: torch.Tensor | None = None, *, weights_fp32=False, workspace=None,
                                       stream=None):
    """moe_route_sigmoid_grouped then moe_dispatch as one launch (the same
    outputs, bit for bit): returns (indices, weights[, FP32 weights],
    DispatchedTokens)."""
    lib = load_library()
    _dev_tensor(logits, "logits")
    if bias is not None:
        _dev_tensor(bias, "bias")
        if bias.dtype != torch.float32:
            raise MoeError(3, "bias must be float32")
    o = _options(options)
    T, E = logits.shape
    k = o.top_k
    dev = logits.device
    indices = torch.empty(T, k, dtype=torch.int32, device=dev)
    weights = torch.empty(T, k, dtype=logits.dtype, device=dev)
    w32 = torch.empty(T, k, dtype=torch.float32, device=dev) if weights_fp32 else None
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_src = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    xd = None
    H, xdt = 0, MOE_F32
    if x is not None:
        _dev_tensor(x, "x")
        H, xdt = x.shape[1], _dt(x)
        xd = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    ws = _workspace(lib.moe_route_dispatch_workspace_size(T, E), dev, workspace)
    _check(lib.moe_route_sigmoid_grouped_dispatch(_ptr(logits), _dt(logits), T, E, _ptr(bias), ctypes.byref(o),
                                                  _ptr(indices), _ptr(weights), _ptr(w32), _ptr(x), xdt, H,
                                                  _ptr(counts), _ptr(offsets), _ptr(row_src), _ptr(inv), _ptr(xd),
                                                  _ptr(ws), ws.numel(), _stream(stream)))
    disp = DispatchedTokens(counts, offsets, row_src, inv, xd)
    return (indices, weights, w32, disp) if w32 is not None else (indices, weights, disp)


def moe_forward_sigmoid_grouped(experts: Experts, x: torch.Tensor, logits: torch.Tensor,
                                bias: torch.Tensor | None, options, *, out=None, indices=None, weights=None,
                                workspace=None, stream=None):
    """SwiGluExperts::forward_sigmoid_grouped: the whole chain with grouped
    sigmoid routing, out [T, H]."""
    lib = load_library()
    _dev_tensor(x, "x")
    _dev_tensor(logits, "logits")
    if bias is not None:
        _dev_tensor(bias, "bias")
    o = _options(options)
    T = x.shape[0]
    res = out if out is not None else torch.empty(T, experts.H, dtype=experts.dtype, device=x.device)
    ws = _workspace(lib.moe_forward_workspace_size(experts.handle, T, o.top_k), x.device, workspace)
    _check(lib.moe_forward_sigmoid_grouped(experts.handle, _ptr(x), _ptr(logits), _dt(logits), T, _ptr(bias),
                                           ctypes.byref(o), _ptr(res), _ptr(indices), _ptr(weights), _ptr(ws),
                                           ws.numel(), _stream(stream)))
    return res


def _router_opts(options) -> RouterWeightOptions:
    if isinstance(options, RouterWeightOptions):
        return options
    return RouterWeightOptions(options.scoring, options.renormalize, options.scale)


def _index_type(indices: torch.Tensor) -> int:
    if indices.dtype not in _INDEX:
        raise MoeError(3, f"indices must be uint32, int32 or int64, not {indices.dtype}")
    return _INDEX[indices.dtype]


def moe_router_weights(logits: torch.Tensor, indices: torch.Tensor, options, *, out=None, stream=None):
    """selected_router_weights: FP32 [T, top_k] weights of a fixed selection."""
    lib = load_library()
    _dev_tensor(logits, "logits")
    _dev_tensor(indices, "indices")
    T, E = logits.shape
    k = indices.shape[1]
    o = _router_opts(options)
    w = out if out is not None else torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _check(lib.moe_router_weights(_ptr(logits), _dt(logits), T, E, _ptr(indices), _index_type(indices), k,
                                  ctypes.byref(o), _ptr(w), _stream(stream)))
    return w


def moe_router_backward(logits: torch.Tensor, indices: torch.Tensor, grad_weights: torch.Tensor, options, *,
                        out=None, stream=None):
    """selected_router_backward: dlogits [T, E] in the logits dtype."""
    lib = load_library()
    for name, t in (("logits", logits), ("indices", indices), ("grad_weights", grad_weights)):
        _dev_tensor(t, name)
    if grad_weights.dtype != torch.float32:
        raise MoeError(3, "grad_weights must be float32")
    T, E = logits.shape
    k = indices.shape[1]
    o = _router_opts(options)
    d = out if out is not None else torch.empty_like(logits)
    _check(lib.moe_router_backward(_ptr(logits), _dt(logits), T, E, _ptr(indices), _index_type(indices), k,
                                   ctypes.byref(o), _ptr(grad_weights), _ptr(d), _stream(stream)))
    return d


TrainingCache = namedtuple("TrainingCache", "x_dispatched offsets h g u")


def moe_experts_forward_training(experts: Experts, x_dispatched: torch.Tensor, offsets: torch.Tensor,
                                 workspace=None, stream=None):
    """forward_dispatched_training: (y_dispatched [rows, H], cache) where the
    cache holds what moe_experts_backward needs (h, g, u)."""
    lib = load_library()
    _dev_tensor(x_dispatched, "x_dispatched")
    rows = x_dispatched.shape[0]
    dev = x_dispatched.device
    y = torch.empty(rows, experts.H, dtype=experts.dtype, device=dev)
    h, g, u = (torch.empty(rows, experts.I, dtype=experts.dtype, device=dev) for _ in range(3))
    ws = _workspace(lib.moe_experts_forward_training_workspace_size(experts.handle), dev, workspace)
    _check(lib.moe_experts_forward_training(experts.handle, _ptr(x_dispatched), _ptr(offsets), rows, _ptr(h),
                                            _ptr(y), _ptr(g), _ptr(u), _ptr(ws), ws.numel(), _stream(stream)))
    return y, TrainingCache(x_dispatched, offsets, h, g, u)


ExpertGrads = namedtuple("ExpertGrads", "dx_dispatched dgate dup ddown")


def moe_experts_backward(experts: Experts, cache: TrainingCache, dexpert: torch.Tensor, workspace=None,
                         stream=None) -> ExpertGrads:
    """cache.backward(dexpert): dx_dispatched [rows, H] and FP32 dgate, dup
    [E, I, H] and ddown [E, H, I]."""
    lib = load_library()
    _dev_tensor(dexpert, "dexpert")
    rows = cache.x_dispatched.shape[0]
    dev = dexpert.device
    dx = torch.empty(rows, experts.H, dtype=experts.dtype, device=dev)
    dgate = torch.empty(experts.E, experts.I, experts.H, dtype=torch.float32, device=dev)
    dup = torch.empty_like(dgate)
    ddown = torch.empty(experts.E, experts.H, experts.I, dtype=torch.float32, device=dev)
    ws = _workspace(lib.moe_experts_backward_workspace_size(experts.handle, rows), dev, workspace)
    _check(lib.moe_experts_backward(experts.handle, _ptr(cache.x_dispatched), _ptr(cache.offsets), rows,
                                    _ptr(cache.h), _ptr(cache.g), _ptr(cache.u), _ptr(dexpert), _ptr(dx),
                                    _ptr(dgate), _ptr(dup), _ptr(ddown), _ptr(ws), ws.numel(), _stream(stream)))
    return ExpertGrads(dx, dgate, dup, ddown)


def moe_combine_backward(y_dispatched: torch.Tensor, inv: torch.Tensor, row_src: torch.Tensor,
                         weights: torch.Tensor, grad_out: torch.Tensor, stream=None):
    """combine_backward: (dexpert [rows, H] in y's dtype, dweights [T, top_k]
    FP32). inv and row_src are moe_dispatch's two maps."""
    lib = load_library()
    for name, t in (("y_dispatched", y_dispatched), ("inv", inv), ("row_src", row_src), ("weights", weights),
                    ("grad_out", grad_out)):
        _dev_tensor(t, name)
    T, k = weights.shape
    if inv.numel() != T * k or row_src.numel() != T * k:
        raise MoeError(2, "inv and row_src must hold T * top_k entries")
    H = y_dispatched.shape[1]
    dexp = torch.empty_like(y_dispatched)
    dw = torch.empty(T, k, dtype=torch.float32, device=y_dispatched.device)
    _check(lib.moe_combine_backward(_ptr(y_dispatched), _dt(y_dispatched), _ptr(inv), _ptr(row_src), _ptr(weights),
                                    _dt(weights), _ptr(grad_out), T, k, H, _ptr(dexp), _ptr(dw), _stream(stream)))
    return dexp, dw


def moe_dispatch_backward(dinput: torch.Tensor, inv: torch.Tensor, T: int, top_k: int, stream=None):
    """dispatch_backward: dx [T, H], each token's dispatched rows added in slot order."""
    lib = load_library()
    _dev_tensor(dinput, "dinput")
    _dev_tensor(inv, "inv")
    H = dinput.shape[1]
    dx = torch.empty(T, H, dtype=dinput.dtype, device=dinput.device)
    _check(lib.moe_dispatch_backward(_ptr(dinput), _dt(dinput), _ptr(inv), T, top_k, H, _ptr(dx), _stream(stream)))
    return dx


# ---- experts in microscaled 4-bit floating point (MXFP4)

Mxfp4 = namedtuple("Mxfp4", "codes scales")
Mxfp4.__doc__ = """An MXFP4 matrix [.., K]: codes uint8 [.., K/2] (element 2i in the low half of byte i) and
scales uint8 [.., moe_mxfp4_scale_pitch(K)] (E8M0, one per 32 elements; rows of K / 32 bytes from elsewhere are padded
to the pitch, with any bytes)."""


def _here(stream, *tensors) -> int:
    """The raw stream of a call. The library launches on the current device: tensors of another one are refused
    (host tensors by the callers' own checks)."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise MoeError(7, f"a tensor is on {t.device}, the current device is cuda:{cur}")
    return torch._C._cuda_getCurrentRawStream(cur) if stream is None else stream.cuda_stream


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """torch.empty on the stream the call runs on: memory that an earlier use on another stream may still touch is
    not handed out, and scratch that the call drops is reused in that stream's order only."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(nbytes: int, device, workspace, stream) -> torch.Tensor:
    if workspace is not None:
        return _dev_tensor(workspace, "workspace").view(torch.uint8)
    return _empty((max(int(nbytes), 1),), torch.uint8, device, stream)


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _mx(q, name: str) -> tuple[torch.Tensor, torch.Tensor, int]:
    """(codes, scales, K) of an Mxfp4, checked: contiguous uint8 on the device, shapes that belong together."""
    codes, scales = q
    _dev_tensor(codes, name)
    _dev_tensor(scales, name)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise MoeError(3, f"{name}: codes and scales must be uint8")
    cs, ss = codes.shape, scales.shape
    if len(cs) < 1 or len(ss) != len(cs):
        raise MoeError(2, f"{name}: codes and scales need the same number of dimensions, at least one")
    K = cs[-1] * 2
    if ss[-1] != _pitch(K) or ss[:-1] != cs[:-1]:
        raise MoeError(2, f"{name}: scales {tuple(ss)} do not belong to codes {tuple(cs)}")
    return codes, scales, K


def _pitch(K: int) -> int:
    if K < 32 or K % 32:
        raise MoeError(2, "K must be a positive multiple of 32")
    return (K + 127) // 128 * 4


def moe_mxfp4_scale_pitch(K: int) -> int:
    """Bytes of one row of scales: K / 32 rounded up to 4."""
    pitch = int(load_library().moe_mxfp4_scale_pitch(K))
    if pitch == 0:
        raise MoeError(2, "K must be a positive multiple of 32")
    return pitch


def moe_mxfp4_quantize(x: torch.Tensor, *, inv: torch.Tensor | None = None, top_k: int = 1, out: Mxfp4 | None = None,
                       stream=None) -> Mxfp4:
    """x [.., K] in float32, float16 or bfloat16 as MXFP4 (K a multiple of 32).
    With inv (moe_dispatch's, [T * top_k]) x is [T, K] and row t goes to the
    rows inv[t * top_k + j] of the [T * top_k, K] result: quantised and
    dispatched at once. Rows that no entry of inv names are left as they were
    (not set, without `out`)."""
    lib = load_library()
    _dev_tensor(x, "x")
    shape = x.shape
    if len(shape) < 1:
        raise MoeError(2, "x needs at least one dimension")
    K = shape[-1]
    pitch = _pitch(K)
    rows = x.numel() // K
    lead = shape[:-1]
    if inv is not None:
        _dev_tensor(inv, "inv")
        if len(shape) != 2 or inv.numel() != rows * top_k:
            raise MoeError(2, "inv must hold one entry per slot of x [T, K]")
        if inv.dtype != torch.int32 and inv.dtype != getattr(torch, "uint32", torch.int32):
            raise MoeError(3, "inv must be uint32 (or its int32 view)")
        lead = (rows * top_k,)
    raw = _here(stream, x, inv)
    if out is None:
        codes = _empty((*lead, K // 2), torch.uint8, x.device, stream)
        scales = _empty((*lead, pitch), torch.uint8, x.device, stream)
        out = Mxfp4(codes, scales)
    else:
        codes, scales, k_out = _mx(out, "out")
        if k_out != K or codes.numel() * 2 != (rows * top_k if inv is not None else rows) * K:
            raise MoeError(2, "out does not have the result's shape")
        _here(stream, codes, scales)
    _check(lib.moe_mxfp4_quantize(x.data_ptr(), _dt(x), rows, K, _addr(inv), top_k, codes.data_ptr(),
                                  scales.data_ptr(), raw))
    return out


def moe_mxfp4_dequantize(q: Mxfp4, dtype: torch.dtype = torch.bfloat16, *, out=None, stream=None) -> torch.Tensor:
    """The values an MXFP4 matrix stands for, [.., K] in `dtype`."""
    lib = load_library()
    codes, scales, K = _mx(q, "q")
    raw = _here(stream, codes, scales)
    if out is None:
        out = _empty((*codes.shape[:-1], K), dtype, codes.device, stream)
    else:
        _dev_tensor(out, "out")
        if out.dtype != dtype or out.numel() != codes.numel() * 2:
            raise MoeError(2, "out does not have the result's shape and dtype")
        _here(stream, out)
    _check(lib.moe_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), codes.numel() * 2 // K, K, out.data_ptr(),
                                    _dt(out), raw))
    return out


class ExpertsMxfp4:
    """SwiGLU experts in MXFP4: a handle over gate/up [E, I, H] and down
    [E, H, I] (Mxfp4 tensors; the codes are kept alive here, the scales are
    laid out once for the tensor cores). Waits for its set-up, so that the
    handle can be used on any stream, and may be dropped while a call's work
    is still queued: its memory is handed out again only after the streams that
    used it. A captured graph is not such a stream: the handle has to outlive
    its replays. Not to be made during a graph capture."""

    def __init__(self, gate: Mxfp4, up: Mxfp4, down: Mxfp4):
        lib = load_library()
        (gc, gs, H), (uc, us, Hu), (dc, ds, I) = _mx(gate, "gate"), _mx(up, "up"), _mx(down, "down")
        if gc.dim() != 3:
            raise MoeError(2, "gate must be [E, I, H]")
        E = gc.shape[0]
        if (tuple(gc.shape) != (E, I, H // 2) or tuple(uc.shape) != tuple(gc.shape) or Hu != H or
                tuple(dc.shape) != (E, H, I // 2)):
            raise MoeError(2, "gate and up must be [E, I, H] and down [E, H, I]")
        _here(None, gc, gs, uc, us, dc, ds)
        self.E, self.H, self.I = E, H, I
        self.device = gc.device
        self._codes = (gc, uc, dc)
        self._streams = set()   # the raw streams that the allocator knows as users of the codes and scales
        self._storage = torch.empty(max(1, lib.moe_experts_mxfp4_storage_size(E, H, I)), dtype=torch.uint8,
                                    device=gc.device)
        handle = ctypes.c_void_p()
        _check(lib.moe_experts_mxfp4_create(_ptr(gc), _ptr(gs), _ptr(uc), _ptr(us), _ptr(dc), _ptr(ds), E, H, I,
                                            _ptr(self._storage), self._storage.numel(), _stream(),
                                            ctypes.byref(handle)))
        self.handle = handle
        torch.cuda.current_stream().synchronize()

    @classmethod
    def from_float(cls, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor) -> "ExpertsMxfp4":
        """Quantise float gate/up [E, I, H] and down [E, H, I]."""
        return cls(*(moe_mxfp4_quantize(t) for t in (gate, up, down)))

    def _used_on(self, raw: int, stream) -> None:
        """Tells the allocator, once per stream, that a call reads the codes and scales on it: a handle that is
        dropped with work queued there keeps its blocks until that work is done."""
        if raw not in self._streams:
            s = torch.cuda.current_stream() if stream is None else stream
            for t in (*self._codes, self._storage):
                t.record_stream(s)
            self._streams.add(raw)

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_experts_mxfp4_destroy(self.handle)
            self.handle = None


def _mx_rows(experts: ExpertsMxfp4, q: Mxfp4, name: str, K: int, offsets: torch.Tensor):
    """(codes, scales, rows) of dispatched MXFP4 rows, with the experts' offsets checked."""
    codes, scales, k = _mx(q, name)
    if codes.dim() != 2 or k != K:
        raise MoeError(2, f"{name} must be [rows, {K}]")
    _dev_tensor(offsets, "offsets")
    if offsets.dtype != torch.int32 and offsets.dtype != getattr(torch, "uint32", torch.int32):
        raise MoeError(3, "offsets must be uint32 (or its int32 view)")
    if offsets.numel() != experts.E + 1:
        raise MoeError(2, "offsets must hold E + 1 entries")
    return codes, scales, codes.shape[0]


def _mx_out(out, rows: int, cols: int, dtype: torch.dtype, device, stream) -> torch.Tensor:
    if out is None:
        return _empty((rows, cols), dtype, device, stream)
    _dev_tensor(out, "out")
    if out.dtype != dtype or tuple(out.shape) != (rows, cols):
        raise MoeError(2, f"out must be [{rows}, {cols}] in {dtype}")
    _here(stream, out)
    return out


def moe_experts_mxfp4_gate_up(experts: ExpertsMxfp4, x: Mxfp4, offsets: torch.Tensor, *,
                              dtype: torch.dtype = torch.bfloat16, quantized: bool = False, out=None, stream=None):
    """First stage on dispatched MXFP4 rows: h [rows, I] = SiLU(x W_gate^T) *
    (x W_up^T) per expert in `dtype`, or with quantized=True h rounded to
    `dtype` and quantised, an Mxfp4 (what moe_mxfp4_quantize gives on h)."""
    lib = load_library()
    codes, scales, rows = _mx_rows(experts, x, "x", experts.H, offsets)
    raw = _here(stream, codes, scales, offsets)
    experts._used_on(raw, stream)
    if dtype not in _DTYPE:
        raise MoeError(3, f"unsupported dtype {dtype}")
    h, hc, hs = None, None, None
    if quantized:
        if out is None:
            out = Mxfp4(_empty((rows, experts.I // 2), torch.uint8, codes.device, stream),
                        _empty((rows, _pitch(experts.I)), torch.uint8, codes.device, stream))
        hc, hs, k = _mx(out, "out")
        if k != experts.I or hc.dim() != 2 or hc.shape[0] != rows:
            raise MoeError(2, f"out must be [{rows}, {experts.I}]")
        _here(stream, hc, hs)
    else:
        out = h = _mx_out(out, rows, experts.I, dtype, codes.device, stream)
    _check(lib.moe_experts_mxfp4_gate_up(experts.handle, codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(), rows,
                                         _DTYPE[dtype], _addr(h), _addr(hc), _addr(hs), raw))
    return out


def moe_experts_mxfp4_down(experts: ExpertsMxfp4, h: Mxfp4, offsets: torch.Tensor, *,
                           dtype: torch.dtype = torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """Second stage: y [rows, H] = h W_down^T per expert, from MXFP4 h."""
    lib = load_library()
    codes, scales, rows = _mx_rows(experts, h, "h", experts.I, offsets)
    raw = _here(stream, codes, scales, offsets)
    experts._used_on(raw, stream)
    y = _mx_out(out, rows, experts.H, dtype, codes.device, stream)
    _check(lib.moe_experts_mxfp4_down(experts.handle, codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(), rows,
                                      _dt(y), y.data_ptr(), raw))
    return y


def moe_experts_mxfp4_forward_dispatched(experts: ExpertsMxfp4, x: Mxfp4, offsets: torch.Tensor, *,
                                         dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                                         stream=None) -> torch.Tensor:
    """Both stages on dispatched MXFP4 rows: y [rows, H] in `dtype`; h passes
    between them as MXFP4 (rounded to `dtype` first)."""
    lib = load_library()
    codes, scales, rows = _mx_rows(experts, x, "x", experts.H, offsets)
    raw = _here(stream, codes, scales, offsets, workspace)
    experts._used_on(raw, stream)
    y = _mx_out(out, rows, experts.H, dtype, codes.device, stream)
    need = lib.moe_experts_mxfp4_forward_dispatched_workspace_size(experts.handle, rows)
    ws = _scratch(need, codes.device, workspace, stream)
    _check(lib.moe_experts_mxfp4_forward_dispatched(experts.handle, codes.data_ptr(), scales.data_ptr(),
                                                    offsets.data_ptr(), rows, _dt(y), y.data_ptr(), ws.data_ptr(),
                                                    ws.numel(), raw))
    return y


def moe_forward_mxfp4(experts: ExpertsMxfp4, x: torch.Tensor, logits: torch.Tensor, top_k: int, renormalize: bool, *,
                      out=None, indices=None, weights=None, workspace=None, stream=None) -> torch.Tensor:
    """The whole local chain on MXFP4 experts: x [T, H] (float32, float16 or
    bfloat16) is routed, quantised into dispatched order, run through the
    experts' 4-bit products and combined to out [T, H] in x's dtype. indices
    and weights, where given, receive the routing: T * top_k entries, uint32
    (or its int32 view) and the logits' dtype."""
    lib = load_library()
    _dev_tensor(x, "x")
    _dev_tensor(logits, "logits")
    if x.dim() != 2 or x.shape[1] != experts.H:
        raise MoeError(2, f"x must be [T, {experts.H}]")
    T = x.shape[0]
    if tuple(logits.shape) != (T, experts.E):
        raise MoeError(2, f"logits must be [{T}, {experts.E}]")
    for t, name in ((indices, "indices"), (weights, "weights")):
        if t is not None and _dev_tensor(t, name).numel() != T * top_k:
            raise MoeError(2, f"{name} must hold T * top_k entries")
    if indices is not None and indices.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)):
        raise MoeError(3, "indices must be uint32 (or its int32 view)")
    if weights is not None and weights.dtype != logits.dtype:
        raise MoeError(3, f"weights must be in the logits' dtype, {logits.dtype}")
    raw = _here(stream, x, logits, indices, weights, workspace)
    experts._used_on(raw, stream)
    o = _mx_out(out, T, experts.H, x.dtype, x.device, stream)
    ws = _scratch(lib.moe_forward_mxfp4_workspace_size(experts.handle, T, top_k, _dt(x)), x.device, workspace, stream)
    _check(lib.moe_forward_mxfp4(experts.handle, x.data_ptr(), _dt(x), logits.data_ptr(), _dt(logits), T, top_k,
                                 int(bool(renormalize)), o.data_ptr(), _addr(indices), _addr(weights), ws.data_ptr(),
                                 ws.numel(), raw))
    return o


# ---- gradient norm and clipping

def _grad_table(tensors, out, cur: int) -> array:
    """The moe_grad_tensor array of a list of gradients and of their destinations (`out` is the same list to clip in
    place): rows of four 64-bit words, the dtype code in the low half of the last. Column by column, because a
    model's list is long and this is the call's host time."""
    lists = (tensors,) if out is tensors else (tensors, out)
    for ts in lists:
        if not all([t.is_contiguous() for t in ts]):
            raise ValueError("gradients must be contiguous CUDA tensors")
        if any([t.get_device() != cur for t in ts]):
            raise MoeError(7, f"a gradient is not on the current device, cuda:{cur}")
    numel = [t.numel() for t in tensors]
    dtypes = [t.dtype for t in tensors]
    src = dst = [t.data_ptr() for t in tensors]
    if out is not tensors:
        if len(out) != len(tensors):
            raise MoeError(2, "out must hold one tensor per gradient")
        if [t.numel() for t in out] != numel or [t.dtype for t in out] != dtypes:
            raise MoeError(2, "out must have the gradients' sizes and dtypes")
        dst = [t.data_ptr() for t in out]
    try:
        codes = [_DTYPE[d] for d in dtypes]
    except KeyError as e:
        raise MoeError(3, f"unsupported dtype {e.args[0]}") from None
    table = array("q", bytes(32 * max(1, len(src))))
    n = len(src)
    for i, column in enumerate((src, dst, numel, codes)):
        table[i:4 * n:4] = array("q", column)
    return table


def _grad_norm(lib, table, n: int, cur: int, out, workspace, stream, raw) -> torch.Tensor:
    device = torch.device("cuda", cur)
    norm = out if out is not None else _empty((), torch.float32, device, stream)
    ws = _scratch(lib.moe_grad_norm_workspace_size(n), device, workspace, stream)
    _check(lib.moe_grad_norm(table.buffer_info()[0], n, norm.data_ptr(), ws.data_ptr(), ws.numel(), raw))
    return norm


def _one_float(t: torch.Tensor):
    _dev_tensor(t, "norm")
    if t.dtype != torch.float32 or t.numel() != 1:
        raise MoeError(3, "the norm must be one float32")
    return t


def moe_grad_norm(tensors, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """The L2 norm over all elements of a list of float32, float16 or bfloat16
    gradients, one float32 on the device (nothing waits for it)."""
    lib = load_library()
    tensors = list(tensors)
    if tensors and not tensors[0].is_cuda:
        raise ValueError("gradients must be contiguous CUDA tensors")
    raw = _here(stream, out if out is None else _one_float(out), workspace)
    cur = torch.cuda.current_device()
    return _grad_norm(lib, _grad_table(tensors, tensors, cur), len(tensors), cur, out, workspace, stream, raw)


def moe_grad_clip(tensors, norm: torch.Tensor, max_norm: float, *, out=None, stream=None):
    """Every gradient times max_norm / norm where norm (one float32 on the
    device, as moe_grad_norm gives it) is finite and larger than max_norm; in
    place, or into the list `out`. Returns the clipped list."""
    lib = load_library()
    tensors = list(tensors)
    out = tensors if out is None else list(out)
    raw = _here(stream, _one_float(norm))
    table = _grad_table(tensors, out, torch.cuda.current_device())
    _check(lib.moe_grad_clip(table.buffer_info()[0], len(tensors), norm.data_ptr(), float(max_norm), raw))
    return out


def moe_clip_grad_norm(tensors, max_norm: float, *, out=None, workspace=None, stream=None) -> torch.Tensor:
    """moe_grad_norm and moe_grad_clip in turn: returns the norm before the clip."""
    lib = load_library()
    tensors = list(tensors)
    if tensors and not tensors[0].is_cuda:
        raise ValueError("gradients must be contiguous CUDA tensors")
    raw = _here(stream, workspace)
    cur = torch.cuda.current_device()
    table = _grad_table(tensors, tensors if out is None else list(out), cur)
    norm = _grad_norm(lib, table, len(tensors), cur, None, workspace, stream, raw)
    _check(lib.moe_grad_clip(table.buffer_info()[0], len(tensors), norm.data_ptr(), float(max_norm), raw))
    return norm


def moe_device_status(clear: bool = True) -> int:
    code = ctypes.c_uint32(0)
    _check(load_library().moe_device_status(ctypes.byref(code), int(clear)))
    return code.value


def moe_selftest_bounded_wait(limit_us: int, stream=None):
    _check(load_library().moe_selftest_bounded_wait(limit_us, _stream(stream)))
