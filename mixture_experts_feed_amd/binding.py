"""ctypes binding of libinkling_moe.so (argument marshalling only).

Every step of the layer runs in the HIP library; torch supplies device memory
and the current stream.  Names mirror the C ABI in include/inkling_moe.h.
If the library is missing this module raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libinkling_moe.so")

INKLING_OK = 0
INKLING_ERR_INVALID_ARGUMENT = -1
INKLING_ERR_UNSUPPORTED = -2
INKLING_ERR_WORKSPACE = -3
INKLING_ERR_HIP = -4
INKLING_ERR_TOO_LARGE = -5
INKLING_NOALLOC_SCRATCH_BYTES = 64 << 20
INKLING_F32 = 0
INKLING_BF16 = 1

EXPORTED = ("inkling_moe_workspace_size", "inkling_moe_route", "inkling_moe_forward",
            "inkling_moe_strerror", "inkling_moe_last_hip_error", "inkling_moe_set_stage_events",
            "inkling_dense_mlp_workspace_size", "inkling_dense_mlp_forward",
            "inkling_moe_backward_workspace_size", "inkling_moe_backward", "inkling_moe_saved_size",
            "inkling_moe_forward_train", "inkling_moe_forward_noalloc",
            "inkling_grouped_workspace_size", "inkling_grouped_weight_grad_workspace_size",
            "inkling_grouped_linear", "inkling_grouped_input_grad", "inkling_grouped_weight_grad",
            "inkling_swiglu_checkpoint_size", "inkling_swiglu_forward", "inkling_swiglu_backward",
            "inkling_norm_forward", "inkling_norm_backward_workspace_size", "inkling_norm_backward")
INKLING_NORM_LAYER = 0
INKLING_NORM_RMS = 1
NORM_KINDS = {"layer": INKLING_NORM_LAYER, "rms": INKLING_NORM_RMS}
INKLING_STAGE_EVENTS = 7
STAGES = ("router_logits", "router_select", "permutation", "gate_up", "down", "shared_down_combine")


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("hidden", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class DenseDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class Grads(ctypes.Structure):
    _fields_ = [("d_gate_bank", ctypes.c_void_p), ("d_routed_gate_up", ctypes.c_void_p),
                ("d_routed_down", ctypes.c_void_p), ("d_shared_gate_up", ctypes.c_void_p),
                ("d_shared_down", ctypes.c_void_p), ("weight_grad_dtype", ctypes.c_int32)]


class GroupedDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("x_rows", ctypes.c_int64), ("n_groups", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class SwigluDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("intermediate", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("hidden", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class Gate(ctypes.Structure):
    _fields_ = [("gate_bank", ctypes.c_void_p), ("correction_bias", ctypes.c_void_p),
                ("route_scale", ctypes.c_float), ("global_scale", ctypes.c_float)]


class Experts(ctypes.Structure):
    _fields_ = [("routed_gate_up", ctypes.c_void_p), ("routed_down", ctypes.c_void_p),
                ("shared_gate_up", ctypes.c_void_p), ("shared_down", ctypes.c_void_p)]


class RouteOut(ctypes.Structure):
    _fields_ = [("topk_indices", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
                ("shared_gammas", ctypes.c_void_p), ("expert_counts", ctypes.c_void_p),
                ("expert_offsets", ctypes.c_void_p), ("sorted_slots", ctypes.c_void_p)]


class InklingError(RuntimeError):
    def __init__(self, code: int, where: str):
        lib = load()
        msg = lib.inkling_moe_strerror(code).decode()
        if code == INKLING_ERR_HIP:
            msg += f" (hipError {lib.inkling_moe_last_hip_error()})"
        super().__init__(f"{where}: {msg} [{code}]")
        self.code = code


_LIB: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load the in-tree HIP library (built by mixture_experts_feed_amd.build)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m mixture_experts_feed_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.inkling_moe_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ctypes.c_size_t)]
    lib.inkling_moe_workspace_size.restype = ctypes.c_int
    lib.inkling_moe_route.argtypes = [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.POINTER(Gate), ctypes.c_void_p,
                                      ctypes.POINTER(RouteOut), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.inkling_moe_route.restype = ctypes.c_int
    lib.inkling_moe_forward.argtypes = [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.POINTER(Gate),
                                        ctypes.POINTER(Experts), ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.POINTER(RouteOut), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.inkling_moe_forward.restype = ctypes.c_int
    lib.inkling_moe_forward_noalloc.argtypes = [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.POINTER(Gate),
                                                ctypes.POINTER(Experts), ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.POINTER(RouteOut), ctypes.c_void_p]
    lib.inkling_moe_forward_noalloc.restype = ctypes.c_int
    lib.inkling_moe_strerror.argtypes = [ctypes.c_int]
    lib.inkling_moe_strerror.restype = ctypes.c_char_p
    lib.inkling_moe_last_hip_error.argtypes = []
    lib.inkling_moe_last_hip_error.restype = ctypes.c_int
    lib.inkling_moe_set_stage_events.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.inkling_moe_set_stage_events.restype = ctypes.c_int
    lib.inkling_dense_mlp_workspace_size.argtypes = [ctypes.POINTER(DenseDims), ctypes.POINTER(ctypes.c_size_t)]
    lib.inkling_dense_mlp_workspace_size.restype = ctypes.c_int
    lib.inkling_dense_mlp_forward.argtypes = [ctypes.POINTER(DenseDims), ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_size_t, ctypes.c_void_p]
    lib.inkling_dense_mlp_forward.restype = ctypes.c_int
    lib.inkling_moe_backward_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ctypes.c_size_t)]
    lib.inkling_moe_backward_workspace_size.restype = ctypes.c_int
    lib.inkling_moe_backward.argtypes = [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.POINTER(Gate),
                                         ctypes.POINTER(Experts), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.POINTER(Grads), ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]
    lib.inkling_moe_backward.restype = ctypes.c_int
    lib.inkling_moe_saved_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ctypes.c_size_t)]
    lib.inkling_moe_saved_size.restype = ctypes.c_int
    lib.inkling_moe_forward_train.argtypes = [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.POINTER(Gate),
                                              ctypes.POINTER(Experts), ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.inkling_moe_forward_train.restype = ctypes.c_int
    ptr, size = ctypes.c_void_p, ctypes.c_size_t
    gdims, sdims, ndims = (ctypes.POINTER(c) for c in (GroupedDims, SwigluDims, NormDims))
    for name, args in (
            ("inkling_grouped_workspace_size", [gdims, ctypes.POINTER(size)]),
            ("inkling_grouped_weight_grad_workspace_size", [gdims, ctypes.POINTER(size)]),
            ("inkling_grouped_linear", [gdims, ptr, ptr, ptr, ptr, ptr, ptr, size, ptr]),
            ("inkling_grouped_input_grad", [gdims, ptr, ptr, ptr, ptr, ptr, size, ptr]),
            ("inkling_grouped_weight_grad", [gdims, ptr, ptr, ptr, ptr, ptr, ptr, size, ptr]),
            ("inkling_swiglu_checkpoint_size", [sdims, ctypes.POINTER(size)]),
            ("inkling_swiglu_forward", [sdims, ptr, ptr, ptr, ptr, ptr, size, ptr]),
            ("inkling_swiglu_backward", [sdims, ptr, ptr, size, ptr, ptr, ptr, ptr, ptr, ptr]),
            ("inkling_norm_forward", [ndims, ptr, ptr, ptr, ptr, ptr, ptr]),
            ("inkling_norm_backward_workspace_size", [ndims, ctypes.POINTER(size)]),
            ("inkling_norm_backward", [ndims, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr, size, ptr])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    _LIB = lib
    return lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return INKLING_F32
    if dt == torch.bfloat16:
        return INKLING_BF16
    raise ValueError(f"unsupported dtype {dt}")


def _ints32(*sizes):
    """Ints that C int32 fields hold (ctypes would keep their low 32 bits)."""
    sizes = [int(v) for v in sizes]
    if max(sizes) >= 2 ** 31 or min(sizes) < -2 ** 31:
        raise ValueError(f"sizes must fit in 32 bits, got {sizes}")
    return sizes


def make_dims(T, hidden, n_routed, top_k, n_shared, intermediate, dtype, out_dtype=None) -> Dims:
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    ocode = code if out_dtype is None else (out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype))
    return Dims(int(T), *_ints32(hidden, n_routed, top_k, n_shared, intermediate), code, ocode)


def workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    rc = load().inkling_moe_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_workspace_size")
    return int(n.value)


# the stream's handle without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def alloc_workspace(dims: Dims, device) -> torch.Tensor:
    return torch.empty(max(1, workspace_size(dims)), dtype=torch.uint8, device=device)


def route(x: torch.Tensor, gate_bank: torch.Tensor, bias: torch.Tensor, top_k: int, route_scale: float,
          global_scale: float, padding_mask: Optional[torch.Tensor] = None, permutation: bool = True,
          workspace: Optional[torch.Tensor] = None, intermediate: int = 64):
    """inkling_moe_route: returns dict(topk_indices, topk_weights, shared_gammas[, expert_counts,
    expert_offsets, sorted_slots])."""
    T, H = x.shape
    E = bias.shape[0]
    S = gate_bank.shape[0] - E
    _need(x, "x")
    _need(gate_bank, "gate_bank", torch.float32)
    _need(bias, "bias", torch.float32)
    dims = make_dims(T, H, E, top_k, S, intermediate, x.dtype)
    dev = x.device
    res = {
        "topk_indices": torch.empty((T, top_k), dtype=torch.int32, device=dev),
        "topk_weights": torch.empty((T, top_k), dtype=torch.float32, device=dev),
        "shared_gammas": torch.empty((T, S), dtype=torch.float32, device=dev),
    }
    if permutation:
        res["expert_counts"] = torch.empty((E,), dtype=torch.int32, device=dev)
        res["expert_offsets"] = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        res["sorted_slots"] = torch.full((max(1, T * top_k),), -1, dtype=torch.int32, device=dev)
    ro = RouteOut(*[_ptr(res.get(n)) for n in ("topk_indices", "topk_weights", "shared_gammas", "expert_counts",
                                               "expert_offsets", "sorted_slots")])
    gate = Gate(gate_bank.data_ptr(), bias.data_ptr(), float(route_scale), float(global_scale))
    if padding_mask is not None:
        _need(padding_mask, "padding_mask", torch.uint8)
    if workspace is None:
        workspace = alloc_workspace(dims, dev)
    rc = load().inkling_moe_route(ctypes.byref(dims), x.data_ptr(), ctypes.byref(gate), _ptr(padding_mask),
                                  ctypes.byref(ro), workspace.data_ptr(), workspace.numel(), _stream(dev))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_route")
    return res


def _forward_args(x, gate_bank, bias, w_gu, w_d, wsh_gu, wsh_d, top_k, route_scale, global_scale, padding_mask,
                  out, return_routing, out_dtype):
    """Checks and C structs shared by forward() and forward_noalloc()."""
    T, H = x.shape
    E, twoI, _ = w_gu.shape
    S = 0 if wsh_gu is None else wsh_gu.shape[0]
    for t, n in ((x, "x"), (w_gu, "w_gu"), (w_d, "w_d")):
        _need(t, n, x.dtype)
    if S:
        _need(wsh_gu, "wsh_gu", x.dtype)
        _need(wsh_d, "wsh_d", x.dtype)
    _need(gate_bank, "gate_bank", torch.float32)
    _need(bias, "bias", torch.float32)
    if gate_bank.shape[0] != E + S:
        raise ValueError("gate_bank must hold n_routed + n_shared rows")
    if out is not None:
        out_dtype = out.dtype
    out_dtype = x.dtype if out_dtype is None else out_dtype
    dims = make_dims(T, H, E, top_k, S, twoI // 2, x.dtype, out_dtype)
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype)
    if padding_mask is not None:
        _need(padding_mask, "padding_mask", torch.uint8)
    routing = None
    ro = None
    if return_routing:
        routing = {
            "topk_indices": torch.empty((T, top_k), dtype=torch.int32, device=dev),
            "topk_weights": torch.empty((T, top_k), dtype=torch.float32, device=dev),
            "shared_gammas": torch.empty((T, S), dtype=torch.float32, device=dev),
            "expert_counts": torch.empty((E,), dtype=torch.int32, device=dev),
            "expert_offsets": torch.empty((E + 1,), dtype=torch.int32, device=dev),
            "sorted_slots": torch.full((max(1, T * top_k),), -1, dtype=torch.int32, device=dev),
        }
        ro = RouteOut(*[_ptr(routing[n]) for n in ("topk_indices", "topk_weights", "shared_gammas",
                                                   "expert_counts", "expert_offsets", "sorted_slots")])
    gate = Gate(gate_bank.data_ptr(), bias.data_ptr(), float(route_scale), float(global_scale))
    ex = Experts(w_gu.data_ptr(), w_d.data_ptr(), _ptr(wsh_gu) if S else None, _ptr(wsh_d) if S else None)
    return dims, gate, ex, out, routing, ro


def forward(x: torch.Tensor, gate_bank: torch.Tensor, bias: torch.Tensor, w_gu: torch.Tensor, w_d: torch.Tensor,
            wsh_gu: Optional[torch.Tensor], wsh_d: Optional[torch.Tensor], top_k: int, route_scale: float,
            global_scale: float, padding_mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, return_routing: bool = False,
            out_dtype: Optional[torch.dtype] = None, saved: Optional[torch.Tensor] = None):
    """inkling_moe_forward: out [T, H] (x's dtype unless out / out_dtype says
    otherwise) and the routing dict if asked.  With `saved` (uint8, saved_size
    bytes) it is inkling_moe_forward_train, which also keeps the gate_up
    projections there for backward()."""
    dims, gate, ex, out, routing, ro = _forward_args(x, gate_bank, bias, w_gu, w_d, wsh_gu, wsh_d, top_k,
                                                     route_scale, global_scale, padding_mask, out, return_routing,
                                                     out_dtype)
    dev = x.device
    if workspace is None:
        workspace = alloc_workspace(dims, dev)
    if saved is not None:
        if return_routing:
            raise ValueError("the training forward does not return the routing")
        if saved.dtype != torch.uint8 or not saved.is_contiguous() or saved.numel() < saved_size(dims):
            raise ValueError("saved must be a contiguous uint8 tensor of saved_size(dims) bytes")
        rc = load().inkling_moe_forward_train(ctypes.byref(dims), x.data_ptr(), ctypes.byref(gate), ctypes.byref(ex),
                                              _ptr(padding_mask), out.data_ptr(), saved.data_ptr(),
                                              workspace.data_ptr(), workspace.numel(), _stream(dev))
        if rc != INKLING_OK:
            raise InklingError(rc, "inkling_moe_forward_train")
        return out
    rc = load().inkling_moe_forward(ctypes.byref(dims), x.data_ptr(), ctypes.byref(gate), ctypes.byref(ex),
                                    _ptr(padding_mask), out.data_ptr(), None if ro is None else ctypes.byref(ro),
                                    workspace.data_ptr(), workspace.numel(), _stream(dev))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_forward")
    return (out, routing) if return_routing else out


def forward_noalloc(x: torch.Tensor, gate_bank: torch.Tensor, bias: torch.Tensor, w_gu: torch.Tensor,
                    w_d: torch.Tensor, wsh_gu: Optional[torch.Tensor], wsh_d: Optional[torch.Tensor], top_k: int,
                    route_scale: float, global_scale: float, padding_mask: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, return_routing: bool = False,
                    out_dtype: Optional[torch.dtype] = None):
    """inkling_moe_forward_noalloc: forward() without a workspace (the
    library's static scratch of INKLING_NOALLOC_SCRATCH_BYTES per GPU).  With
    `out` given and no routing asked for, this allocates nothing."""
    dims, gate, ex, out, routing, ro = _forward_args(x, gate_bank, bias, w_gu, w_d, wsh_gu, wsh_d, top_k,
                                                     route_scale, global_scale, padding_mask, out, return_routing,
                                                     out_dtype)
    rc = load().inkling_moe_forward_noalloc(ctypes.byref(dims), x.data_ptr(), ctypes.byref(gate), ctypes.byref(ex),
                                            _ptr(padding_mask), out.data_ptr(),
                                            None if ro is None else ctypes.byref(ro), _stream(x.device))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_forward_noalloc")
    return (out, routing) if return_routing else out


def saved_size(dims: Dims) -> int:
    """inkling_moe_saved_size: bytes of the activations the training forward keeps."""
    n = ctypes.c_size_t(0)
    rc = load().inkling_moe_saved_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_saved_size")
    return n.value


def set_stage_events(events: Optional[ctypes.Array]) -> None:
    """Install (or clear with None) an array of INKLING_STAGE_EVENTS hipEvent_t
    handles recorded by later forward calls on this thread."""
    n = 0 if events is None else len(events)
    rc = load().inkling_moe_set_stage_events(None if events is None else ctypes.cast(events, ctypes.c_void_p), n)
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_set_stage_events")


def make_dense_dims(T, hidden, intermediate, dtype, out_dtype=None) -> DenseDims:
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    ocode = code if out_dtype is None else (out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype))
    return DenseDims(int(T), *_ints32(hidden, intermediate), code, ocode)


def dense_workspace_size(dims: DenseDims) -> int:
    n = ctypes.c_size_t(0)
    rc = load().inkling_dense_mlp_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_dense_mlp_workspace_size")
    return int(n.value)


def dense_mlp_forward(x: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, global_scale: float,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """inkling_dense_mlp_forward: InklingDenseMLP on x [T, H] with gate_up
    [2I, H] (interleaved) and down [H, I]."""
    T, H = x.shape
    twoI = gate_up.shape[0]
    for t, n in ((x, "x"), (gate_up, "gate_up"), (down, "down")):
        _need(t, n, x.dtype)
    if gate_up.shape != (twoI, H) or down.shape != (H, twoI // 2):
        raise ValueError("gate_up must be [2I, H] and down [H, I]")
    if out is not None:
        out_dtype = out.dtype
    out_dtype = x.dtype if out_dtype is None else out_dtype
    dims = make_dense_dims(T, H, twoI // 2, x.dtype, out_dtype)
    dev = x.device
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype)
    if workspace is None:
        workspace = torch.empty(max(1, dense_workspace_size(dims)), dtype=torch.uint8, device=dev)
    rc = load().inkling_dense_mlp_forward(ctypes.byref(dims), x.data_ptr(), gate_up.data_ptr(), down.data_ptr(),
                                          float(global_scale), out.data_ptr(), workspace.data_ptr(),
                                          workspace.numel(), _stream(dev))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_dense_mlp_forward")
    return out


def backward_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    rc = load().inkling_moe_backward_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_backward_workspace_size")
    return int(n.value)


def backward(x: torch.Tensor, gate_bank: torch.Tensor, bias: torch.Tensor, w_gu: torch.Tensor, w_d: torch.Tensor,
             wsh_gu: Optional[torch.Tensor], wsh_d: Optional[torch.Tensor], top_k: int, route_scale: float,
             global_scale: float, dout: torch.Tensor, padding_mask: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, dx_dtype: Optional[torch.dtype] = None,
             grads: Optional[dict] = None, saved: Optional[torch.Tensor] = None,
             weight_grad_dtype: Optional[torch.dtype] = None) -> dict:
    """inkling_moe_backward: dict(dx, d_gate_bank, d_w_gu, d_w_d, d_wsh_gu, d_wsh_d).
    `saved`: the tensor a training forward with the same arguments filled, or
    None to recompute the gate_up projections.  The weight gradients are fp32
    (default) or bf16 (`weight_grad_dtype`, or the dtype of the given
    `grads` tensors)."""
    T, H = x.shape
    E, twoI, _ = w_gu.shape
    S = 0 if wsh_gu is None else wsh_gu.shape[0]
    for t, n in ((x, "x"), (w_gu, "w_gu"), (w_d, "w_d"), (dout, "dout")):
        _need(t, n, x.dtype)
    if S:
        _need(wsh_gu, "wsh_gu", x.dtype)
        _need(wsh_d, "wsh_d", x.dtype)
    _need(gate_bank, "gate_bank", torch.float32)
    _need(bias, "bias", torch.float32)
    dx_dtype = x.dtype if dx_dtype is None else dx_dtype
    dims = make_dims(T, H, E, top_k, S, twoI // 2, x.dtype, dx_dtype)
    dev = x.device
    if grads is None:
        wdt = dict(dtype=torch.float32 if weight_grad_dtype is None else weight_grad_dtype, device=dev)
        grads = {"dx": torch.empty((T, H), dtype=dx_dtype, device=dev),
                 "d_gate_bank": torch.empty(tuple(gate_bank.shape), dtype=torch.float32, device=dev),
                 "d_w_gu": torch.empty(tuple(w_gu.shape), **wdt), "d_w_d": torch.empty(tuple(w_d.shape), **wdt),
                 "d_wsh_gu": torch.empty(tuple(wsh_gu.shape), **wdt) if S else None,
                 "d_wsh_d": torch.empty(tuple(wsh_d.shape), **wdt) if S else None}
    wdtype = grads["d_w_gu"].dtype
    if weight_grad_dtype is not None and weight_grad_dtype != wdtype:
        raise ValueError("weight_grad_dtype differs from the dtype of the given gradient tensors")
    for n in ("d_w_d", "d_wsh_gu", "d_wsh_d"):
        if grads[n] is not None and grads[n].dtype != wdtype:
            raise ValueError("the four weight gradients must share one dtype")
    g = Grads(_ptr(grads["d_gate_bank"]), _ptr(grads["d_w_gu"]), _ptr(grads["d_w_d"]), _ptr(grads["d_wsh_gu"]),
              _ptr(grads["d_wsh_d"]), _dtype_code(wdtype))
    gate = Gate(gate_bank.data_ptr(), bias.data_ptr(), float(route_scale), float(global_scale))
    ex = Experts(w_gu.data_ptr(), w_d.data_ptr(), _ptr(wsh_gu) if S else None, _ptr(wsh_d) if S else None)
    if padding_mask is not None:
        _need(padding_mask, "padding_mask", torch.uint8)
    if workspace is None:
        workspace = torch.empty(max(1, backward_workspace_size(dims)), dtype=torch.uint8, device=dev)
    if saved is not None and (saved.dtype != torch.uint8 or saved.numel() < saved_size(dims)):
        raise ValueError("saved must be the uint8 tensor of saved_size(dims) bytes a training forward filled")
    rc = load().inkling_moe_backward(ctypes.byref(dims), x.data_ptr(), ctypes.byref(gate), ctypes.byref(ex),
                                     _ptr(padding_mask), dout.data_ptr(), _ptr(saved), grads["dx"].data_ptr(),
                                     ctypes.byref(g), workspace.data_ptr(), workspace.numel(), _stream(dev))
    if rc != INKLING_OK:
        raise InklingError(rc, "inkling_moe_backward")
    return grads


# ---- products grouped by expert -------------------------------------------------


def _check(rc: int, where: str) -> None:
    if rc != INKLING_OK:
        raise InklingError(rc, where)


def _operand(t: Optional[torch.Tensor], name: str, dtype, dev) -> None:
    """A contiguous tensor of this dtype on dev, a GPU, or None."""
    if t is None or (t.dtype is dtype and t.get_device() == dev.index and t.is_contiguous()):
        return   # (the CPU's get_device() is -1 and its index None)
    _need(t, name, dtype)
    raise ValueError(f"{name} must be on {dev}, got {t.device}")


_device_count = functools.lru_cache(maxsize=None)(torch.cuda.device_count)


def _call(dev, name: str, *args) -> None:
    """The entry point `name` on dev's current stream, with dev the current device."""
    fn = getattr(_LIB or load(), name)
    if _device_count() == 1 or torch.cuda.current_device() == dev.index:
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    if rc != INKLING_OK:
        raise InklingError(rc, name)


def make_grouped_dims(rows, x_rows, n_groups, in_features, out_features, dtype, out_dtype=None) -> GroupedDims:
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    ocode = code if out_dtype is None else (out_dtype if isinstance(out_dtype, int) else _dtype_code(out_dtype))
    return GroupedDims(int(rows), int(x_rows), *_ints32(n_groups, in_features, out_features), code, ocode)


def grouped_workspace_size(dims: GroupedDims) -> int:
    """inkling_grouped_workspace_size (grouped_linear, grouped_input_grad)."""
    n = ctypes.c_size_t(0)
    _check(load().inkling_grouped_workspace_size(ctypes.byref(dims), ctypes.byref(n)),
           "inkling_grouped_workspace_size")
    return int(n.value)


def grouped_weight_grad_workspace_size(dims: GroupedDims) -> int:
    """inkling_grouped_weight_grad_workspace_size."""
    n = ctypes.c_size_t(0)
    _check(load().inkling_grouped_weight_grad_workspace_size(ctypes.byref(dims), ctypes.byref(n)),
           "inkling_grouped_weight_grad_workspace_size")
    return int(n.value)


# C structs and sizes by the sizes of a call: (pointer to the dims, bytes)
@functools.lru_cache(maxsize=1024)
def _grouped_plan(*sizes):
    dims = make_grouped_dims(*sizes)
    return ctypes.byref(dims), grouped_workspace_size(dims)


@functools.lru_cache(maxsize=1024)
def _grouped_weight_grad_plan(*sizes):
    dims = make_grouped_dims(*sizes)
    return ctypes.byref(dims), grouped_weight_grad_workspace_size(dims)


def _grouped_checks(rows_name, src, weight, offsets, axis, row_index):
    """Checks shared by the row products, whose rows are as wide as weight's
    `axis`; returns (rows, E, N, K)."""
    if src.dim() != 2 or weight.dim() != 3:
        raise ValueError(f"{rows_name} must be [rows, features] and weight [n_groups, out_features, in_features]")
    dev = src.device
    _operand(src, rows_name, weight.dtype, dev)
    _operand(weight, "weight", weight.dtype, dev)
    E, N, K = weight.shape
    R, have = src.shape
    if have != weight.shape[axis]:
        raise ValueError(f"{rows_name} must have {weight.shape[axis]} columns, got {have}")
    _grouped_plan_checks(offsets, E, row_index, dev)
    return (R if row_index is None else row_index.shape[0]), E, N, K


def _grouped_plan_checks(offsets, n_groups, row_index, dev):
    _operand(offsets, "offsets", torch.int32, dev)
    if offsets.dim() != 1 or offsets.shape[0] != n_groups + 1:
        raise ValueError("offsets must hold n_groups + 1 values")
    if row_index is not None:
        _operand(row_index, "row_index", torch.int32, dev)
        if row_index.dim() != 1:
            raise ValueError("row_index must be one-dimensional")


def _result_dtype(name, t, wanted, otherwise):
    """The dtype of the given result t, else the wanted one, else `otherwise`."""
    if t is None:
        return otherwise if wanted is None else wanted
    if wanted is not None and wanted != t.dtype:
        raise ValueError(f"the dtype wanted for {name} is {wanted}, and the given {name} has {t.dtype}")
    return t.dtype


def _result(t, name, shape, dtype, dev, like=None):
    """The given result tensor, checked, or a new one (`like`: a contiguous
    operand of that shape and dtype, from which making one is cheaper)."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like)
    _operand(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _scratch(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _operand(workspace, "workspace", torch.uint8, dev)
    return workspace


def grouped_linear(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                   row_index: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """inkling_grouped_linear: out[r] = weight[e] x[row_index[r]] for the rows
    offsets[e] <= r < offsets[e + 1].  x [rows, K] (with row_index [rows] int32:
    any number of rows), weight [E, N, K], offsets [E + 1] int32 on the device;
    out [rows, N].  Rows outside the groups are left as they are (in an `out`
    made here: unset)."""
    R, E, N, K = _grouped_checks("x", x, weight, offsets, 2, row_index)
    dev = x.device
    out_dtype = _result_dtype("out", out, out_dtype, x.dtype)
    dims, need = _grouped_plan(R, x.shape[0], E, K, N, x.dtype, out_dtype)
    out = _result(out, "out", (R, N), out_dtype, dev)
    ws = _scratch(workspace, need, dev)
    _call(dev, "inkling_grouped_linear", dims, x.data_ptr(), _ptr(row_index), weight.data_ptr(),
          offsets.data_ptr(), out.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return out


def grouped_input_grad(dout: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                       dx: Optional[torch.Tensor] = None, dx_dtype: Optional[torch.dtype] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """inkling_grouped_input_grad: dx[r] = weight[e]^T dout[r], [rows, K]; with a
    row_index in the forward, the rows of one x row are for the caller to sum."""
    R, E, N, K = _grouped_checks("dout", dout, weight, offsets, 1, None)
    dev = dout.device
    dx_dtype = _result_dtype("dx", dx, dx_dtype, dout.dtype)
    dims, need = _grouped_plan(R, R, E, K, N, dout.dtype, dx_dtype)
    dx = _result(dx, "dx", (R, K), dx_dtype, dev)
    ws = _scratch(workspace, need, dev)
    _call(dev, "inkling_grouped_input_grad", dims, dout.data_ptr(), weight.data_ptr(),
          offsets.data_ptr(), dx.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return dx


def grouped_weight_grad(dout: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                        row_index: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                        weight_grad_dtype: Optional[torch.dtype] = None,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """inkling_grouped_weight_grad: dweight[e] = sum over the rows of e of
    dout[r] (x) x[row_index[r]], [E, N, K]: fp32 (default) or bf16
    (`weight_grad_dtype`, or the dtype of the given `dweight`)."""
    if dout.dim() != 2 or x.dim() != 2:
        raise ValueError("dout and x must be [rows, features]")
    dev = dout.device
    _operand(dout, "dout", x.dtype, dev)
    _operand(x, "x", x.dtype, dev)
    E = offsets.shape[0] - 1 if offsets.dim() == 1 else 0
    _grouped_plan_checks(offsets, E, row_index, dev)
    R, N = dout.shape
    K = x.shape[1]
    if (x if row_index is None else row_index).shape[0] != R:
        raise ValueError("dout must have a row for each row of x, or for each entry of row_index")
    wdt = _result_dtype("dweight", dweight, weight_grad_dtype, torch.float32)
    dims, need = _grouped_weight_grad_plan(R, x.shape[0], E, K, N, x.dtype, wdt)
    dweight = _result(dweight, "dweight", (E, N, K), wdt, dev)
    ws = _scratch(workspace, need, dev)
    _call(dev, "inkling_grouped_weight_grad", dims, dout.data_ptr(), x.data_ptr(), _ptr(row_index),
          offsets.data_ptr(), dweight.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return dweight


# ---- SwiGLU with an 8-bit checkpoint ------------------------------------------------


def make_swiglu_dims(rows, intermediate, dtype) -> SwigluDims:
    return SwigluDims(int(rows), *_ints32(intermediate), dtype if isinstance(dtype, int) else _dtype_code(dtype))


def swiglu_checkpoint_size(dims: SwigluDims) -> int:
    """inkling_swiglu_checkpoint_size: bytes of the 8-bit checkpoint."""
    n = ctypes.c_size_t(0)
    _check(load().inkling_swiglu_checkpoint_size(ctypes.byref(dims), ctypes.byref(n)),
           "inkling_swiglu_checkpoint_size")
    return int(n.value)


@functools.lru_cache(maxsize=1024)
def _swiglu_plan(*sizes):
    dims = make_swiglu_dims(*sizes)
    return ctypes.byref(dims), swiglu_checkpoint_size(dims)


def _row_checks(dev, rows, gamma, row_count):
    if gamma is not None:
        _operand(gamma, "gamma", torch.float32, dev)
        if gamma.numel() != rows:
            raise ValueError(f"gamma must hold {rows} values")
    if row_count is not None:
        _operand(row_count, "row_count", torch.int32, dev)
        if row_count.numel() != 1:
            raise ValueError("row_count must hold one value")


def swiglu_forward(h: torch.Tensor, gamma: Optional[torch.Tensor] = None, row_count: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, checkpoint: Optional[torch.Tensor] = None,
                   save: bool = True):
    """inkling_swiglu_forward: (act [rows, I], checkpoint) of h [rows, 2I]
    (interleaved [gate, up] columns), act = gamma silu(gate) up.  The checkpoint
    is a uint8 tensor of swiglu_checkpoint_size bytes (made here unless given);
    save=False keeps none and returns None in its place.  Rows from
    row_count[0] on are left as they are."""
    if h.dim() != 2 or h.shape[1] % 2:
        raise ValueError("h must be [rows, 2 * intermediate]")
    dev = h.device
    _operand(h, "h", h.dtype, dev)
    R, I = h.shape
    I //= 2
    _row_checks(dev, R, gamma, row_count)
    dims, need = _swiglu_plan(R, I, h.dtype)
    out = _result(out, "out", (R, I), h.dtype, dev)
    if not save and checkpoint is not None:
        raise ValueError("save=False keeps no checkpoint: give none")
    if save:
        if checkpoint is None:
            checkpoint = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _operand(checkpoint, "checkpoint", torch.uint8, dev)
    _call(dev, "inkling_swiglu_forward", dims, h.data_ptr(), _ptr(gamma), _ptr(row_count),
          out.data_ptr(), _ptr(checkpoint), 0 if checkpoint is None else checkpoint.numel())
    return out, checkpoint


def swiglu_backward(dact: torch.Tensor, checkpoint: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                    row_count: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None,
                    act: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                    want_act: bool = True, want_dgamma: bool = True) -> dict:
    """inkling_swiglu_backward: dict(dh [rows, 2I], act [rows, I], dgamma
    [rows] fp32) from dact and the checkpoint that swiglu_forward filled with
    the same gamma and row_count; act (for the down projection's weight
    gradient) and dgamma are None where they are not wanted."""
    if dact.dim() != 2:
        raise ValueError("dact must be [rows, intermediate]")
    R, I = dact.shape
    dev = dact.device
    _operand(dact, "dact", dact.dtype, dev)
    _operand(checkpoint, "checkpoint", torch.uint8, dev)
    _row_checks(dev, R, gamma, row_count)
    if (act is not None and not want_act) or (dgamma is not None and not want_dgamma):
        raise ValueError("a result is both given and not wanted")
    dims, _ = _swiglu_plan(R, I, dact.dtype)
    dh = _result(dh, "dh", (R, 2 * I), dact.dtype, dev)
    act = _result(act, "act", (R, I), dact.dtype, dev, like=dact) if want_act else None
    dgamma = _result(dgamma, "dgamma", (R,), torch.float32, dev) if want_dgamma else None
    _call(dev, "inkling_swiglu_backward", dims, dact.data_ptr(), checkpoint.data_ptr(),
          checkpoint.numel(), _ptr(gamma), _ptr(row_count), dh.data_ptr(), _ptr(act), _ptr(dgamma))
    return {"dh": dh, "act": act, "dgamma": dgamma}


# ---- layer norm and RMS norm --------------------------------------------------------


def make_norm_dims(rows, hidden, kind, dtype, eps) -> NormDims:
    if isinstance(kind, str):
        if kind not in NORM_KINDS:
            raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}")
        kind = NORM_KINDS[kind]
    return NormDims(int(rows), *_ints32(hidden), kind, dtype if isinstance(dtype, int) else _dtype_code(dtype),
                    float(eps))


def norm_backward_workspace_size(dims: NormDims) -> int:
    """inkling_norm_backward_workspace_size."""
    n = ctypes.c_size_t(0)
    _check(load().inkling_norm_backward_workspace_size(ctypes.byref(dims), ctypes.byref(n)),
           "inkling_norm_backward_workspace_size")
    return int(n.value)


@functools.lru_cache(maxsize=1024)
def _norm_plan(*sizes):
    dims = make_norm_dims(*sizes)
    return ctypes.byref(dims), norm_backward_workspace_size(dims)


def _norm_checks(x, weight, bias):
    if x.dim() != 2:
        raise ValueError("x must be [rows, hidden]")
    dev, H = x.device, x.shape[1]
    _operand(x, "x", x.dtype, dev)
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _operand(t, n, torch.float32, dev)
            if t.dim() != 1 or t.shape[0] != H:
                raise ValueError(f"{n} must have shape ({H},)")


def norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 kind: str = "layer", out: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                 save: bool = True):
    """inkling_norm_forward: (out, stats) of x [rows, hidden]; kind "layer" or
    "rms" (no mean, no bias).  stats [rows, 2] fp32 (mean, 1 / sqrt(variance +
    eps)) is what norm_backward takes; save=False keeps none (None)."""
    _norm_checks(x, weight, bias)
    R, H = x.shape
    dev = x.device
    dims, _ = _norm_plan(R, H, kind, x.dtype, float(eps))
    out = _result(out, "out", (R, H), x.dtype, dev, like=x)
    if not save and stats is not None:
        raise ValueError("save=False keeps no stats: give none")
    stats = _result(stats, "stats", (R, 2), torch.float32, dev) if save else None
    _call(dev, "inkling_norm_forward", dims, x.data_ptr(), weight.data_ptr(), _ptr(bias),
          out.data_ptr(), _ptr(stats))
    return out, stats


def norm_backward(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, stats: torch.Tensor,
                  kind: str = "layer", bias: bool = False, dx: Optional[torch.Tensor] = None,
                  dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """inkling_norm_backward: dict(dx, dweight, dbias) from dout, the forward's
    x and weight and its stats; dbias is None unless `bias` (or a `dbias`) is
    given."""
    _norm_checks(x, weight, None)
    R, H = x.shape
    dev = x.device
    _operand(dout, "dout", x.dtype, dev)
    _operand(stats, "stats", torch.float32, dev)
    if dout.shape != x.shape or stats.shape != (R, 2):
        raise ValueError("dout must have x's shape and stats be [rows, 2]")
    dims, need = _norm_plan(R, H, kind, x.dtype, 0.0)
    ws = _scratch(workspace, need, dev)
    dx = _result(dx, "dx", (R, H), x.dtype, dev, like=x)
    dweight = _result(dweight, "dweight", (H,), torch.float32, dev, like=weight)
    dbias = _result(dbias, "dbias", (H,), torch.float32, dev, like=weight) if bias or dbias is not None else None
    _call(dev, "inkling_norm_backward", dims, dout.data_ptr(), x.data_ptr(), weight.data_ptr(),
          stats.data_ptr(), dx.data_ptr(), dweight.data_ptr(), _ptr(dbias), _ptr(ws), 0 if ws is None else ws.numel())
    return {"dx": dx, "dweight": dweight, "dbias": dbias}
