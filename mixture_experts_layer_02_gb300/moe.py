"""Thin Python binding of libmoe.so (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
fallback: if libmoe.so is missing or cannot load, every call raises.

Functions carry the C names (``moe_route``, ``moe_permute``,
``moe_grouped_ffn``, ``moe_combine``, ``moe_layer_forward``) and take torch
tensors that already live on the current CUDA device.  Outputs not passed in
are allocated here with torch.  ``ws`` is a workspace tensor from
:func:`workspace`; pass the same one again to avoid re-allocating, and to be
able to ask :func:`read_device_error` whether a kernel gave up: a call without
one makes its own and drops it, the device's error word included.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_BOUNDS = 5
MOE_ERR_DEVICE_TIMEOUT = 6

SOFTMAX_TOPK = 0
SIGMOID_NORM = 1
ACT_SILU = 0
ACT_SWIGLU = 1

FN_NONE = 0
FN_RELU = 1
FN_SILU = 2
FN_GELU = 3
FN_GELU_TANH = 4

EXPORTED = (
    "moe_workspace_size", "moe_route", "moe_permute", "moe_route_permute", "moe_grouped_ffn", "moe_combine",
    "moe_layer_forward", "moe_layer_workspace_layout", "moe_read_device_error",
    "moe_clear_device_error", "moe_set_debug_flags", "moe_status_string",
    "moe_last_error_detail", "moe_version", "moe_permute_static_scratch", "moe_routing_stats",
    "moe_capacity", "moe_workspace_size_padded", "moe_permute_padded", "moe_combine_padded",
    "moe_layer_forward_padded", "moe_layer_padded_workspace_layout", "moe_layer_launches",
    "moe_quantize_e4m3", "moe_permute_e4m3", "moe_grouped_ffn_e4m3", "moe_layer_forward_e4m3",
    "moe_layer_e4m3_workspace_layout", "moe_layer_launches_e4m3", "moe_permute_indices",
    "moe_grouped_ffn_gathered", "moe_grouped_ffn_e4m3_gathered",
    "moe_rmsnorm", "moe_rmsnorm_backward", "moe_gated_linear", "moe_gated_linear_backward",
    "moe_linear", "moe_linear_backward",
    "moe_combine_backward", "moe_permute_backward", "moe_route_backward", "moe_quantize_e4m3_block", "moe_segment_rows",
    "moe_quantize_e4m3_segments", "moe_grouped_linear_e4m3_block", "moe_grouped_linear_e4m3_block_backward",
)

_lock = threading.Lock()
_lib = None


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)}): {detail}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so and declare every exported signature."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libmoe.so not found at {path}: build it with "
                               "`python -m mixture_experts_layer_02_gb300.build`")
        L = ctypes.CDLL(path)
        p, i, sz, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint32
        L.moe_workspace_size.restype = sz
        L.moe_workspace_size.argtypes = [ctypes.c_char_p, i, i, i, i, i]
        L.moe_route.restype = i
        L.moe_route.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, sz, p]
        L.moe_permute.restype = i
        L.moe_permute.argtypes = [p, p, i, i, i, i, p, p, p, p, p, sz, p]
        L.moe_route_permute.restype = i
        L.moe_route_permute.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, p, p, p, sz, p]
        L.moe_permute_static_scratch.restype = i
        L.moe_permute_static_scratch.argtypes = [p, p, i, i, i, i, p, p, p, p, p]
        L.moe_grouped_ffn.restype = i
        L.moe_grouped_ffn.argtypes = [p, p, i, p, p, p, i, i, i, i, p, p, p, sz, p]
        L.moe_combine.restype = i
        L.moe_combine.argtypes = [p, p, p, i, i, i, p, p, sz, p]
        L.moe_layer_forward.restype = i
        L.moe_layer_forward.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, i, p, p, sz, p]
        L.moe_layer_launches.restype = i
        L.moe_layer_launches.argtypes = [i, i, i, i, i, i, i]
        L.moe_capacity.restype = i
        L.moe_capacity.argtypes = [i, i, i, ctypes.c_float]
        L.moe_workspace_size_padded.restype = sz
        L.moe_workspace_size_padded.argtypes = [ctypes.c_char_p, i, i, i, i, i, i]
        L.moe_permute_padded.restype = i
        L.moe_permute_padded.argtypes = [p, p, i, i, i, i, i, p, p, p, p, p, sz, p]
        L.moe_combine_padded.restype = i
        L.moe_combine_padded.argtypes = [p, p, p, i, i, i, i, i, p, p, sz, p]
        L.moe_layer_forward_padded.restype = i
        L.moe_layer_forward_padded.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, i, i, p, p, sz, p]
        L.moe_layer_padded_workspace_layout.restype = i
        L.moe_layer_padded_workspace_layout.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_routing_stats.restype = i
        L.moe_routing_stats.argtypes = [p, i, ctypes.c_float, ctypes.c_float, p, p, p, p]
        L.moe_layer_workspace_layout.restype = i
        L.moe_layer_workspace_layout.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_quantize_e4m3.restype = i
        L.moe_quantize_e4m3.argtypes = [p, ctypes.c_longlong, i, p, p, p]
        L.moe_permute_e4m3.restype = i
        L.moe_permute_e4m3.argtypes = [p, p, i, i, i, i, p, p, p, p, p, sz, p]
        L.moe_grouped_ffn_e4m3.restype = i
        L.moe_grouped_ffn_e4m3.argtypes = [p, p, p, p, i, p, p, p, p, p, p, i, i, i, i, p, p, p, p, p, sz, p]
        L.moe_layer_forward_e4m3.restype = i
        L.moe_layer_forward_e4m3.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, i, i, p, p, sz, p]
        L.moe_layer_e4m3_workspace_layout.restype = i
        L.moe_layer_e4m3_workspace_layout.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_layer_launches_e4m3.restype = i
        L.moe_layer_launches_e4m3.argtypes = [i, i, i, i, i, i]
        L.moe_permute_indices.restype = i
        L.moe_permute_indices.argtypes = [p, i, i, i, p, p, p, p, sz, p]
        L.moe_grouped_ffn_gathered.restype = i
        L.moe_grouped_ffn_gathered.argtypes = [p, i, p, p, i, p, p, p, i, i, i, i, p, p, p, sz, p]
        L.moe_grouped_ffn_e4m3_gathered.restype = i
        L.moe_grouped_ffn_e4m3_gathered.argtypes = [p, p, i, p, p, i, p, p, p, p, p, p, i, i, i, i,
                                                    p, p, p, p, p, sz, p]
        f = ctypes.c_float
        L.moe_rmsnorm.restype = i
        L.moe_rmsnorm.argtypes = [p, p, p, i, i, f, p, p, p, p, p]
        L.moe_rmsnorm_backward.restype = i
        L.moe_rmsnorm_backward.argtypes = [p, p, p, p, i, i, f, p, p, p, sz, p]
        L.moe_gated_linear.restype = i
        L.moe_gated_linear.argtypes = [p, p, p, i, i, i, i, p, p, p, p, sz, p]
        L.moe_gated_linear_backward.restype = i
        L.moe_gated_linear_backward.argtypes = [p, p, p, p, p, p, i, i, i, i, p, p, p, p, sz, p]
        L.moe_linear.restype = i
        L.moe_linear.argtypes = [p, p, p, p, i, i, i, i, p, p, p, sz, p]
        L.moe_linear_backward.restype = i
        L.moe_linear_backward.argtypes = [p, p, p, p, i, i, i, i, p, p, p, p, sz, p]
        L.moe_combine_backward.restype = i
        L.moe_combine_backward.argtypes = [p, p, p, p, i, i, i, i, p, p, p, sz, p]
        L.moe_permute_backward.restype = i
        L.moe_permute_backward.argtypes = [p, p, p, i, i, i, i, p, p, sz, p]
        L.moe_route_backward.restype = i
        L.moe_route_backward.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, p, p, p, p, sz, p]
        L.moe_quantize_e4m3_block.restype = i
        L.moe_quantize_e4m3_block.argtypes = [p, i, i, i, i, p, p, p]
        L.moe_segment_rows.restype = ctypes.c_longlong
        L.moe_segment_rows.argtypes = [i, i]
        L.moe_quantize_e4m3_segments.restype = i
        L.moe_quantize_e4m3_segments.argtypes = [p, p, i, i, i, p, p, p, p, p, sz, p]
        L.moe_grouped_linear_e4m3_block.restype = i
        L.moe_grouped_linear_e4m3_block.argtypes = [p, p, p, i, p, i, p, p, i, i, i, p, p, sz, p]
        L.moe_grouped_linear_e4m3_block_backward.restype = i
        L.moe_grouped_linear_e4m3_block_backward.argtypes = [p, p, p, p, p, p, p, i, p, p, i, i, i, p, p, p, sz, p]
        L.moe_read_device_error.restype = i
        L.moe_read_device_error.argtypes = [p, p]
        L.moe_clear_device_error.restype = i
        L.moe_clear_device_error.argtypes = [p, p]
        L.moe_set_debug_flags.restype = i
        L.moe_set_debug_flags.argtypes = [p, u32, p]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i]
        L.moe_last_error_detail.restype = ctypes.c_char_p
        L.moe_last_error_detail.argtypes = []
        L.moe_version.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        _lib = L
        return L


def status_string(s: int) -> str:
    return load().moe_status_string(s).decode()


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status, load().moe_last_error_detail().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: must be a contiguous CUDA tensor")


# ---------------------------------------------------------------- workspace
def workspace_size(op: str, N=0, D=0, E=0, K=0, Dff=0) -> int:
    return int(load().moe_workspace_size(op.encode(), N, D, E, K, Dff))


def workspace(op: str, N=0, D=0, E=0, K=0, Dff=0, device=None) -> torch.Tensor:
    """A zero-initialised workspace tensor (uint8) for ``op``."""
    n = workspace_size(op, N, D, E, K, Dff)
    if n == 0:
        raise ValueError(f"invalid workspace request {op} N={N} D={D} E={E} K={K} Dff={Dff}")
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def layer_launches(N, D, E, K, Dff, act, cap=-1) -> int:
    """Kernels one layer call launches (cap >= 0: the padded paradigm)."""
    return int(load().moe_layer_launches(N, D, E, K, Dff, act, cap))


def layer_workspace_layout(N, D, E, K, Dff) -> list:
    arr = (ctypes.c_size_t * 8)()
    if load().moe_layer_workspace_layout(N, D, E, K, Dff, arr) != 0:
        raise ValueError("invalid sizes")
    return list(arr)


def read_device_error(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the workspace's device status."""
    return int(load().moe_read_device_error(_ptr(ws), _stream(stream)))


def clear_device_error(ws: torch.Tensor, stream=None):
    _check("moe_clear_device_error", load().moe_clear_device_error(_ptr(ws), _stream(stream)))


def set_debug_flags(ws: torch.Tensor, flags: int, stream=None):
    _check("moe_set_debug_flags", load().moe_set_debug_flags(_ptr(ws), flags, _stream(stream)))


# ---------------------------------------------------------------- entry points
def moe_route(x, w_gate, bias, K: int, mode: int, topk_ids=None, topk_w=None,
              logits_out=None, ws=None, stream=None):
    N, D = x.shape
    E = w_gate.shape[0]
    _need(x, torch.bfloat16, (N, D), "x")
    _need(w_gate, torch.bfloat16, (E, D), "w_gate")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    dev = x.device
    topk_ids = torch.empty((N, K), dtype=torch.int32, device=dev) if topk_ids is None else topk_ids
    topk_w = torch.empty((N, K), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    _need(topk_w, torch.float32, (N, K), "topk_w")
    if logits_out is not None:
        _need(logits_out, torch.float32, (N, E), "logits_out")
    ws = workspace("route", N, D, E, K, device=dev) if ws is None else ws
    _check("moe_route", load().moe_route(
        _ptr(x), _ptr(w_gate), _ptr(bias), N, D, E, K, mode, _ptr(topk_ids), _ptr(topk_w),
        _ptr(logits_out), _ptr(ws), ws.numel(), _stream(stream)))
    return topk_ids, topk_w


def moe_permute(x, topk_ids, E: int, expert_offsets=None, perm_src=None, inv_perm=None,
                x_perm=None, ws=None, stream=None):
    N, D = x.shape
    K = topk_ids.shape[1]
    _need(x, torch.bfloat16, (N, D), "x")
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    dev = x.device
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    perm_src = torch.empty(N * K, dtype=torch.int32, device=dev) if perm_src is None else perm_src
    inv_perm = torch.empty((N, K), dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    x_perm = torch.empty((N * K, D), dtype=torch.bfloat16, device=dev) if x_perm is None else x_perm
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(perm_src, torch.int32, (N * K,), "perm_src")
    _need(inv_perm, torch.int32, (N, K), "inv_perm")
    _need(x_perm, torch.bfloat16, (N * K, D), "x_perm")
    ws = workspace("permute", N=N, E=E, device=dev) if ws is None else ws
    _check("moe_permute", load().moe_permute(
        _ptr(x), _ptr(topk_ids), N, D, E, K, _ptr(expert_offsets), _ptr(perm_src),
        _ptr(inv_perm), _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return expert_offsets, perm_src, inv_perm, x_perm


def moe_route_permute(x, w_gate, bias, K: int, mode: int, topk_ids=None, topk_w=None, expert_offsets=None,
                      perm_src=None, inv_perm=None, x_perm=None, ws=None, stream=None):
    """moe_route then moe_permute as one call; decode-sized calls (up to 8
    tokens, N*K <= 256) select and permute in one launch.  Returns (topk_ids, topk_w,
    expert_offsets, perm_src, inv_perm, x_perm)."""
    N, D = x.shape
    E = w_gate.shape[0]
    _need(x, torch.bfloat16, (N, D), "x")
    _need(w_gate, torch.bfloat16, (E, D), "w_gate")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    dev = x.device
    topk_ids = torch.empty((N, K), dtype=torch.int32, device=dev) if topk_ids is None else topk_ids
    topk_w = torch.empty((N, K), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    perm_src = torch.empty(N * K, dtype=torch.int32, device=dev) if perm_src is None else perm_src
    inv_perm = torch.empty((N, K), dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    x_perm = torch.empty((N * K, D), dtype=torch.bfloat16, device=dev) if x_perm is None else x_perm
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    _need(topk_w, torch.float32, (N, K), "topk_w")
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(perm_src, torch.int32, (N * K,), "perm_src")
    _need(inv_perm, torch.int32, (N, K), "inv_perm")
    _need(x_perm, torch.bfloat16, (N * K, D), "x_perm")
    ws = workspace("route_permute", N, D, E, K, device=dev) if ws is None else ws
    _check("moe_route_permute", load().moe_route_permute(
        _ptr(x), _ptr(w_gate), _ptr(bias), N, D, E, K, mode, _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets),
        _ptr(perm_src), _ptr(inv_perm), _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return topk_ids, topk_w, expert_offsets, perm_src, inv_perm, x_perm


def moe_permute_static_scratch(x, topk_ids, E: int, expert_offsets=None, perm_src=None,
                               inv_perm=None, x_perm=None, stream=None):
    """moe_permute for callers that cannot allocate: the scratch is a fixed
    4 MiB array inside the library (see include/moe.h); no workspace."""
    N, D = x.shape
    K = topk_ids.shape[1]
    _need(x, torch.bfloat16, (N, D), "x")
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    dev = x.device
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    perm_src = torch.empty(N * K, dtype=torch.int32, device=dev) if perm_src is None else perm_src
    inv_perm = torch.empty((N, K), dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    x_perm = torch.empty((N * K, D), dtype=torch.bfloat16, device=dev) if x_perm is None else x_perm
    _check("moe_permute_static_scratch", load().moe_permute_static_scratch(
        _ptr(x), _ptr(topk_ids), N, D, E, K, _ptr(expert_offsets), _ptr(perm_src),
        _ptr(inv_perm), _ptr(x_perm), _stream(stream)))
    return expert_offsets, perm_src, inv_perm, x_perm


def moe_grouped_ffn(x_perm, expert_offsets, w1, w3, w2, act: int, h=None, y_perm=None,
                    ws=None, stream=None):
    rows, D = x_perm.shape
    E, Dff, _ = w1.shape
    _need(x_perm, torch.bfloat16, (rows, D), "x_perm")
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(w1, torch.bfloat16, (E, Dff, D), "w1")
    if act == ACT_SWIGLU:
        _need(w3, torch.bfloat16, (E, Dff, D), "w3")
    _need(w2, torch.bfloat16, (E, D, Dff), "w2")
    dev = x_perm.device
    h = torch.empty((rows, Dff), dtype=torch.bfloat16, device=dev) if h is None else h
    y_perm = torch.empty((rows, D), dtype=torch.bfloat16, device=dev) if y_perm is None else y_perm
    _need(h, torch.bfloat16, (rows, Dff), "h")
    _need(y_perm, torch.bfloat16, (rows, D), "y_perm")
    ws = workspace("ffn", rows, D, E, 1, Dff, device=dev) if ws is None else ws
    _check("moe_grouped_ffn", load().moe_grouped_ffn(
        _ptr(x_perm), _ptr(expert_offsets), rows, _ptr(w1),
        _ptr(w3) if act == ACT_SWIGLU else None, _ptr(w2), E, D, Dff, act, _ptr(h),
        _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return h, y_perm


def moe_permute_indices(topk_ids, E: int, expert_offsets=None, perm_src=None, inv_perm=None, ws=None,
                        stream=None):
    """The permutation's indices without the row copy (for the gathered FFN)."""
    N, K = topk_ids.shape
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    dev = topk_ids.device
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    perm_src = torch.empty(N * K, dtype=torch.int32, device=dev) if perm_src is None else perm_src
    inv_perm = torch.empty((N, K), dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    ws = workspace("permute", N=N, E=E, device=dev) if ws is None else ws
    _check("moe_permute_indices", load().moe_permute_indices(
        _ptr(topk_ids), N, E, K, _ptr(expert_offsets), _ptr(perm_src), _ptr(inv_perm), _ptr(ws), ws.numel(),
        _stream(stream)))
    return expert_offsets, perm_src, inv_perm


def moe_grouped_ffn_gathered(x, perm_src, expert_offsets, w1, w3, w2, act: int, h=None, y_perm=None,
                             ws=None, stream=None):
    """moe_grouped_ffn with GEMM1 reading token rows of x through perm_src."""
    N, D = x.shape
    rows = perm_src.shape[0]
    E, Dff, _ = w1.shape
    _need(x, torch.bfloat16, (N, D), "x")
    _need(perm_src, torch.int32, (rows,), "perm_src")
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    dev = x.device
    h = torch.empty((rows, Dff), dtype=torch.bfloat16, device=dev) if h is None else h
    y_perm = torch.empty((rows, D), dtype=torch.bfloat16, device=dev) if y_perm is None else y_perm
    ws = workspace("ffn", rows, D, E, 1, Dff, device=dev) if ws is None else ws
    _check("moe_grouped_ffn_gathered", load().moe_grouped_ffn_gathered(
        _ptr(x), N, _ptr(perm_src), _ptr(expert_offsets), rows, _ptr(w1),
        _ptr(w3) if act == ACT_SWIGLU else None, _ptr(w2), E, D, Dff, act, _ptr(h), _ptr(y_perm),
        _ptr(ws), ws.numel(), _stream(stream)))
    return h, y_perm


def moe_combine(y_perm, inv_perm, topk_w, out=None, ws=None, stream=None):
    N, K = inv_perm.shape
    D = y_perm.shape[1]
    _need(y_perm, torch.bfloat16, (N * K, D), "y_perm")
    _need(inv_perm, torch.int32, (N, K), "inv_perm")
    _need(topk_w, torch.float32, (N, K), "topk_w")
    dev = y_perm.device
    out = torch.empty((N, D), dtype=torch.bfloat16, device=dev) if out is None else out
    _need(out, torch.bfloat16, (N, D), "out")
    ws = workspace("combine", device=dev) if ws is None else ws
    _check("moe_combine", load().moe_combine(
        _ptr(y_perm), _ptr(inv_perm), _ptr(topk_w), N, D, K, _ptr(out), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def moe_layer_forward(x, w_gate, bias, w1, w3, w2, K: int, mode: int, act: int, out=None,
                      ws=None, stream=None):
    N, D = x.shape
    E, Dff, _ = w1.shape
    _need(x, torch.bfloat16, (N, D), "x")
    _need(w_gate, torch.bfloat16, (E, D), "w_gate")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    _need(w1, torch.bfloat16, (E, Dff, D), "w1")
    if act == ACT_SWIGLU:
        _need(w3, torch.bfloat16, (E, Dff, D), "w3")
    _need(w2, torch.bfloat16, (E, D, Dff), "w2")
    dev = x.device
    out = torch.empty((N, D), dtype=torch.bfloat16, device=dev) if out is None else out
    _need(out, torch.bfloat16, (N, D), "out")
    ws = workspace("layer", N, D, E, K, Dff, device=dev) if ws is None else ws
    _check("moe_layer_forward", load().moe_layer_forward(
        _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(w1), _ptr(w3) if act == ACT_SWIGLU else None,
        _ptr(w2), N, D, E, K, Dff, mode, act, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_routing_stats(expert_offsets, ema, bias=None, decay: float = 0.99, bias_step: float = 0.1,
                      kl_out=None, stream=None):
    """EMA of per-expert fractions, KL to uniform and the bias step (in place
    on ema / bias).  Returns kl_out (a 1-element fp32 tensor)."""
    E = expert_offsets.shape[0] - 1
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(ema, torch.float32, (E,), "ema")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    kl_out = torch.empty(1, dtype=torch.float32, device=ema.device) if kl_out is None else kl_out
    _check("moe_routing_stats", load().moe_routing_stats(
        _ptr(expert_offsets), E, decay, bias_step, _ptr(ema), _ptr(bias), _ptr(kl_out), _stream(stream)))
    return kl_out


def layer_intermediates(ws: torch.Tensor, N, D, E, K, Dff) -> dict:
    """Views of the intermediates moe_layer_forward left in its workspace."""
    o = layer_workspace_layout(N, D, E, K, Dff)
    A = N * K

    def view(off, n, dtype, shape):
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype).view(shape)

    return dict(topk_ids=view(o[0], A, torch.int32, (N, K)),
                topk_w=view(o[1], A, torch.float32, (N, K)),
                expert_offsets=view(o[2], E + 1, torch.int32, (E + 1,)),
                perm_src=view(o[3], A, torch.int32, (A,)),
                inv_perm=view(o[4], A, torch.int32, (N, K)),
                x_perm=view(o[5], A * D, torch.bfloat16, (A, D)),
                h=view(o[6], A * Dff, torch.bfloat16, (A, Dff)),
                y_perm=view(o[7], A * D, torch.bfloat16, (A, D)))


# ---------------------------------------------------------------- paradigm B (fixed capacity)
def capacity(N: int, E: int, K: int, capacity_factor: float = 1.5) -> int:
    c = int(load().moe_capacity(N, E, K, capacity_factor))
    if c < 0:
        raise ValueError("invalid capacity arguments")
    return c


def workspace_padded(op: str, N=0, D=0, E=0, K=0, Dff=0, cap=0, device=None) -> torch.Tensor:
    n = int(load().moe_workspace_size_padded(op.encode(), N, D, E, K, Dff, cap))
    if n == 0:
        raise ValueError(f"invalid padded workspace request {op}")
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def moe_permute_padded(x, topk_ids, E: int, cap: int, expert_offsets=None, kept=None, slot=None,
                       x_pad=None, ws=None, stream=None):
    N, D = x.shape
    K = topk_ids.shape[1]
    _need(x, torch.bfloat16, (N, D), "x")
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    dev = x.device
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    kept = torch.empty(E, dtype=torch.int32, device=dev) if kept is None else kept
    slot = torch.empty((N, K), dtype=torch.int32, device=dev) if slot is None else slot
    x_pad = torch.empty((E * cap, D), dtype=torch.bfloat16, device=dev) if x_pad is None else x_pad
    ws = workspace_padded("permute", N=N, E=E, cap=cap, device=dev) if ws is None else ws
    _check("moe_permute_padded", load().moe_permute_padded(
        _ptr(x), _ptr(topk_ids), N, D, E, K, cap, _ptr(expert_offsets), _ptr(kept), _ptr(slot),
        _ptr(x_pad) if x_pad.numel() else None, _ptr(ws), ws.numel(), _stream(stream)))
    return expert_offsets, kept, slot, x_pad


def moe_combine_padded(y_pad, slot, topk_w, E: int, cap: int, out=None, ws=None, stream=None):
    N, K = slot.shape
    D = y_pad.shape[1]
    _need(slot, torch.int32, (N, K), "slot")
    _need(topk_w, torch.float32, (N, K), "topk_w")
    out = torch.empty((N, D), dtype=torch.bfloat16, device=slot.device) if out is None else out
    ws = workspace("combine", device=slot.device) if ws is None else ws
    _check("moe_combine_padded", load().moe_combine_padded(
        _ptr(y_pad) if y_pad.numel() else None, _ptr(slot), _ptr(topk_w), N, D, K, E, cap, _ptr(out),
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_layer_forward_padded(x, w_gate, bias, w1, w3, w2, K: int, mode: int, act: int, cap: int,
                             out=None, ws=None, stream=None):
    N, D = x.shape
    E, Dff, _ = w1.shape
    _need(x, torch.bfloat16, (N, D), "x")
    dev = x.device
    out = torch.empty((N, D), dtype=torch.bfloat16, device=dev) if out is None else out
    ws = workspace_padded("layer", N, D, E, K, Dff, cap, device=dev) if ws is None else ws
    _check("moe_layer_forward_padded", load().moe_layer_forward_padded(
        _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(w1), _ptr(w3) if act == ACT_SWIGLU else None, _ptr(w2),
        N, D, E, K, Dff, mode, act, cap, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def layer_padded_intermediates(ws: torch.Tensor, N, D, E, K, Dff, cap) -> dict:
    arr = (ctypes.c_size_t * 8)()
    if load().moe_layer_padded_workspace_layout(N, D, E, K, Dff, cap, arr) != 0:
        raise ValueError("invalid sizes")
    o = list(arr)
    A, R = N * K, E * cap

    def view(off, n, dtype, shape):
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype).view(shape)

    return dict(topk_ids=view(o[0], A, torch.int32, (N, K)), topk_w=view(o[1], A, torch.float32, (N, K)),
                expert_offsets=view(o[2], E + 1, torch.int32, (E + 1,)), kept=view(o[3], E, torch.int32, (E,)),
                slot=view(o[4], A, torch.int32, (N, K)), x_pad=view(o[5], R * D, torch.bfloat16, (R, D)),
                h=view(o[6], R * Dff, torch.bfloat16, (R, Dff)), y_pad=view(o[7], R * D, torch.bfloat16, (R, D)))


# ---------------------------------------------------------------- FP8 (e4m3) experts
def moe_quantize_e4m3(src, q=None, scale=None, stream=None):
    """Per-row e4m3 quantisation of a bf16 tensor (last dim = row): returns
    (codes uint8 of src's shape, scale fp32 of src.shape[:-1])."""
    if src.dtype != torch.bfloat16 or not src.is_cuda or not src.is_contiguous():
        raise TypeError("src: expected a contiguous bf16 CUDA tensor")
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    q = torch.empty(src.shape, dtype=torch.uint8, device=src.device) if q is None else q
    scale = torch.empty(src.shape[:-1], dtype=torch.float32, device=src.device) if scale is None else scale
    _need(q, torch.uint8, src.shape, "q")
    _need(scale, torch.float32, src.shape[:-1], "scale")
    _check("moe_quantize_e4m3", load().moe_quantize_e4m3(
        _ptr(src), rows, cols, _ptr(q), _ptr(scale), _stream(stream)))
    return q, scale


def quantize_experts_e4m3(w1, w3, w2, stream=None) -> dict:
    """e4m3 codes and per-output-channel scales of the three expert tensors."""
    w1q, s1 = moe_quantize_e4m3(w1, stream=stream)
    w3q, s3 = moe_quantize_e4m3(w3, stream=stream) if w3 is not None else (None, None)
    w2q, s2 = moe_quantize_e4m3(w2, stream=stream)
    return dict(w1q=w1q, s1=s1, w3q=w3q, s3=s3, w2q=w2q, s2=s2)


def moe_permute_e4m3(xq, topk_ids, E: int, expert_offsets=None, perm_src=None, inv_perm=None,
                     xq_perm=None, ws=None, stream=None):
    N, D = xq.shape
    K = topk_ids.shape[1]
    _need(xq, torch.uint8, (N, D), "xq")
    _need(topk_ids, torch.int32, (N, K), "topk_ids")
    dev = xq.device
    expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if expert_offsets is None else expert_offsets
    perm_src = torch.empty(N * K, dtype=torch.int32, device=dev) if perm_src is None else perm_src
    inv_perm = torch.empty((N, K), dtype=torch.int32, device=dev) if inv_perm is None else inv_perm
    xq_perm = torch.empty((N * K, D), dtype=torch.uint8, device=dev) if xq_perm is None else xq_perm
    _need(xq_perm, torch.uint8, (N * K, D), "xq_perm")
    ws = workspace("permute", N=N, E=E, device=dev) if ws is None else ws
    _check("moe_permute_e4m3", load().moe_permute_e4m3(
        _ptr(xq), _ptr(topk_ids), N, D, E, K, _ptr(expert_offsets), _ptr(perm_src),
        _ptr(inv_perm), _ptr(xq_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return expert_offsets, perm_src, inv_perm, xq_perm


def moe_grouped_ffn_e4m3(xq_perm, x_scale, x_scale_index, expert_offsets, w1q, s1, w3q, s3, w2q, s2,
                         act: int, h=None, hq=None, h_scale=None, y_perm=None, ws=None, stream=None):
    rows, D = xq_perm.shape
    E, Dff, _ = w1q.shape
    _need(xq_perm, torch.uint8, (rows, D), "xq_perm")
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(w1q, torch.uint8, (E, Dff, D), "w1q")
    _need(s1, torch.float32, (E, Dff), "s1")
    if act == ACT_SWIGLU:
        _need(w3q, torch.uint8, (E, Dff, D), "w3q")
        _need(s3, torch.float32, (E, Dff), "s3")
    _need(w2q, torch.uint8, (E, D, Dff), "w2q")
    _need(s2, torch.float32, (E, D), "s2")
    dev = xq_perm.device
    h = torch.empty((rows, Dff), dtype=torch.bfloat16, device=dev) if h is None else h
    hq = torch.empty((rows, Dff), dtype=torch.uint8, device=dev) if hq is None else hq
    h_scale = torch.empty(rows, dtype=torch.float32, device=dev) if h_scale is None else h_scale
    y_perm = torch.empty((rows, D), dtype=torch.bfloat16, device=dev) if y_perm is None else y_perm
    _need(h, torch.bfloat16, (rows, Dff), "h")
    _need(hq, torch.uint8, (rows, Dff), "hq")
    _need(h_scale, torch.float32, (rows,), "h_scale")
    _need(y_perm, torch.bfloat16, (rows, D), "y_perm")
    ws = workspace("ffn", rows, D, E, 1, Dff, device=dev) if ws is None else ws
    sw = act == ACT_SWIGLU
    _check("moe_grouped_ffn_e4m3", load().moe_grouped_ffn_e4m3(
        _ptr(xq_perm), _ptr(x_scale), _ptr(x_scale_index), _ptr(expert_offsets), rows, _ptr(w1q), _ptr(s1),
        _ptr(w3q) if sw else None, _ptr(s3) if sw else None, _ptr(w2q), _ptr(s2), E, D, Dff, act,
        _ptr(h), _ptr(hq), _ptr(h_scale), _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return h, hq, h_scale, y_perm


def moe_layer_forward_e4m3(x, w_gate, bias, qw: dict, K: int, mode: int, act: int, out=None, ws=None,
                           stream=None):
    """The layer with e4m3 experts; ``qw`` as returned by quantize_experts_e4m3."""
    N, D = x.shape
    E, Dff, _ = qw["w1q"].shape
    _need(x, torch.bfloat16, (N, D), "x")
    _need(w_gate, torch.bfloat16, (E, D), "w_gate")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    dev = x.device
    out = torch.empty((N, D), dtype=torch.bfloat16, device=dev) if out is None else out
    _need(out, torch.bfloat16, (N, D), "out")
    ws = workspace("layer_e4m3", N, D, E, K, Dff, device=dev) if ws is None else ws
    sw = act == ACT_SWIGLU
    _check("moe_layer_forward_e4m3", load().moe_layer_forward_e4m3(
        _ptr(x), _ptr(w_gate), _ptr(bias), _ptr(qw["w1q"]), _ptr(qw["s1"]),
        _ptr(qw["w3q"]) if sw else None, _ptr(qw["s3"]) if sw else None, _ptr(qw["w2q"]), _ptr(qw["s2"]),
        N, D, E, K, Dff, mode, act, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def layer_launches_e4m3(N, D, E, K, Dff, act) -> int:
    return int(load().moe_layer_launches_e4m3(N, D, E, K, Dff, act))


def layer_e4m3_intermediates(ws: torch.Tensor, N, D, E, K, Dff) -> dict:
    """Views of the intermediates moe_layer_forward_e4m3 left in its workspace."""
    arr = (ctypes.c_size_t * 12)()
    if load().moe_layer_e4m3_workspace_layout(N, D, E, K, Dff, arr) != 0:
        raise ValueError("invalid sizes")
    o = list(arr)
    A = N * K

    def view(off, n, dtype, shape):
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + nbytes].view(dtype).view(shape)

    return dict(topk_ids=view(o[0], A, torch.int32, (N, K)), topk_w=view(o[1], A, torch.float32, (N, K)),
                expert_offsets=view(o[2], E + 1, torch.int32, (E + 1,)), perm_src=view(o[3], A, torch.int32, (A,)),
                inv_perm=view(o[4], A, torch.int32, (N, K)), xq=view(o[5], N * D, torch.uint8, (N, D)),
                x_scale=view(o[6], N, torch.float32, (N,)), xq_perm=view(o[7], A * D, torch.uint8, (A, D)),
                h=view(o[8], A * Dff, torch.bfloat16, (A, Dff)), hq=view(o[9], A * Dff, torch.uint8, (A, Dff)),
                h_scale=view(o[10], A, torch.float32, (A,)), y_perm=view(o[11], A * D, torch.bfloat16, (A, D)))


def moe_grouped_ffn_e4m3_gathered(xq, x_scale, perm_src, expert_offsets, w1q, s1, w3q, s3, w2q, s2, act: int,
                                  h=None, hq=None, h_scale=None, y_perm=None, ws=None, stream=None):
    """moe_grouped_ffn_e4m3 with GEMM1 reading token codes of xq through perm_src."""
    N, D = xq.shape
    rows = perm_src.shape[0]
    E, Dff, _ = w1q.shape
    _need(xq, torch.uint8, (N, D), "xq")
    _need(x_scale, torch.float32, (N,), "x_scale")
    _need(perm_src, torch.int32, (rows,), "perm_src")
    dev = xq.device
    h = torch.empty((rows, Dff), dtype=torch.bfloat16, device=dev) if h is None else h
    hq = torch.empty((rows, Dff), dtype=torch.uint8, device=dev) if hq is None else hq
    h_scale = torch.empty(rows, dtype=torch.float32, device=dev) if h_scale is None else h_scale
    y_perm = torch.empty((rows, D), dtype=torch.bfloat16, device=dev) if y_perm is None else y_perm
    ws = workspace("ffn", rows, D, E, 1, Dff, device=dev) if ws is None else ws
    sw = act == ACT_SWIGLU
    _check("moe_grouped_ffn_e4m3_gathered", load().moe_grouped_ffn_e4m3_gathered(
        _ptr(xq), _ptr(x_scale), N, _ptr(perm_src), _ptr(expert_offsets), rows, _ptr(w1q), _ptr(s1),
        _ptr(w3q) if sw else None, _ptr(s3) if sw else None, _ptr(w2q), _ptr(s2), E, D, Dff, act,
        _ptr(h), _ptr(hq), _ptr(h_scale), _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)))
    return h, hq, h_scale, y_perm


# ---------------------------------------------------------------- dense operators (norm, gated and linear products)
# Small calls run in a few microseconds on the GPU, so the host side counts:
# each function tests its arguments in one expression and goes through _explain
# only to say what is wrong, and the stream handle is read without a Stream
# object (3 us).
_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_of(t, stream):
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def _new(stream, *specs):
    """Empty tensors (shape, dtype, device), each None where the spec is None,
    that belong to the stream the call runs on: the allocator then does not hand
    a freed one to another stream too early."""
    if stream is None:
        return [None if s is None else torch.empty(s[0], dtype=s[1], device=s[2]) for s in specs]
    with torch.cuda.stream(stream):
        return _new(None, *specs)


def _scratch(stream, op, N, D, F, device):
    """A workspace of one call: only its header is zeroed.  Invalid sizes get a
    bare header: the entry point then says what is wrong with them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _scratch(None, op, N, D, F, device)
    ws = torch.empty(max(workspace_size(op, N=N, D=D, Dff=F), 256), dtype=_U8, device=device)
    ws[:256].zero_()
    return ws


def _fits(t, dtype, shape):
    return t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()


def _explain(ws, *specs):
    """Raise for the first (tensor or None, dtype, shape, name) that does not fit, or a workspace off the GPU."""
    for t, dtype, shape, name in specs:
        if t is not None:
            _need(t, dtype, shape, name)
    if ws is not None and not ws.is_cuda:
        raise ValueError("ws: must be a CUDA tensor")


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(t, name):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected [rows, width], got {tuple(shape)}")
    return shape


def moe_rmsnorm(x, weight, residual=None, eps: float = 1e-6, quantize: bool = False, y=None, yq=None, y_scale=None,
                residual_out=None, stream=None):
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * weight.  Returns
    (y, yq, y_scale, s): yq and y_scale (e4m3 codes as uint8 and one scale a
    row, as moe_permute_e4m3 takes them) with quantize=True or when passed, s
    (the new residual stream) when a residual is given or residual_out is
    passed; None for the others."""
    shape = _rows(x, "x")
    N, D = shape
    codes = quantize or yq is not None or y_scale is not None
    if y is None:
        y, = _new(stream, (shape, _BF16, x.device))
    if codes and (yq is None or y_scale is None):
        q, sc = _new(stream, (shape, _U8, x.device), ((N,), _F32, x.device))
        yq, y_scale = q if yq is None else yq, sc if y_scale is None else y_scale
    if residual is not None and residual_out is None:
        residual_out, = _new(stream, (shape, _BF16, x.device))
    if not (_fits(x, _BF16, shape) and _fits(weight, _BF16, (D,)) and _fits(y, _BF16, shape)
            and (residual is None or _fits(residual, _BF16, shape))
            and (residual_out is None or _fits(residual_out, _BF16, shape))
            and (not codes or (_fits(yq, _U8, shape) and _fits(y_scale, _F32, (N,))))):
        _explain(None, (x, _BF16, shape, "x"), (weight, _BF16, (D,), "weight"), (residual, _BF16, shape, "residual"),
                 (y, _BF16, shape, "y"), (yq, _U8, shape, "yq"), (y_scale, _F32, (N,), "y_scale"),
                 (residual_out, _BF16, shape, "residual_out"))
    s = (_lib or load()).moe_rmsnorm(_addr(x), _addr(residual), _addr(weight), N, D, eps, _addr(y), _addr(yq),
                                     _addr(y_scale), _addr(residual_out), _stream_of(x, stream))
    if s:
        _check("moe_rmsnorm", s)
    return y, yq, y_scale, residual_out


def moe_rmsnorm_backward(dy, s, weight, dresidual=None, eps: float = 1e-6, dx=None, dweight=None, ws=None, stream=None):
    """Gradient of moe_rmsnorm from dy and s (its fourth result, or x without a
    residual): (dx, dweight), dx for x and the residual alike, dweight fp32.
    dresidual is the gradient that reached s itself."""
    shape = _rows(s, "s")
    N, D = shape
    if dx is None:
        dx, = _new(stream, (shape, _BF16, s.device))
    if dweight is None:
        dweight, = _new(stream, ((D,), _F32, s.device))
    if ws is None:
        ws = _scratch(stream, "rmsnorm_backward", N, D, 0, s.device)
    if not (_fits(dy, _BF16, shape) and _fits(s, _BF16, shape) and _fits(weight, _BF16, (D,)) and _fits(dx, _BF16, shape)
            and _fits(dweight, _F32, (D,)) and ws.is_cuda and (dresidual is None or _fits(dresidual, _BF16, shape))):
        _explain(ws, (dy, _BF16, shape, "dy"), (s, _BF16, shape, "s"), (weight, _BF16, (D,), "weight"),
                 (dresidual, _BF16, shape, "dresidual"), (dx, _BF16, shape, "dx"), (dweight, _F32, (D,), "dweight"))
    st = (_lib or load()).moe_rmsnorm_backward(_addr(dy), _addr(s), _addr(weight), _addr(dresidual), N, D, eps, _addr(dx),
                                               _addr(dweight), _addr(ws), ws.numel(), _stream_of(s, stream))
    if st:
        _check("moe_rmsnorm_backward", st)
    return dx, dweight


def moe_gated_linear(x, w1, w3, fn: int = FN_SILU, save: bool = False, h=None, g=None, u=None, ws=None, stream=None):
    """h = fn(x w1^T) * (x w3^T) for weights [F, D].  Returns (h, g, u); g and u
    (the two projections, for the backward pass) are None unless save=True or
    they are passed."""
    N, D = _rows(x, "x")
    wide = _rows(w1, "w1")
    F = wide[0]
    if h is None:
        h, = _new(stream, ((N, F), _BF16, x.device))
    if save and (g is None or u is None):
        g2, u2 = _new(stream, ((N, F), _BF16, x.device), ((N, F), _BF16, x.device))
        g, u = g2 if g is None else g, u2 if u is None else u
    if ws is None:
        ws = _scratch(stream, "gated_linear", N, D, F, x.device)
    if not (_fits(x, _BF16, (N, D)) and _fits(w1, _BF16, (F, D)) and _fits(w3, _BF16, (F, D)) and _fits(h, _BF16, (N, F)) and ws.is_cuda
            and (g is None or _fits(g, _BF16, (N, F))) and (u is None or _fits(u, _BF16, (N, F)))):
        _explain(ws, (x, _BF16, (N, D), "x"), (w1, _BF16, (F, D), "w1"), (w3, _BF16, (F, D), "w3"), (h, _BF16, (N, F), "h"),
                 (g, _BF16, (N, F), "g"), (u, _BF16, (N, F), "u"))
    s = (_lib or load()).moe_gated_linear(_addr(x), _addr(w1), _addr(w3), N, D, F, fn, _addr(h), _addr(g), _addr(u),
                                          _addr(ws), ws.numel(), _stream_of(x, stream))
    if s:
        _check("moe_gated_linear", s)
    return h, g, u


def moe_gated_linear_backward(dh, x, w1, w3, g, u, fn: int = FN_SILU, dx=None, dw1=None, dw3=None, ws=None, stream=None):
    """Gradient of moe_gated_linear from dh and the g, u it kept: (dx, dw1, dw3)."""
    N, D = _rows(x, "x")
    F = _rows(w1, "w1")[0]
    dev = x.device
    if dx is None:
        dx, = _new(stream, ((N, D), _BF16, dev))
    if dw1 is None:
        dw1, = _new(stream, ((F, D), _BF16, dev))
    if dw3 is None:
        dw3, = _new(stream, ((F, D), _BF16, dev))
    if ws is None:
        ws = _scratch(stream, "gated_linear_backward", N, D, F, dev)
    _explain(ws, (dh, _BF16, (N, F), "dh"), (x, _BF16, (N, D), "x"), (w1, _BF16, (F, D), "w1"), (w3, _BF16, (F, D), "w3"),
             (g, _BF16, (N, F), "g"), (u, _BF16, (N, F), "u"), (dx, _BF16, (N, D), "dx"), (dw1, _BF16, (F, D), "dw1"),
             (dw3, _BF16, (F, D), "dw3"))
    s = (_lib or load()).moe_gated_linear_backward(_addr(dh), _addr(x), _addr(w1), _addr(w3), _addr(g), _addr(u), N, D, F,
                                                   fn, _addr(dx), _addr(dw1), _addr(dw3), _addr(ws), ws.numel(),
                                                   _stream_of(x, stream))
    if s:
        _check("moe_gated_linear_backward", s)
    return dx, dw1, dw3


def moe_linear(x, w, bias=None, residual=None, fn: int = FN_NONE, save: bool = False, y=None, z=None, ws=None,
               stream=None):
    """y = residual + fn(x w^T + bias) for a weight [F, D] and an fp32 bias [F].
    Returns (y, z); z (the pre-activation, for the backward pass) is None unless
    save=True or it is passed."""
    N, D = _rows(x, "x")
    F = _rows(w, "w")[0]
    if y is None:
        y, = _new(stream, ((N, F), _BF16, x.device))
    if save and z is None:
        z, = _new(stream, ((N, F), _BF16, x.device))
    if ws is None:
        ws = _scratch(stream, "linear", N, D, F, x.device)
    if not (_fits(x, _BF16, (N, D)) and _fits(w, _BF16, (F, D)) and _fits(y, _BF16, (N, F)) and ws.is_cuda
            and (bias is None or _fits(bias, _F32, (F,))) and (residual is None or _fits(residual, _BF16, (N, F)))
            and (z is None or _fits(z, _BF16, (N, F)))):
        _explain(ws, (x, _BF16, (N, D), "x"), (w, _BF16, (F, D), "w"), (bias, _F32, (F,), "bias"),
                 (residual, _BF16, (N, F), "residual"), (y, _BF16, (N, F), "y"), (z, _BF16, (N, F), "z"))
    s = (_lib or load()).moe_linear(_addr(x), _addr(w), _addr(bias), _addr(residual), N, D, F, fn, _addr(y), _addr(z),
                                    _addr(ws), ws.numel(), _stream_of(x, stream))
    if s:
        _check("moe_linear", s)
    return y, z


def moe_linear_backward(dy, x, w, z=None, fn: int = FN_NONE, need_dbias: bool = False, dx=None, dw=None, dbias=None,
                        ws=None, stream=None):
    """Gradient of moe_linear from dy and the z it kept (not needed for
    FN_NONE): (dx, dw, dbias); dbias is fp32, None unless need_dbias=True or it
    is passed.  The residual's gradient is dy."""
    N, D = _rows(x, "x")
    F = _rows(w, "w")[0]
    dev = x.device
    if dx is None:
        dx, = _new(stream, ((N, D), _BF16, dev))
    if dw is None:
        dw, = _new(stream, ((F, D), _BF16, dev))
    if need_dbias and dbias is None:
        dbias, = _new(stream, ((F,), _F32, dev))
    if ws is None:
        ws = _scratch(stream, "linear_backward", N, D, F, dev)
    _explain(ws, (dy, _BF16, (N, F), "dy"), (x, _BF16, (N, D), "x"), (w, _BF16, (F, D), "w"), (z, _BF16, (N, F), "z"),
             (dx, _BF16, (N, D), "dx"), (dw, _BF16, (F, D), "dw"), (dbias, _F32, (F,), "dbias"))
    s = (_lib or load()).moe_linear_backward(_addr(dy), _addr(x), _addr(w), _addr(z), N, D, F, fn, _addr(dx), _addr(dw),
                                             _addr(dbias), _addr(ws), ws.numel(), _stream_of(x, stream))
    if s:
        _check("moe_linear_backward", s)
    return dx, dw, dbias


# ---------------------------------------------------------------- training the routed layer
_I32 = torch.int32
BLOCK = 128  # values that share a scale, along each blocked dimension
_current_device = torch._C._cuda_getDevice


def _blocks(n):
    return -(-n // BLOCK)


def _ready(fn, ws, *specs):
    """Check (tensor or None, dtype, shape, name) of one call: contiguous CUDA tensors of one device, the current one."""
    dev = specs[0][0].get_device()
    for t, dtype, shape, name in specs:
        if t is not None and not (t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()):
            _need(t, dtype, shape, name)
            raise ValueError(f"{name}: on cuda:{t.get_device()}, {specs[0][3]} on cuda:{dev}")
    if dev < 0:
        _need(*specs[0])
    if ws is not None and not (ws.get_device() == dev and ws.dtype is _U8 and ws.is_contiguous()):
        raise ValueError(f"ws: must be a contiguous uint8 tensor on cuda:{dev}")
    if dev != _current_device():
        raise ValueError(f"{fn}: its tensors are on cuda:{dev}, not on the current device")


def _header(stream, op, device, **sizes):
    """A workspace of one call, only its header zeroed (see _scratch)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _header(None, op, device, **sizes)
    ws = torch.empty(max(workspace_size(op, **sizes), 256), dtype=_U8, device=device)
    ws[:256].zero_()
    return ws


def moe_combine_backward(dout, y_perm, inv_perm, topk_w, dy_perm=None, dtopk_w=None, ws=None, stream=None):
    """Gradient of moe_combine, or of moe_combine_padded with its slot as inv_perm: (dy_perm, dtopk_w).
    Rows of dy_perm that no assignment names are left as they were (zero in a buffer made here)."""
    shape = _rows(dout, "dout")
    N, D = shape
    K = _rows(inv_perm, "inv_perm")[1]
    rows = _rows(y_perm, "y_perm")[0]
    if dy_perm is None:
        dy_perm, = _new(stream, ((rows, D), _BF16, dout.device))
        with torch.cuda.stream(stream):  # as many rows as assignments may still hold empty slots
            dy_perm.zero_()
    if dtopk_w is None:
        dtopk_w, = _new(stream, ((N, K), _F32, dout.device))
    if ws is None:
        ws = _header(stream, "combine", dout.device)
    _ready("moe_combine_backward", ws, (dout, _BF16, shape, "dout"), (y_perm, _BF16, (rows, D), "y_perm"),
           (inv_perm, _I32, (N, K), "inv_perm"), (topk_w, _F32, (N, K), "topk_w"), (dy_perm, _BF16, (rows, D), "dy_perm"),
           (dtopk_w, _F32, (N, K), "dtopk_w"))
    s = (_lib or load()).moe_combine_backward(_addr(dout), _addr(y_perm), _addr(inv_perm), _addr(topk_w), N, D, K, rows,
                                              _addr(dy_perm), _addr(dtopk_w), _addr(ws), ws.numel(), _stream_of(dout, stream))
    if s:
        _check("moe_combine_backward", s)
    return dy_perm, dtopk_w


def moe_permute_backward(dx_perm, inv_perm, dresidual=None, dx=None, ws=None, stream=None):
    """Gradient of moe_permute (or, with its slot, of moe_permute_padded) for the tokens, added to dresidual: dx."""
    rows, D = _rows(dx_perm, "dx_perm")
    N, K = _rows(inv_perm, "inv_perm")
    if dx is None:
        dx, = _new(stream, ((N, D), _BF16, dx_perm.device))
    if ws is None:
        ws = _header(stream, "combine", dx_perm.device)
    _ready("moe_permute_backward", ws, (dx_perm, _BF16, (rows, D), "dx_perm"), (inv_perm, _I32, (N, K), "inv_perm"),
           (dresidual, _BF16, (N, D), "dresidual"), (dx, _BF16, (N, D), "dx"))
    s = (_lib or load()).moe_permute_backward(_addr(dx_perm), _addr(inv_perm), _addr(dresidual), N, D, K, rows, _addr(dx),
                                              _addr(ws), ws.numel(), _stream_of(dx_perm, stream))
    if s:
        _check("moe_permute_backward", s)
    return dx


def moe_route_backward(dtopk_w, topk_ids, topk_w, logits, x, w_gate, mode: int, dresidual=None, need_dbias: bool = False,
                       dx=None, dw_gate=None, dbias=None, ws=None, stream=None):
    """Gradient of moe_route through its weights: (dx, dw_gate, dbias).  logits is moe_route's logits_out (may be None
    for SOFTMAX_TOPK); dx is added to dresidual; dbias is fp32, None unless need_dbias=True or it is passed."""
    N, D = _rows(x, "x")
    E = _rows(w_gate, "w_gate")[0]
    K = _rows(topk_ids, "topk_ids")[1]
    if logits is None and mode == SIGMOID_NORM:
        raise ValueError("logits: needed with SIGMOID_NORM")
    if dx is None:
        dx, = _new(stream, ((N, D), _BF16, x.device))
    if dw_gate is None:
        dw_gate, = _new(stream, ((E, D), _BF16, x.device))
    if need_dbias and dbias is None:
        dbias, = _new(stream, ((E,), _F32, x.device))
    if ws is None:
        ws = _header(stream, "route_backward", x.device, N=N, D=D, E=E)
    _ready("moe_route_backward", ws, (x, _BF16, (N, D), "x"), (w_gate, _BF16, (E, D), "w_gate"),
           (dtopk_w, _F32, (N, K), "dtopk_w"), (topk_ids, _I32, (N, K), "topk_ids"), (topk_w, _F32, (N, K), "topk_w"),
           (logits, _F32, (N, E), "logits"), (dresidual, _BF16, (N, D), "dresidual"), (dx, _BF16, (N, D), "dx"),
           (dw_gate, _BF16, (E, D), "dw_gate"), (dbias, _F32, (E,), "dbias"))
    s = (_lib or load()).moe_route_backward(_addr(dtopk_w), _addr(topk_ids), _addr(topk_w), _addr(logits), _addr(x),
                                            _addr(w_gate), _addr(dresidual), N, D, E, K, mode, _addr(dx), _addr(dw_gate),
                                            _addr(dbias), _addr(ws), ws.numel(), _stream_of(x, stream))
    if s:
        _check("moe_route_backward", s)
    return dx, dw_gate, dbias


def moe_quantize_e4m3_block(src, block_rows: int = 1, q=None, scale=None, stream=None):
    """e4m3 codes of a bf16 tensor [rows, cols] or [mats, rows, cols] with a scale for each 1 x 128 (block_rows=1) or
    128 x 128 (block_rows=128) of each matrix: (q uint8 of src's shape, scale fp32)."""
    shape = src.shape
    if len(shape) == 2:
        (rows, cols), mats = shape, 1
        grid = (_blocks(rows) if block_rows == BLOCK else rows, _blocks(cols))
    elif len(shape) == 3:
        mats, rows, cols = shape
        grid = (mats, _blocks(rows) if block_rows == BLOCK else rows, _blocks(cols))
    else:
        raise ValueError(f"src: expected [rows, cols] or [mats, rows, cols], got {tuple(shape)}")
    if q is None:
        q, = _new(stream, (shape, _U8, src.device))
    if scale is None:
        scale, = _new(stream, (grid, _F32, src.device))
    _ready("moe_quantize_e4m3_block", None, (src, _BF16, shape, "src"), (q, _U8, shape, "q"), (scale, _F32, grid, "scale"))
    s = (_lib or load()).moe_quantize_e4m3_block(_addr(src), mats, rows, cols, block_rows, _addr(q), _addr(scale),
                                                 _stream_of(src, stream))
    if s:
        _check("moe_quantize_e4m3_block", s)
    return q, scale


def segment_rows(rows: int, E: int) -> int:
    """Rows of the buffers whose segments start at multiples of 128, whatever the routing."""
    n = int(load().moe_segment_rows(rows, E))
    if n < 0:
        raise ValueError(f"invalid sizes: rows={rows}, E={E}")
    return n


def moe_quantize_e4m3_segments(src, expert_offsets, both: bool = True, q=None, scale=None, q_seg=None, scale_seg=None,
                               ws=None, stream=None):
    """e4m3 codes of src [rows, cols] along each expert's rows, as the weight gradient reads them, and (with both=True,
    or where passed) along its columns: (q, scale, q_seg, scale_seg).  expert_offsets [E+1], or None for one segment.
    Rows behind the last segment are not written."""
    rows, cols = _rows(src, "src")
    E = 1 if expert_offsets is None else expert_offsets.shape[0] - 1
    seg = segment_rows(rows, E)
    dev = src.device
    if (both or scale is not None) and q is None:
        q, = _new(stream, ((rows, cols), _U8, dev))
    if q is not None and scale is None:
        scale, = _new(stream, ((rows, _blocks(cols)), _F32, dev))
    if q_seg is None:
        q_seg, = _new(stream, ((seg, cols), _U8, dev))
    if scale_seg is None:
        scale_seg, = _new(stream, ((seg // BLOCK, cols), _F32, dev))
    if ws is None:
        ws = _header(stream, "combine", dev)
    _ready("moe_quantize_e4m3_segments", ws, (src, _BF16, (rows, cols), "src"), (expert_offsets, _I32, (E + 1,), "expert_offsets"),
           (q, _U8, (rows, cols), "q"), (scale, _F32, (rows, _blocks(cols)), "scale"), (q_seg, _U8, (seg, cols), "q_seg"),
           (scale_seg, _F32, (seg // BLOCK, cols), "scale_seg"))
    s = (_lib or load()).moe_quantize_e4m3_segments(_addr(src), _addr(expert_offsets), rows, cols, E, _addr(q), _addr(scale),
                                                    _addr(q_seg), _addr(scale_seg), _addr(ws), ws.numel(),
                                                    _stream_of(src, stream))
    if s:
        _check("moe_quantize_e4m3_segments", s)
    return q, scale, q_seg, scale_seg


def _weights(wq):
    if wq.dim() != 3:
        raise ValueError(f"wq: expected [E, F, D], got {tuple(wq.shape)}")
    return wq.shape


def moe_grouped_linear_e4m3_block(xq, x_scale, wq, w_scale, expert_offsets=None, x_scale_index=None, y=None, ws=None,
                                  stream=None):
    """y = x w^T of each expert's rows, both in e4m3 with a scale for each block of 128 (as moe_quantize_e4m3_block makes
    them, or any fp32 scales): xq [rows, D], wq [E, F, D].  x_scale_index (perm_src) finds the row of x_scale; without
    expert_offsets E is 1: a dense product.  Rows of y behind the last segment are not written."""
    rows, D = _rows(xq, "xq")
    E, F, _ = _weights(wq)
    n = _rows(x_scale, "x_scale")[0]
    if y is None:
        y, = _new(stream, ((rows, F), _BF16, xq.device))
    if ws is None:
        ws = _header(stream, "combine", xq.device)
    _ready("moe_grouped_linear_e4m3_block", ws, (xq, _U8, (rows, D), "xq"), (x_scale, _F32, (n, _blocks(D)), "x_scale"),
           (wq, _U8, (E, F, D), "wq"), (w_scale, _F32, (E, _blocks(F), _blocks(D)), "w_scale"),
           (expert_offsets, _I32, (E + 1,), "expert_offsets"), (x_scale_index, _I32, (rows,), "x_scale_index"),
           (y, _BF16, (rows, F), "y"))
    s = (_lib or load()).moe_grouped_linear_e4m3_block(_addr(xq), _addr(x_scale), _addr(x_scale_index), n,
                                                       _addr(expert_offsets), rows, _addr(wq), _addr(w_scale), E, D, F, _addr(y),
                                                       _addr(ws), ws.numel(), _stream_of(xq, stream))
    if s:
        _check("moe_grouped_linear_e4m3_block", s)
    return y


def moe_grouped_linear_e4m3_block_backward(wq, w_scale, dyq, dy_scale, dyq_seg, dy_scale_seg, xq_seg, x_scale_seg,
                                           expert_offsets=None, dx=None, dw=None, ws=None, stream=None):
    """Gradients (dx, dw) of moe_grouped_linear_e4m3_block from quantised operands: the incoming gradient along its columns
    (dyq, dy_scale) for dx and along its rows (dyq_seg, dy_scale_seg) for dw, x along its rows (xq_seg, x_scale_seg).  Rows of dx
    behind the last segment are not written; dw of an expert without rows is zero."""
    E, F, D = _weights(wq)
    rows = _rows(dyq, "dyq")[0]
    seg = segment_rows(rows, E)
    if dx is None:
        dx, = _new(stream, ((rows, D), _BF16, wq.device))
    if dw is None:
        dw, = _new(stream, ((E, F, D), _BF16, wq.device))
    if ws is None:
        ws = _header(stream, "combine", wq.device)
    _ready("moe_grouped_linear_e4m3_block_backward", ws, (wq, _U8, (E, F, D), "wq"),
           (w_scale, _F32, (E, _blocks(F), _blocks(D)), "w_scale"), (dyq, _U8, (rows, F), "dyq"),
           (dy_scale, _F32, (rows, _blocks(F)), "dy_scale"), (dyq_seg, _U8, (seg, F), "dyq_seg"),
           (dy_scale_seg, _F32, (seg // BLOCK, F), "dy_scale_seg"), (xq_seg, _U8, (seg, D), "xq_seg"),
           (x_scale_seg, _F32, (seg // BLOCK, D), "x_scale_seg"), (expert_offsets, _I32, (E + 1,), "expert_offsets"),
           (dx, _BF16, (rows, D), "dx"), (dw, _BF16, (E, F, D), "dw"))
    s = (_lib or load()).moe_grouped_linear_e4m3_block_backward(
        _addr(dyq), _addr(dy_scale), _addr(dyq_seg), _addr(dy_scale_seg), _addr(xq_seg), _addr(x_scale_seg),
        _addr(expert_offsets), rows, _addr(wq), _addr(w_scale), E, D, F, _addr(dx), _addr(dw), _addr(ws), ws.numel(),
        _stream_of(wq, stream))
    if s:
        _check("moe_grouped_linear_e4m3_block_backward", s)
    return dx, dw
