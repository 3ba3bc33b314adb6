"""ctypes binding of ``libmi355moe.so``: argument marshalling only.

Each function has the name of the C entry point it calls.  It checks dtype,
device, shape and contiguity of the torch tensors it is given (raising
``ValueError`` before anything reaches C), allocates outputs the caller did
not pass, and forwards raw device pointers plus the current HIP stream.  All
arithmetic of the layer runs in the library's HIP kernels; there is no other
path.  PyTorch serves only as the device-memory and stream provider.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmi355moe.so")

MOE_STATUS = {
    0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN", 4: "MOE_ERR_ENUM",
    5: "MOE_ERR_WORKSPACE", 6: "MOE_ERR_HIP", 7: "MOE_ERR_UNSUPPORTED_DEVICE",
    8: "MOE_ERR_SCRATCH_LIMIT",
}

# Entry points declared in include/mi355moe.h.
EXPORTS = (
    "moe_abi_version", "moe_strerror", "moe_workspace_size", "moe_route", "moe_quant_mxfp8",
    "moe_permute", "moe_fc1_situ", "moe_fc2_combine", "moe_prepack_w13", "moe_prepack_w2",
    "moe_fc1_situ_tiled", "moe_fc2_combine_tiled", "moe_route_quant_permute",
    "moe_prepack_w13_layout", "moe_permute_noalloc", "moe_quant_permute",
    "moe_add_rmsnorm", "moe_quant_int8", "moe_int8_workspace_size",
    "moe_int8_matmul_workspace_size", "moe_int8_matmul", "moe_int8_linear",
    "moe_gate_workspace_size", "moe_gate_logits", "moe_route_groups",
)

# moe_w13_layout_t values (row order of a w13 tensor)
W13_GATE_UP, W13_UP_GATE, W13_INTERLEAVED = 0, 1, 2
# moe_combine_t values (how moe_fc2_combine sums a token's top-k rows)
COMBINE_DETERMINISTIC, COMBINE_ATOMIC = 0, 1
# moe_q8_t values (the 8-bit output of moe_add_rmsnorm)
Q8_NONE, Q8_MXFP8, Q8_INT8 = 0, 1, 2
# moe_out_t values, by output dtype
_OUT_TYPE = {torch.bfloat16: 0, torch.float32: 1}
# moe_score_t and moe_group_score_t values (moe_route_groups)
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t


def load_library(path: str = _LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m mxfp8_mxfp4_experts_amd.build` "
            "(the MoE layer has no other implementation to fall back to)")
    lib = ctypes.CDLL(path)
    lib.moe_abi_version.restype = _I
    lib.moe_abi_version.argtypes = []
    lib.moe_strerror.restype = ctypes.c_char_p
    lib.moe_strerror.argtypes = [_I]
    lib.moe_workspace_size.restype = _SZ
    lib.moe_workspace_size.argtypes = [_I, _I, _I, _I, _I, _I]
    lib.moe_route.restype = _I
    lib.moe_route.argtypes = [_P, _I64, _P, _I, _I, _I, _F, _P, _P, _P]
    lib.moe_quant_mxfp8.restype = _I
    lib.moe_quant_mxfp8.argtypes = [_P, _I64, _I, _I, _P, _P, _P]
    lib.moe_permute.restype = _I
    lib.moe_permute.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]
    lib.moe_permute_noalloc.restype = _I
    lib.moe_permute_noalloc.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P]
    lib.moe_quant_permute.restype = _I
    lib.moe_quant_permute.argtypes = [_P, _I64, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                                      _SZ, _P]
    lib.moe_route_quant_permute.restype = _I
    lib.moe_route_quant_permute.argtypes = [_P, _I64, _P, _I, _I, _I, _F, _P, _I64, _I, _I, _I,
                                            _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
    lib.moe_fc1_situ.restype = _I
    lib.moe_fc1_situ.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _F, _F, _P, _P, _P,
                                 _SZ, _P]
    lib.moe_fc2_combine.restype = _I
    lib.moe_fc2_combine.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P,
                                    _I64, _P, _SZ, _P]
    lib.moe_fc1_situ_tiled.restype = _I
    lib.moe_fc1_situ_tiled.argtypes = lib.moe_fc1_situ.argtypes
    lib.moe_fc2_combine_tiled.restype = _I
    lib.moe_fc2_combine_tiled.argtypes = lib.moe_fc2_combine.argtypes
    for name in ("moe_prepack_w13", "moe_prepack_w2"):
        getattr(lib, name).restype = _I
        getattr(lib, name).argtypes = [_P, _P, _I, _I, _I, _P, _P, _P]
    lib.moe_prepack_w13_layout.restype = _I
    lib.moe_prepack_w13_layout.argtypes = [_P, _P, _I, _I, _I, _I, _P, _P, _P]
    lib.moe_add_rmsnorm.restype = _I
    lib.moe_add_rmsnorm.argtypes = [_P, _I64, _P, _I64, _P, _F, _I, _I, _I, _P, _I64, _P, _I64,
                                    _P, _P, _P]
    lib.moe_quant_int8.restype = _I
    lib.moe_quant_int8.argtypes = [_P, _I64, _I, _I, _P, _P, _P]
    for name in ("moe_int8_workspace_size", "moe_int8_matmul_workspace_size",
                 "moe_gate_workspace_size"):
        getattr(lib, name).restype = _SZ
        getattr(lib, name).argtypes = [_I, _I, _I]
    lib.moe_int8_matmul.restype = _I
    lib.moe_int8_matmul.argtypes = [_P, _I64, _P, _P, _P, _I, _I, _I, _I, _P, _I64, _P, _SZ, _P]
    lib.moe_int8_linear.restype = _I
    lib.moe_int8_linear.argtypes = [_P, _I64, _P, _P, _I, _I, _I, _I, _P, _I64, _P, _SZ, _P]
    lib.moe_gate_logits.restype = _I
    lib.moe_gate_logits.argtypes = [_P, _I64, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]
    lib.moe_route_groups.restype = _I
    lib.moe_route_groups.argtypes = [_P, _I64, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]
    return lib


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


class MoEError(RuntimeError):
    def __init__(self, name: str, status: int):
        msg = lib().moe_strerror(status).decode()
        super().__init__(f"{name} returned {MOE_STATUS.get(status, status)}: {msg}")
        self.status = status


def _check(name: str, status: int):
    if status != 0:
        raise MoEError(name, status)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _need(t: torch.Tensor, name: str, dtype, shape=None, contiguous=True, device=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _as_u16(x: torch.Tensor, name: str) -> torch.Tensor:
    if x.dtype == torch.bfloat16:
        return x.view(torch.uint16)   # same element size: any strides
    if x.dtype == torch.uint16:
        return x
    raise ValueError(f"{name} must be bfloat16 (or uint16 bf16 bits), got {x.dtype}")


def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_workspace_size(T: int, top_k: int, E_local: int, H: int, I: int,
                       mode: int = COMBINE_DETERMINISTIC) -> int:
    n = lib().moe_workspace_size(T, top_k, E_local, H, I, int(mode))
    if n == 0:
        raise ValueError("invalid sizes or combine mode for moe_workspace_size")
    return n


def moe_route(logits: torch.Tensor, bias: Optional[torch.Tensor], top_k: int,
              routed_scaling: float = 1.0, topk_idx: Optional[torch.Tensor] = None,
              topk_w: Optional[torch.Tensor] = None):
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [T, E] with unit column stride")
    _need(logits, "logits", torch.float32, contiguous=False)
    T, E = logits.shape
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,), device=logits.device)
    if topk_idx is None:
        topk_idx = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _need(topk_idx, "topk_idx", torch.int32, (T, top_k), device=logits.device)
    _need(topk_w, "topk_w", torch.float32, (T, top_k), device=logits.device)
    _check("moe_route", lib().moe_route(_ptr(logits), logits.stride(0), _ptr(bias), T, E, top_k,
                                        float(routed_scaling), _ptr(topk_idx), _ptr(topk_w),
                                        _stream()))
    return topk_idx, topk_w


def moe_quant_mxfp8(x: torch.Tensor, xq: Optional[torch.Tensor] = None,
                    xs: Optional[torch.Tensor] = None):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [T, H] with unit column stride")
    xb = x if x.dtype == torch.uint16 else (x.view(torch.uint16) if x.dtype == torch.bfloat16 else None)
    if xb is None:
        raise ValueError(f"x must be bfloat16 (or uint16 bf16 bits), got {x.dtype}")
    _need(xb, "x", torch.uint16, contiguous=False)
    T, H = x.shape
    if xq is None:
        xq = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    if xs is None:
        xs = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    _need(xq, "xq", torch.uint8, (T, H), device=x.device)
    _need(xs, "xs", torch.uint8, (T, H // 32), device=x.device)
    _check("moe_quant_mxfp8", lib().moe_quant_mxfp8(_ptr(xb), x.stride(0), T, H, _ptr(xq),
                                                    _ptr(xs), _stream()))
    return xq, xs


def moe_route_quant_permute(logits: torch.Tensor, bias: Optional[torch.Tensor], top_k: int,
                            routed_scaling: float, x: torch.Tensor, expert_offset: int,
                            E_local: int, workspace: torch.Tensor, topk_idx=None, topk_w=None,
                            xq=None, xs=None, expert_offsets=None, sorted_route=None,
                            route_row=None):
    """moe_route, moe_quant_mxfp8 and moe_permute as one call (same results)."""
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [T, E] with unit column stride")
    _need(logits, "logits", torch.float32, contiguous=False)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [T, H] with unit column stride")
    xb = x if x.dtype == torch.uint16 else (x.view(torch.uint16) if x.dtype == torch.bfloat16 else None)
    if xb is None:
        raise ValueError(f"x must be bfloat16 (or uint16 bf16 bits), got {x.dtype}")
    _need(xb, "x", torch.uint16, contiguous=False)
    T, E = logits.shape
    H = x.shape[1]
    if x.shape[0] != T:
        raise ValueError("x and logits must have the same number of rows")
    dev = logits.device
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,), device=dev)
    R = T * top_k
    topk_idx = torch.empty((T, top_k), dtype=torch.int32, device=dev) if topk_idx is None else topk_idx
    topk_w = torch.empty((T, top_k), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    xq = torch.empty((T, H), dtype=torch.uint8, device=dev) if xq is None else xq
    xs = torch.empty((T, H // 32), dtype=torch.uint8, device=dev) if xs is None else xs
    if expert_offsets is None:
        expert_offsets = torch.empty(E_local + 1, dtype=torch.int32, device=dev)
    sorted_route = torch.empty(R, dtype=torch.int32, device=dev) if sorted_route is None else sorted_route
    route_row = torch.empty(R, dtype=torch.int32, device=dev) if route_row is None else route_row
    _need(topk_idx, "topk_idx", torch.int32, (T, top_k), device=dev)
    _need(topk_w, "topk_w", torch.float32, (T, top_k), device=dev)
    _need(xq, "xq", torch.uint8, (T, H), device=dev)
    _need(xs, "xs", torch.uint8, (T, H // 32), device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (R,), device=dev)
    _need(route_row, "route_row", torch.int32, (R,), device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    _check("moe_route_quant_permute", lib().moe_route_quant_permute(
        _ptr(logits), logits.stride(0), _ptr(bias), T, E, top_k, float(routed_scaling), _ptr(xb),
        x.stride(0), H, expert_offset, E_local, _ptr(topk_idx), _ptr(topk_w), _ptr(xq), _ptr(xs),
        _ptr(expert_offsets), _ptr(sorted_route), _ptr(route_row), _ptr(workspace),
        workspace.numel(), _stream()))
    return topk_idx, topk_w, xq, xs, expert_offsets, sorted_route, route_row


def moe_permute(topk_idx: torch.Tensor, expert_offset: int, E_local: int, workspace: torch.Tensor,
                expert_offsets=None, sorted_route=None, route_row=None):
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, top_k]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    _need(workspace, "workspace", torch.uint8, device=dev)
    if expert_offsets is None:
        expert_offsets = torch.empty(E_local + 1, dtype=torch.int32, device=dev)
    if sorted_route is None:
        sorted_route = torch.empty(T * K, dtype=torch.int32, device=dev)
    if route_row is None:
        route_row = torch.empty(T * K, dtype=torch.int32, device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (T * K,), device=dev)
    _need(route_row, "route_row", torch.int32, (T * K,), device=dev)
    _check("moe_permute", lib().moe_permute(_ptr(topk_idx), T, K, expert_offset, E_local,
                                            _ptr(expert_offsets), _ptr(sorted_route),
                                            _ptr(route_row), _ptr(workspace), workspace.numel(),
                                            _stream()))
    return expert_offsets, sorted_route, route_row


def moe_quant_permute(x: torch.Tensor, topk_idx: torch.Tensor, expert_offset: int, E_local: int,
                      workspace: torch.Tensor, xq=None, xs=None, expert_offsets=None,
                      sorted_route=None, route_row=None):
    """moe_quant_mxfp8 and moe_permute as one call (same results), for top-k
    ids computed elsewhere."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [T, H] with unit column stride")
    xb = x if x.dtype == torch.uint16 else (x.view(torch.uint16) if x.dtype == torch.bfloat16 else None)
    if xb is None:
        raise ValueError(f"x must be bfloat16 (or uint16 bf16 bits), got {x.dtype}")
    _need(xb, "x", torch.uint16, contiguous=False)
    _need(topk_idx, "topk_idx", torch.int32, device=x.device)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != x.shape[0]:
        raise ValueError("topk_idx must be [T, top_k] with the rows of x")
    T, H = x.shape
    K = topk_idx.shape[1]
    dev = x.device
    _need(workspace, "workspace", torch.uint8, device=dev)
    if xq is None:
        xq = torch.empty((T, H), dtype=torch.uint8, device=dev)
    if xs is None:
        xs = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
    if expert_offsets is None:
        expert_offsets = torch.empty(E_local + 1, dtype=torch.int32, device=dev)
    if sorted_route is None:
        sorted_route = torch.empty(T * K, dtype=torch.int32, device=dev)
    if route_row is None:
        route_row = torch.empty(T * K, dtype=torch.int32, device=dev)
    _need(xq, "xq", torch.uint8, (T, H), device=dev)
    _need(xs, "xs", torch.uint8, (T, H // 32), device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (T * K,), device=dev)
    _need(route_row, "route_row", torch.int32, (T * K,), device=dev)
    _check("moe_quant_permute", lib().moe_quant_permute(
        _ptr(xb), x.stride(0), T, H, _ptr(topk_idx), K, expert_offset, E_local, _ptr(xq),
        _ptr(xs), _ptr(expert_offsets), _ptr(sorted_route), _ptr(route_row), _ptr(workspace),
        workspace.numel(), _stream()))
    return xq, xs, expert_offsets, sorted_route, route_row


def moe_permute_noalloc(topk_idx: torch.Tensor, expert_offset: int, E_local: int,
                        expert_offsets=None, sorted_route=None, route_row=None):
    """moe_permute without a workspace (the library's static scratch holds
    the schedule); same grouping outputs."""
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, top_k]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if expert_offsets is None:
        expert_offsets = torch.empty(E_local + 1, dtype=torch.int32, device=dev)
    if sorted_route is None:
        sorted_route = torch.empty(T * K, dtype=torch.int32, device=dev)
    if route_row is None:
        route_row = torch.empty(T * K, dtype=torch.int32, device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (T * K,), device=dev)
    _need(route_row, "route_row", torch.int32, (T * K,), device=dev)
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        _ptr(topk_idx), T, K, expert_offset, E_local, _ptr(expert_offsets), _ptr(sorted_route),
        _ptr(route_row), _stream()))
    return expert_offsets, sorted_route, route_row


def moe_fc1_situ(xq, xs, top_k, expert_offsets, sorted_route, w13, w13_s, workspace,
                 situ_alpha: float = 4.0, situ_beta: float = 25.0, hq=None, hs=None,
                 tiled: bool = False):
    """``tiled``: w13 / w13_s come from ``moe_prepack_w13`` (calls
    moe_fc1_situ_tiled); they keep the checkpoint tensor shapes."""
    _need(xq, "xq", torch.uint8)
    T, H = xq.shape
    dev = xq.device
    _need(w13, "w13", torch.uint8, device=dev)
    if w13.dim() != 3 or w13.shape[2] != H // 2:
        raise ValueError("w13 must be [E_local, 2I, H/2]")
    E_local, twoI, _ = w13.shape
    I = twoI // 2
    _need(xs, "xs", torch.uint8, (T, H // 32), device=dev)
    _need(w13_s, "w13_s", torch.uint8, (E_local, twoI, H // 32), device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (T * top_k,), device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    R = T * top_k
    if hq is None:
        hq = torch.empty((R, I), dtype=torch.uint8, device=dev)
    if hs is None:
        hs = torch.empty((R, I // 32), dtype=torch.uint8, device=dev)
    _need(hq, "hq", torch.uint8, (R, I), device=dev)
    _need(hs, "hs", torch.uint8, (R, I // 32), device=dev)
    name = "moe_fc1_situ_tiled" if tiled else "moe_fc1_situ"
    _check(name, getattr(lib(), name)(
        _ptr(xq), _ptr(xs), T, H, I, top_k, E_local, _ptr(expert_offsets), _ptr(sorted_route),
        _ptr(w13), _ptr(w13_s), float(situ_alpha), float(situ_beta), _ptr(hq), _ptr(hs),
        _ptr(workspace), workspace.numel(), _stream()))
    return hq, hs


def moe_fc2_combine(hq, hs, T, top_k, expert_offsets, sorted_route, route_row, topk_w, w2, w2_s,
                    workspace, out=None, tiled: bool = False, mode: int = COMBINE_DETERMINISTIC):
    """``tiled``: w2 / w2_s come from ``moe_prepack_w2`` (calls
    moe_fc2_combine_tiled).  ``mode``: COMBINE_DETERMINISTIC or
    COMBINE_ATOMIC (the workspace must be sized for it)."""
    _need(hq, "hq", torch.uint8)
    R, I = hq.shape
    dev = hq.device
    _need(w2, "w2", torch.uint8, device=dev)
    if w2.dim() != 3 or w2.shape[2] != I // 2:
        raise ValueError("w2 must be [E_local, H, I/2]")
    E_local, H, _ = w2.shape
    if R != T * top_k:
        raise ValueError("hq must have T * top_k rows")
    _need(hs, "hs", torch.uint8, (R, I // 32), device=dev)
    _need(w2_s, "w2_s", torch.uint8, (E_local, H, I // 32), device=dev)
    _need(expert_offsets, "expert_offsets", torch.int32, (E_local + 1,), device=dev)
    _need(sorted_route, "sorted_route", torch.int32, (R,), device=dev)
    _need(route_row, "route_row", torch.int32, (R,), device=dev)
    _need(topk_w, "topk_w", torch.float32, (T, top_k), device=dev)
    _need(workspace, "workspace", torch.uint8, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if out.dim() != 2 or out.shape[0] != T or out.shape[1] != H or out.stride(1) != 1:
        raise ValueError("out must be [T, H] with unit column stride")
    ob = _as_u16(out, "out")
    _need(ob, "out", torch.uint16, contiguous=False, device=dev)
    name = "moe_fc2_combine_tiled" if tiled else "moe_fc2_combine"
    _check(name, getattr(lib(), name)(
        _ptr(hq), _ptr(hs), T, H, I, top_k, E_local, _ptr(expert_offsets), _ptr(sorted_route),
        _ptr(route_row), _ptr(topk_w), _ptr(w2), _ptr(w2_s), int(mode), _ptr(ob), out.stride(0),
        _ptr(workspace), workspace.numel(), _stream()))
    return out


def _weight_pair(name, w, w_s):
    """A checkpoint weight [E, N, K/2] and its scales [E, N, K/32]: shapes and
    dtypes checked here, since the kernels read every byte they imply."""
    _need(w, name + " weights", torch.uint8)
    if w.dim() != 3 or w.shape[2] % 16 != 0:
        raise ValueError(f"{name} weights must be [E, N, K/2] with K a multiple of 32")
    E, N, half_k = w.shape
    _need(w_s, name + " scales", torch.uint8, (E, N, 2 * half_k // 32), device=w.device)
    return E, N, 2 * half_k


def _prepack(name, w, w_s, H, I):
    tw = torch.empty_like(w)
    tws = torch.empty_like(w_s)
    _check(name, getattr(lib(), name)(_ptr(w), _ptr(w_s), w.shape[0], H, I, _ptr(tw), _ptr(tws),
                                      _stream()))
    return tw, tws


def moe_prepack_w13(w13, w13_s):
    """Checkpoint w13 [E, 2I, H/2] + scales [E, 2I, H/32] -> tiled copies
    (same shapes)."""
    E, twoI, H = _weight_pair("moe_prepack_w13", w13, w13_s)
    return _prepack("moe_prepack_w13", w13, w13_s, H, twoI // 2)


def moe_prepack_w13_layout(w13, w13_s, layout: int):
    """w13 [E, 2I, H/2] + scales [E, 2I, H/32] whose rows are in ``layout``
    order (W13_GATE_UP, W13_UP_GATE or W13_INTERLEAVED) -> tiled copies."""
    E, twoI, H = _weight_pair("moe_prepack_w13_layout", w13, w13_s)
    tw, tws = torch.empty_like(w13), torch.empty_like(w13_s)
    _check("moe_prepack_w13_layout", lib().moe_prepack_w13_layout(
        _ptr(w13), _ptr(w13_s), E, H, twoI // 2, int(layout), _ptr(tw), _ptr(tws), _stream()))
    return tw, tws


def moe_prepack_w2(w2, w2_s):
    """Checkpoint w2 [E, H, I/2] + scales [E, H, I/32] -> tiled copies (same
    shapes)."""
    E, H, I = _weight_pair("moe_prepack_w2", w2, w2_s)
    return _prepack("moe_prepack_w2", w2, w2_s, H, I)


# ---------------------------------------------------------------------------
# Around the experts.  In a decode step these kernels run for a few
# microseconds, so what a call costs on the host counts: a compiled helper
# (csrc_py/tensor_args.cpp) looks at each tensor once.  It only says whether a
# tensor is plainly right; strided rows and what is wrong are found here.

_BF16, _F32, _U8, _I8, _I32 = (torch.bfloat16, torch.float32, torch.uint8, torch.int8,
                               torch.int32)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _load_args():
    global _head, _plain
    try:
        from . import _tensor_args
    except ImportError as e:
        raise ImportError("_tensor_args.so is missing or does not fit this torch: build it with "
                          "`python -m mxfp8_mxfp4_experts_amd.build`") from e
    _head, _plain = _tensor_args.head, _tensor_args.plain


def _head(x):
    """(device index, rows, columns) of a 2-D tensor on the current GPU, or
    None (the helper's function takes this one's place on the first call)."""
    _load_args()
    return _head(x)


def _plain(t, dtype, rows, cols, idx):
    """The address of a contiguous tensor of this dtype, shape (``cols`` -1:
    one-dimensional) and device, or -1 (replaced as ``_head`` is)."""
    _load_args()
    return _plain(t, dtype, rows, cols, idx)


def _no_head(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    raise ValueError(f"{name} is on {x.device}, which is not the current device")


def _wrong(t, name, dtype, shape, idx):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.shape != shape or t.get_device() != idx:
        raise ValueError(f"{name} must be {dtype} {shape} on cuda:{idx}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


def _rows(t, name, dtype, T, C, idx):
    """Address and row stride of a [T, C] tensor whose rows may be strided."""
    _wrong(t, name, dtype, (T, C), idx)
    ld, one = t.stride()
    if one != 1 and C != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld if T > 1 else C   # one row's stride says nothing


def _refuse(t, name, dtype, shape, idx):
    _wrong(t, name, dtype, shape, idx)
    raise ValueError(f"{name} must be contiguous")


def _new(shape, dtype, idx):
    return torch.empty(shape, dtype=dtype, device=torch.device("cuda", idx))


def _workspace(ws, size_of, sizes, idx):
    """The given workspace, or a new one of the size that the library names
    (the library refuses a given one that is too small)."""
    if ws is None:
        return _new(size_of(*sizes), _U8, idx)
    if ws.dtype is not _U8 or ws.get_device() != idx or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{idx}")
    return ws


def moe_add_rmsnorm(x, weight, eps: float, residual=None, q8: int = Q8_NONE, residual_out=None,
                    y=None, want_y: bool = True, xq=None, xs=None):
    """h = x + residual, y = h * weight / sqrt(mean(h^2) + eps), and y in 8
    bits.  Returns ``(residual_out, y, xq, xs)``: bf16(h) (None without a
    residual, unless a buffer is given), bf16(y) (None with ``want_y=False``
    and no buffer), and for ``q8`` Q8_MXFP8 uint8 [T, H] and [T, H/32], for
    Q8_INT8 int8 [T, H] and float [T], else None.  ``residual_out`` may be
    ``x`` or ``residual`` itself."""
    head = _head(x)
    if head is None:
        _no_head(x, "x")
    idx, T, H = head
    x_p, ld_x = _plain(x, _BF16, T, H, idx), H
    if x_p < 0:
        x_p, ld_x = _rows(x, "x", _BF16, T, H, idx)
    w_p = _plain(weight, _BF16, H, -1, idx)
    if w_p < 0:
        _refuse(weight, "weight", _BF16, (H,), idx)
    r_p = h_p = y_p = q_p = s_p = None
    ld_r = ld_h = ld_y = H
    if residual is not None:
        r_p = _plain(residual, _BF16, T, H, idx)
        if r_p < 0:
            r_p, ld_r = _rows(residual, "residual", _BF16, T, H, idx)
        if residual_out is None:
            residual_out = _new((T, H), _BF16, idx)
    if residual_out is not None:
        h_p = _plain(residual_out, _BF16, T, H, idx)
        if h_p < 0:
            h_p, ld_h = _rows(residual_out, "residual_out", _BF16, T, H, idx)
    if y is None and want_y:
        y = _new((T, H), _BF16, idx)
    if y is not None:
        y_p = _plain(y, _BF16, T, H, idx)
        if y_p < 0:
            y_p, ld_y = _rows(y, "y", _BF16, T, H, idx)
    if q8 == Q8_MXFP8 or q8 == Q8_INT8:
        kind, s_kind, s_cols = (_U8, _U8, H // 32) if q8 == Q8_MXFP8 else (_I8, _F32, -1)
        s_shape = (T, s_cols) if s_cols >= 0 else (T,)
        if xq is None:
            xq = _new((T, H), kind, idx)
        if xs is None:
            xs = _new(s_shape, s_kind, idx)
        q_p = _plain(xq, kind, T, H, idx)
        if q_p < 0:
            _refuse(xq, "xq", kind, (T, H), idx)
        s_p = _plain(xs, s_kind, T, s_cols, idx)
        if s_p < 0:
            _refuse(xs, "xs", s_kind, s_shape, idx)
    else:
        xq = xs = None
    st = (_lib or lib()).moe_add_rmsnorm(x_p, ld_x, r_p, ld_r, w_p, eps, T, H, q8, h_p, ld_h, y_p,
                                         ld_y, q_p, s_p, _raw_stream(idx))
    if st:
        raise MoEError("moe_add_rmsnorm", st)
    return residual_out, y, xq, xs


def moe_quant_int8(x, xq=None, xs=None):
    """bf16 rows [T, H] -> int8 [T, H] and one float scale per row [T]."""
    head = _head(x)
    if head is None:
        _no_head(x, "x")
    idx, T, H = head
    x_p, ld_x = _plain(x, _BF16, T, H, idx), H
    if x_p < 0:
        x_p, ld_x = _rows(x, "x", _BF16, T, H, idx)
    if xq is None:
        xq = _new((T, H), _I8, idx)
    if xs is None:
        xs = _new((T,), _F32, idx)
    q_p, s_p = _plain(xq, _I8, T, H, idx), _plain(xs, _F32, T, -1, idx)
    if q_p < 0:
        _refuse(xq, "xq", _I8, (T, H), idx)
    if s_p < 0:
        _refuse(xs, "xs", _F32, (T,), idx)
    st = (_lib or lib()).moe_quant_int8(x_p, ld_x, T, H, q_p, s_p, _raw_stream(idx))
    if st:
        raise MoEError("moe_quant_int8", st)
    return xq, xs


def moe_int8_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of moe_int8_linear and moe_int8_matmul; a buffer for M
    rows serves fewer."""
    n = lib().moe_int8_workspace_size(M, N, K)
    if n == 0:
        raise ValueError("invalid sizes for moe_int8_workspace_size")
    return n


def moe_int8_matmul_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of moe_int8_matmul alone; a buffer for M rows serves
    fewer."""
    return lib().moe_int8_matmul_workspace_size(M, N, K)


def _int8_out(out, out_dtype, M, N, idx):
    """The output tensor, its address, row stride and moe_out_t value."""
    if out is None:
        if out_dtype not in _OUT_TYPE:
            raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
        out = _new((M, N), out_dtype, idx)
    kind = out.dtype
    if kind not in _OUT_TYPE:
        raise ValueError(f"out must be bfloat16 or float32, got {kind}")
    o_p, ld_out = _plain(out, kind, M, N, idx), N
    if o_p < 0:
        o_p, ld_out = _rows(out, "out", kind, M, N, idx)
    return out, o_p, ld_out, _OUT_TYPE[kind]


def _int8_weight(w, w_s, K, idx):
    """N and the addresses of an int8 weight [N, K] and its scales."""
    N = w.shape[0] if isinstance(w, torch.Tensor) and w.dim() == 2 else -1
    w_p = _plain(w, _I8, N, K, idx)
    if w_p < 0:
        if N < 0 or w.shape[1] != K:
            raise ValueError(f"w must be [N, {K}]")
        _refuse(w, "w", _I8, (N, K), idx)
    s_p = _plain(w_s, _F32, N, -1, idx)
    if s_p < 0:
        _refuse(w_s, "w_s", _F32, (N,), idx)
    return N, w_p, s_p


def moe_int8_matmul(xq, xs, w, w_s, out=None, out_dtype=torch.bfloat16, workspace=None):
    """out [M, N] = (xq [M, K] . w [N, K]) * xs [M] * w_s [N], the sum exact in
    int32; ``out`` or ``out_dtype`` says bf16 or float32."""
    head = _head(xq)
    if head is None:
        _no_head(xq, "xq")
    idx, M, K = head
    q_p, ld_xq = _plain(xq, _I8, M, K, idx), K
    if q_p < 0:
        q_p, ld_xq = _rows(xq, "xq", _I8, M, K, idx)
    x_p = _plain(xs, _F32, M, -1, idx)
    if x_p < 0:
        _refuse(xs, "xs", _F32, (M,), idx)
    N, w_p, s_p = _int8_weight(w, w_s, K, idx)
    out, o_p, ld_out, kind = _int8_out(out, out_dtype, M, N, idx)
    L = _lib or lib()
    workspace = _workspace(workspace, L.moe_int8_matmul_workspace_size, (M, N, K), idx)
    st = L.moe_int8_matmul(q_p, ld_xq, x_p, w_p, s_p, M, N, K, kind, o_p, ld_out,
                           workspace.data_ptr(), workspace.numel(), _raw_stream(idx))
    if st:
        raise MoEError("moe_int8_matmul", st)
    return out


def moe_int8_linear(x, w, w_s, out=None, out_dtype=torch.bfloat16, workspace=None):
    """moe_quant_int8 of x [M, K] (bf16) and moe_int8_matmul as one call."""
    head = _head(x)
    if head is None:
        _no_head(x, "x")
    idx, M, K = head
    x_p, ld_x = _plain(x, _BF16, M, K, idx), K
    if x_p < 0:
        x_p, ld_x = _rows(x, "x", _BF16, M, K, idx)
    N, w_p, s_p = _int8_weight(w, w_s, K, idx)
    out, o_p, ld_out, kind = _int8_out(out, out_dtype, M, N, idx)
    L = _lib or lib()
    workspace = _workspace(workspace, L.moe_int8_workspace_size, (M, N, K), idx)
    st = L.moe_int8_linear(x_p, ld_x, w_p, s_p, M, N, K, kind, o_p, ld_out, workspace.data_ptr(),
                           workspace.numel(), _raw_stream(idx))
    if st:
        raise MoEError("moe_int8_linear", st)
    return out


def moe_gate_workspace_size(T: int, E: int, H: int) -> int:
    """Workspace bytes of moe_gate_logits; a buffer for T tokens serves fewer."""
    return lib().moe_gate_workspace_size(T, E, H)


def moe_gate_logits(x, w, out=None, workspace=None):
    """Router logits float [T, E] of x [T, H] and w [E, H], both bf16."""
    head = _head(x)
    if head is None:
        _no_head(x, "x")
    idx, T, H = head
    x_p, ld_x = _plain(x, _BF16, T, H, idx), H
    if x_p < 0:
        x_p, ld_x = _rows(x, "x", _BF16, T, H, idx)
    E = w.shape[0] if isinstance(w, torch.Tensor) and w.dim() == 2 else -1
    w_p = _plain(w, _BF16, E, H, idx)
    if w_p < 0:
        if E < 0:
            raise ValueError(f"w must be [E, {H}]")
        _refuse(w, "w", _BF16, (E, H), idx)
    if out is None:
        out = _new((T, E), _F32, idx)
    o_p, ld_out = _plain(out, _F32, T, E, idx), E
    if o_p < 0:
        o_p, ld_out = _rows(out, "out", _F32, T, E, idx)
    L = _lib or lib()
    workspace = _workspace(workspace, L.moe_gate_workspace_size, (T, E, H), idx)
    st = L.moe_gate_logits(x_p, ld_x, w_p, T, E, H, o_p, ld_out, workspace.data_ptr(),
                           workspace.numel(), _raw_stream(idx))
    if st:
        raise MoEError("moe_gate_logits", st)
    return out


def moe_route_groups(logits, bias, top_k: int, n_group: int = 1, topk_group: int = 1,
                     score: int = SCORE_SIGMOID, group_score: int = GROUP_TOP2,
                     renormalise: bool = True, routed_scaling: float = 1.0, topk_idx=None,
                     topk_w=None):
    """Group-limited top-k routing of float logits [T, E]: ids int32 and
    weights float [T, top_k]; -1 with weight 0 where no unmasked expert is
    left.  ``score``: SCORE_SIGMOID or SCORE_SOFTMAX; ``group_score``:
    GROUP_MAX or GROUP_TOP2."""
    head = _head(logits)
    if head is None:
        _no_head(logits, "logits")
    idx, T, E = head
    l_p, ld = _plain(logits, _F32, T, E, idx), E
    if l_p < 0:
        l_p, ld = _rows(logits, "logits", _F32, T, E, idx)
    b_p = None
    if bias is not None:
        b_p = _plain(bias, _F32, E, -1, idx)
        if b_p < 0:
            _refuse(bias, "bias", _F32, (E,), idx)
    if topk_idx is None:
        topk_idx = _new((T, top_k), _I32, idx)
    if topk_w is None:
        topk_w = _new((T, top_k), _F32, idx)
    i_p, w_p = _plain(topk_idx, _I32, T, top_k, idx), _plain(topk_w, _F32, T, top_k, idx)
    if i_p < 0:
        _refuse(topk_idx, "topk_idx", _I32, (T, top_k), idx)
    if w_p < 0:
        _refuse(topk_w, "topk_w", _F32, (T, top_k), idx)
    st = (_lib or lib()).moe_route_groups(l_p, ld, b_p, T, E, top_k, n_group, topk_group, score,
                                          group_score, 1 if renormalise else 0, routed_scaling,
                                          i_p, w_p, _raw_stream(idx))
    if st:
        raise MoEError("moe_route_groups", st)
    return topk_idx, topk_w
