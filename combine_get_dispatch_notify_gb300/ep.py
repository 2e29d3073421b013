"""Thin Python binding of libep_gb300.so (the C ABI in include/ep.h).

Functions carry the C names and only marshal arguments: they check that each
tensor is a contiguous CUDA tensor of the right dtype and shape, pass its
device address and the current CUDA stream, and raise :class:`EpError` on a
non-OK status.  Every step runs in the library's sm_103a kernels; there is no
CPU path.  ``alloc_*`` helpers allocate output tensors with torch.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_gb300.so")

EP_OK = 0
EP_ERR_INVALID_ARG = -1
EP_ERR_CUDA = -2
EP_ERR_CAPACITY = -3
EP_ERR_TIMEOUT = -4
EP_ERR_INCONSISTENT = -5
EP_ERR_INPUT = -6

EP_DEV_CAPACITY = 0x1
EP_DEV_TIMEOUT = 0x2
EP_DEV_INCONSISTENT = 0x4
EP_DEV_INPUT = 0x8

NODE_SIZE = 8

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class EpShape(ctypes.Structure):
    """Mirror of ep_shape_t."""

    _fields_ = [("num_ranks", _i32), ("num_tokens", _i32), ("num_topk", _i32),
                ("num_experts", _i32), ("hidden", _i32), ("num_channels", _i32),
                ("expert_alignment", _i32)]

    @classmethod
    def make(cls, R, T, K, E, H, C, expert_alignment=1) -> "EpShape":
        return cls(R, T, K, E, H, C, expert_alignment)

    @property
    def N(self) -> int:
        return 1 if self.num_ranks <= NODE_SIZE else self.num_ranks // NODE_SIZE

    @property
    def E_loc(self) -> int:
        return self.num_experts // self.num_ranks


class EpRoute(ctypes.Structure):
    """Mirror of ep_route_t: how ep_route scores and selects experts."""

    _fields_ = [("score", _i32), ("num_groups", _i32), ("topk_groups", _i32), ("group_top", _i32),
                ("renormalize", _i32), ("scale", ctypes.c_float)]

    @classmethod
    def make(cls, score="softmax", num_groups=1, topk_groups=1, group_top=1, renormalize=True,
             scale=1.0) -> "EpRoute":
        """``score`` is "softmax" or "sigmoid"."""
        if score not in ("softmax", "sigmoid"):
            raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
        return cls(int(score == "sigmoid"), num_groups, topk_groups, group_top, int(bool(renormalize)), scale)


class EpGemmShape(ctypes.Structure):
    """Mirror of ep_gemm_shape_t."""

    _fields_ = [("num_experts", _i32), ("capacity", _i32), ("n", _i32), ("k", _i32)]


class EpError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {ep_status_string(status)} ({status})")


_SIGS = {
    "ep_status_string": (ctypes.c_char_p, [_i32]),
    "ep_check_shape": (_i32, [ctypes.POINTER(EpShape)]),
    "ep_num_nodes": (_i32, [ctypes.POINTER(EpShape)]),
    "ep_notify_workspace_bytes": (_sz, [ctypes.POINTER(EpShape)]),
    "ep_get_dispatch_layout": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 6 + [_vp]),
    "ep_notify_dispatch": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 16 + [_sz, _vp, _vp, _vp]),
    "ep_dispatch": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 5 + [_i64] + [_vp] * 6 + [_vp]),
    "ep_dispatch_fp8": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _i32] + [_vp] * 4 + [_i64] +
                        [_vp] * 7 + [_vp]),
    "ep_combine": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _i64] + [_vp] * 5 + [_vp]),
    "ep_layout_notify": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 16 + [_vp, _sz, _vp, _vp, _vp]),
    "ep_layout_notify_fused": (_i32, [ctypes.POINTER(EpShape)]),
    "ep_layout_notify_workspace_bytes": (_sz, [ctypes.POINTER(EpShape)]),
    "ep_debug_layout_notify_tiled": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 16 +
                                     [_vp, _sz, _vp, _vp, _i32, _i32, _i32, _vp]),
    "ep_layout_notify_dispatch": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 18 + [_vp, _sz, _i64] + [_vp] * 7 +
                                  [_vp]),
    "ep_debug_layout_notify_dispatch_stall": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 18 + [_vp, _sz, _i64] +
                                              [_vp] * 6 + [_i32, _i32, _vp]),
    "ep_notify_dispatch_noalloc": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 15 + [_vp, _vp, _vp]),
    "ep_ll_layout": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "ep_ll_dispatch": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "ep_ll_combine": (_i32, [ctypes.POINTER(EpShape), _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "ep_check_route": (_i32, [ctypes.POINTER(EpShape), ctypes.POINTER(EpRoute)]),
    "ep_route": (_i32, [ctypes.POINTER(EpShape), ctypes.POINTER(EpRoute), _vp, _i32] + [_vp] * 4 + [_vp]),
    "ep_route_backward": (_i32, [ctypes.POINTER(EpShape), ctypes.POINTER(EpRoute), _vp, _i32] + [_vp] * 4 + [_vp]),
    "ep_ll_dispatch_fp8": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _vp, _i32] + [_vp] * 4 + [_vp]),
    "ep_check_gemm_shape": (_i32, [ctypes.POINTER(EpGemmShape)]),
    "ep_ll_gemm_fp8": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 7 + [_vp]),
    "ep_ll_gemm_swiglu_fp8": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 8 + [_vp]),
    "ep_debug_ll_gemm_fp8_stall": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 8 + [_i32] * 3 + [_vp]),
    "ep_ll_combine_backward": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _i32] + [_vp] * 6 + [_vp]),
    "ep_check_gemm_shape_bf16": (_i32, [ctypes.POINTER(EpGemmShape)]),
    "ep_ll_gemm_bf16": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 5 + [_vp]),
    "ep_ll_gemm_swiglu_bf16": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 6 + [_vp]),
    "ep_ll_gemm_dgrad_bf16": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 5 + [_vp]),
    "ep_ll_gemm_dswiglu_bf16": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 6 + [_vp]),
    "ep_ll_gemm_wgrad_bf16": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 4 + [_i32, _vp, _vp]),
    "ep_ll_dispatch_int8": (_i32, [ctypes.POINTER(EpShape), _vp, _vp, _vp, _i32] + [_vp] * 4 + [_vp]),
    "ep_ll_gemm_int8": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 7 + [_vp]),
    "ep_ll_gemm_swiglu_int8_workspace_bytes": (_sz, [ctypes.POINTER(EpGemmShape)]),
    "ep_ll_gemm_swiglu_int8": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 8 + [_sz, _vp, _vp]),
    "ep_debug_ll_gemm_bf16_stall": (_i32, [ctypes.POINTER(EpGemmShape), _i32] + [_vp] * 7 + [_i32] * 3 + [_vp]),
    "ep_debug_ll_gemm_int8_stall": (_i32, [ctypes.POINTER(EpGemmShape)] + [_vp] * 8 + [_sz, _vp] + [_i32] * 3 + [_vp]),
    "ep_sync_status": (_i32, [_vp, _vp]),
    "ep_debug_notify_dispatch_stall": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 16 +
                                       [_sz, _vp, _i32, _i32, _vp]),
    "ep_debug_dispatch_stall": (_i32, [ctypes.POINTER(EpShape)] + [_vp] * 5 + [_i64] + [_vp] * 6 +
                                [_i32, _i32, _vp]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libep_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c \"import "
                               "__graft_entry__ as g; g.build()\"` (needs nvcc)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


# --------------------------------------------------------------------------- helpers
def _current_stream() -> int:
    """Raw handle of torch's current stream on the current device.  The raw getter costs a
    fraction of building a torch.cuda.Stream, which is most of a short call's host time."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream().cuda_stream
    return raw(torch.cuda.current_device())


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _t(t: torch.Tensor | None, dtype, shape, name: str, nullable=False) -> int | None:
    """Device address of a checked tensor (None for a missing one), as ctypes takes it for a
    ``void*``."""
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str) -> int:
    if t.dim() < 1:
        raise ValueError(f"{name} must have a row axis")
    return t.shape[0]


def _check(fn: str, rc: int) -> None:
    if rc != EP_OK:
        raise EpError(fn, rc)


# --------------------------------------------------------------------------- C names
def ep_status_string(status: int) -> str:
    return lib().ep_status_string(status).decode()


def ep_check_shape(shape: EpShape) -> int:
    return lib().ep_check_shape(ctypes.byref(shape))


def ep_num_nodes(shape: EpShape) -> int:
    return lib().ep_num_nodes(ctypes.byref(shape))


def ep_notify_workspace_bytes(shape: EpShape) -> int:
    return int(lib().ep_notify_workspace_bytes(ctypes.byref(shape)))


def ep_get_dispatch_layout(shape: EpShape, topk_idx, num_tokens_per_rank, num_tokens_per_rdma_rank,
                           num_tokens_per_expert, is_token_in_rank, status, stream=None) -> None:
    R, T, K, E, N = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.N
    rc = lib().ep_get_dispatch_layout(
        ctypes.byref(shape), _t(topk_idx, torch.int64, (R, T, K), "topk_idx"),
        _t(num_tokens_per_rank, torch.int32, (R, R), "num_tokens_per_rank"),
        _t(num_tokens_per_rdma_rank, torch.int32, (R, N), "num_tokens_per_rdma_rank"),
        _t(num_tokens_per_expert, torch.int32, (R, E), "num_tokens_per_expert"),
        _t(is_token_in_rank, torch.uint8, (R, T, R), "is_token_in_rank"),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_get_dispatch_layout", rc)


_NOTIFY_OUT = ("rank_prefix_matrix", "gbl_channel_prefix_matrix", "rdma_channel_prefix_matrix",
               "recv_gbl_rank_prefix_sum", "recv_rdma_rank_prefix_sum", "recv_channel_offset",
               "num_recv_tokens", "num_rdma_recv_tokens", "num_recv_tokens_per_expert", "recv_base",
               "send_pos")


def notify_shapes(shape: EpShape) -> dict:
    R, T, C, N, El = shape.num_ranks, shape.num_tokens, shape.num_channels, shape.N, shape.E_loc
    return dict(
        rank_prefix_matrix=((R, R), torch.int32),
        gbl_channel_prefix_matrix=((R, R, C), torch.int32),
        rdma_channel_prefix_matrix=((R, N, C), torch.int32),
        recv_gbl_rank_prefix_sum=((R, R), torch.int32),
        recv_rdma_rank_prefix_sum=((R, N), torch.int32),
        recv_channel_offset=((R, R, C), torch.int32),
        num_recv_tokens=((R,), torch.int32),
        num_rdma_recv_tokens=((R,), torch.int32),
        num_recv_tokens_per_expert=((R, El), torch.int32),
        recv_base=((R + 1,), torch.int64),
        send_pos=((R, T, R), torch.int32),
    )


def _notify_args(shape, is_token_in_rank, num_tokens_per_rank, num_tokens_per_rdma_rank,
                 num_tokens_per_expert, outs: dict):
    R, T, E, N = shape.num_ranks, shape.num_tokens, shape.num_experts, shape.N
    shapes = notify_shapes(shape)
    args = [_t(is_token_in_rank, torch.uint8, (R, T, R), "is_token_in_rank"),
            _t(num_tokens_per_rank, torch.int32, (R, R), "num_tokens_per_rank"),
            _t(num_tokens_per_rdma_rank, torch.int32, (R, N), "num_tokens_per_rdma_rank"),
            _t(num_tokens_per_expert, torch.int32, (R, E), "num_tokens_per_expert")]
    for k in _NOTIFY_OUT:
        shp, dt = shapes[k]
        args.append(_t(outs[k], dt, shp, k))
    return args


def ep_notify_dispatch(shape: EpShape, is_token_in_rank, num_tokens_per_rank,
                       num_tokens_per_rdma_rank, num_tokens_per_expert, outs: dict, workspace,
                       status, host_num_recv_tokens=None, stream=None) -> None:
    """``outs`` maps each notify output name (see :func:`notify_shapes`) to its tensor.
    ``host_num_recv_tokens`` may be a pinned, host-mapped int32 tensor of R+1."""
    args = _notify_args(shape, is_token_in_rank, num_tokens_per_rank, num_tokens_per_rdma_rank,
                        num_tokens_per_expert, outs)
    need = ep_notify_workspace_bytes(shape)
    if workspace is None or not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA tensor of at least {need} bytes")
    host = _vp(None)
    if host_num_recv_tokens is not None:
        if host_num_recv_tokens.dtype != torch.int32 or host_num_recv_tokens.numel() < shape.num_ranks + 1:
            raise ValueError("host_num_recv_tokens must be int32 with R+1 elements")
        host = _vp(host_num_recv_tokens.data_ptr())
    rc = lib().ep_notify_dispatch(ctypes.byref(shape), *args, _vp(workspace.data_ptr()),
                                  _sz(workspace.numel() * workspace.element_size()),
                                  _t(status, torch.int32, (1,), "status"), host, _stream(stream))
    _check("ep_notify_dispatch", rc)


def ep_layout_notify_fused(shape: EpShape) -> int:
    """Which kernel :func:`ep_layout_notify` runs for ``shape`` on the current
    device: 1 = the cluster form, 2 = the tiled form (both one launch)."""
    return int(lib().ep_layout_notify_fused(ctypes.byref(shape)))


def ep_layout_notify_workspace_bytes(shape: EpShape) -> int:
    return int(lib().ep_layout_notify_workspace_bytes(ctypes.byref(shape)))


def _layout_notify_args(shape, topk_idx, layout: dict, outs: dict):
    R, T, K, E, N = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.N
    shapes = notify_shapes(shape)
    args = [_t(topk_idx, torch.int64, (R, T, K), "topk_idx"),
            _t(layout["num_tokens_per_rank"], torch.int32, (R, R), "num_tokens_per_rank"),
            _t(layout["num_tokens_per_rdma_rank"], torch.int32, (R, N), "num_tokens_per_rdma_rank"),
            _t(layout["num_tokens_per_expert"], torch.int32, (R, E), "num_tokens_per_expert"),
            _t(layout["is_token_in_rank"], torch.uint8, (R, T, R), "is_token_in_rank")]
    for k in _NOTIFY_OUT:
        shp, dt = shapes[k]
        args.append(_t(outs[k], dt, shp, k))
    return args


def _host_counts(shape, host_num_recv_tokens) -> _vp:
    if host_num_recv_tokens is None:
        return _vp(None)
    if host_num_recv_tokens.dtype != torch.int32 or host_num_recv_tokens.numel() < shape.num_ranks + 1:
        raise ValueError("host_num_recv_tokens must be int32 with R+1 elements")
    return _vp(host_num_recv_tokens.data_ptr())


def _workspace(workspace, need: int, name="workspace"):
    if workspace is None or not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"{name} must be a CUDA tensor of at least {need} bytes")
    return _vp(workspace.data_ptr()), _sz(workspace.numel() * workspace.element_size())


def ep_layout_notify(shape: EpShape, topk_idx, layout: dict, outs: dict, workspace, status,
                     host_num_recv_tokens=None, stream=None) -> None:
    """Layout and notify in one call.  ``layout`` holds the four layout outputs
    (see :func:`alloc_layout`), ``outs`` the notify outputs (see
    :func:`notify_shapes`); ``workspace`` from :func:`alloc_layout_notify_workspace`."""
    args = _layout_notify_args(shape, topk_idx, layout, outs)
    ws, nws = _workspace(workspace, ep_layout_notify_workspace_bytes(shape))
    rc = lib().ep_layout_notify(ctypes.byref(shape), *args, ws, nws, _t(status, torch.int32, (1,), "status"),
                                _host_counts(shape, host_num_recv_tokens), _stream(stream))
    _check("ep_layout_notify", rc)


def ep_debug_layout_notify_tiled(shape: EpShape, topk_idx, layout: dict, outs: dict, workspace, status,
                                 tile_tokens: int = 0, stall_tile: int = -1, wait_limit_us: int = 1000000,
                                 host_num_recv_tokens=None, stream=None) -> None:
    """Testing hook: :func:`ep_layout_notify` forced onto the tiled form with
    ``tile_tokens`` tokens per tile (0: default) and optionally one tile
    withholding its lookback words."""
    args = _layout_notify_args(shape, topk_idx, layout, outs)
    ws, nws = _workspace(workspace, 0)
    rc = lib().ep_debug_layout_notify_tiled(
        ctypes.byref(shape), *args, ws, nws, _t(status, torch.int32, (1,), "status"),
        _host_counts(shape, host_num_recv_tokens), _i32(tile_tokens), _i32(stall_tile), _i32(wait_limit_us),
        _stream(stream))
    _check("ep_debug_layout_notify_tiled", rc)


def ep_notify_dispatch_noalloc(shape: EpShape, is_token_in_rank, num_tokens_per_rank,
                               num_tokens_per_rdma_rank, num_tokens_per_expert, outs: dict, status,
                               host_num_recv_tokens=None, stream=None) -> None:
    """ep_notify_dispatch using the library's fixed 1 MiB device scratch instead of a
    caller workspace, for callers that cannot allocate device memory.  Calls share
    that scratch, so calls that overlap on the GPU race; ``outs`` needs no
    "workspace" entry."""
    args = _notify_args(shape, is_token_in_rank, num_tokens_per_rank, num_tokens_per_rdma_rank,
                        num_tokens_per_expert, outs)
    host = _vp(None)
    if host_num_recv_tokens is not None:
        if host_num_recv_tokens.dtype != torch.int32 or host_num_recv_tokens.numel() < shape.num_ranks + 1:
            raise ValueError("host_num_recv_tokens must be int32 with R+1 elements")
        host = _vp(host_num_recv_tokens.data_ptr())
    rc = lib().ep_notify_dispatch_noalloc(ctypes.byref(shape), *args,
                                          _t(status, torch.int32, (1,), "status"), host, _stream(stream))
    _check("ep_notify_dispatch_noalloc", rc)


def ep_debug_notify_dispatch_stall(shape: EpShape, is_token_in_rank, num_tokens_per_rank,
                                   num_tokens_per_rdma_rank, num_tokens_per_expert, outs: dict,
                                   workspace, status, stall_block: int, wait_limit_us: int,
                                   stream=None) -> None:
    args = _notify_args(shape, is_token_in_rank, num_tokens_per_rank, num_tokens_per_rdma_rank,
                        num_tokens_per_expert, outs)
    rc = lib().ep_debug_notify_dispatch_stall(
        ctypes.byref(shape), *args, _vp(workspace.data_ptr()),
        _sz(workspace.numel() * workspace.element_size()), _t(status, torch.int32, (1,), "status"),
        _i32(stall_block), _i32(wait_limit_us), _stream(stream))
    _check("ep_debug_notify_dispatch_stall", rc)


def _sched(sched):
    return _t(sched, torch.int64, (1,), "sched", nullable=True)


def _lnd_args(shape, x, topk_idx, topk_w, layout, outs, workspace, disp, sched):
    R, T, K, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.hidden
    ln = _layout_notify_args(shape, topk_idx, layout, outs)
    cap = _rows(disp["recv_x"], "recv_x")
    ws, nws = _workspace(workspace, ep_layout_notify_workspace_bytes(shape))
    return ([ln[0], _t(topk_w, torch.float32, (R, T, K), "topk_w", nullable=True),
             _t(x, torch.bfloat16, (R, T, H), "x")] + ln[1:] +
            [ws, nws, _i64(cap), _t(disp["recv_x"], torch.bfloat16, (cap, H), "recv_x"),
             _t(disp.get("recv_topk_idx"), torch.int64, (cap, K), "recv_topk_idx", nullable=True),
             _t(disp.get("recv_topk_w"), torch.float32, (cap, K), "recv_topk_w", nullable=True),
             _t(disp.get("recv_src_info"), torch.int32, (cap, 2), "recv_src_info", nullable=True)])


def ep_layout_notify_dispatch(shape: EpShape, x, topk_idx, topk_w, layout: dict, outs: dict, workspace,
                              disp: dict, status, sched=None, host_num_recv_tokens=None, stream=None) -> None:
    """Layout, notify and dispatch in one launch.  ``layout``/``outs`` as for
    :func:`ep_layout_notify`, ``disp`` holds the receive arrays (see
    :func:`alloc_dispatch`; recv_topk_idx / recv_topk_w / recv_src_info may be
    missing or None, and topk_w None with them)."""
    args = _lnd_args(shape, x, topk_idx, topk_w, layout, outs, workspace, disp, sched)
    rc = lib().ep_layout_notify_dispatch(ctypes.byref(shape), *args, _t(status, torch.int32, (1,), "status"),
                                         _sched(sched), _host_counts(shape, host_num_recv_tokens), _stream(stream))
    _check("ep_layout_notify_dispatch", rc)


def ep_debug_layout_notify_dispatch_stall(shape: EpShape, x, topk_idx, topk_w, layout: dict, outs: dict,
                                          workspace, disp: dict, status, stall_tile: int, wait_limit_us: int,
                                          sched=None, stream=None) -> None:
    """Testing hook: :func:`ep_layout_notify_dispatch` with one layout + notify
    tile withholding its lookback words and every wait bounded."""
    args = _lnd_args(shape, x, topk_idx, topk_w, layout, outs, workspace, disp, sched)
    rc = lib().ep_debug_layout_notify_dispatch_stall(
        ctypes.byref(shape), *args, _t(status, torch.int32, (1,), "status"), _sched(sched), _i32(stall_tile),
        _i32(wait_limit_us), _stream(stream))
    _check("ep_debug_layout_notify_dispatch_stall", rc)


def ep_dispatch(shape: EpShape, x, topk_idx, topk_w, send_pos, recv_base, recv_x, recv_topk_idx,
                recv_topk_w, recv_src_info, status, stream=None, sched=None) -> None:
    """Cached mode: pass topk_idx, topk_w, recv_topk_idx and recv_topk_w as None
    (and recv_src_info optionally) to reuse an earlier notify handle.  ``sched``: an
    int64 CUDA tensor of one element, zero before the first call (the calls keep it
    zero), for dynamic assignment of row parts to CTAs; None keeps the static split."""
    R, T, K, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.hidden
    cap = _rows(recv_x, "recv_x")
    rc = lib().ep_dispatch(
        ctypes.byref(shape), _t(x, torch.bfloat16, (R, T, H), "x"),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx", nullable=True),
        _t(topk_w, torch.float32, (R, T, K), "topk_w", nullable=True),
        _t(send_pos, torch.int32, (R, T, R), "send_pos"),
        _t(recv_base, torch.int64, (R + 1,), "recv_base"), _i64(cap),
        _t(recv_x, torch.bfloat16, (cap, H), "recv_x"),
        _t(recv_topk_idx, torch.int64, (cap, K), "recv_topk_idx", nullable=True),
        _t(recv_topk_w, torch.float32, (cap, K), "recv_topk_w", nullable=True),
        _t(recv_src_info, torch.int32, (cap, 2), "recv_src_info", nullable=True),
        _t(status, torch.int32, (1,), "status"), _sched(sched), _stream(stream))
    _check("ep_dispatch", rc)


def ep_debug_dispatch_stall(shape: EpShape, x, topk_idx, topk_w, send_pos, recv_base, recv_x, recv_topk_idx,
                            recv_topk_w, recv_src_info, status, stall_cta: int, wait_limit_us: int,
                            stream=None, sched=None) -> None:
    """Testing hook: ep_dispatch with CTA ``stall_cta`` never freeing a ring slot and
    every device wait bounded by ``wait_limit_us``; the status word then reports a
    timeout and the context stays usable."""
    R, T, K, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.hidden
    cap = _rows(recv_x, "recv_x")
    rc = lib().ep_debug_dispatch_stall(
        ctypes.byref(shape), _t(x, torch.bfloat16, (R, T, H), "x"),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(topk_w, torch.float32, (R, T, K), "topk_w"),
        _t(send_pos, torch.int32, (R, T, R), "send_pos"), _t(recv_base, torch.int64, (R + 1,), "recv_base"),
        _i64(cap), _t(recv_x, torch.bfloat16, (cap, H), "recv_x"),
        _t(recv_topk_idx, torch.int64, (cap, K), "recv_topk_idx"),
        _t(recv_topk_w, torch.float32, (cap, K), "recv_topk_w"),
        _t(recv_src_info, torch.int32, (cap, 2), "recv_src_info"), _t(status, torch.int32, (1,), "status"),
        _sched(sched), _i32(stall_cta), _i32(wait_limit_us), _stream(stream))
    _check("ep_debug_dispatch_stall", rc)


def ep_dispatch_fp8(shape: EpShape, x, x_scales, topk_idx, topk_w, send_pos, recv_base, recv_x,
                    recv_x_scales, recv_topk_idx, recv_topk_w, recv_src_info, status, stream=None,
                    sched=None) -> None:
    """FP8 rows (uint8 e4m3 bytes, H per token) plus per-token fp32 scales
    ([..., num_scales]; None for none).  Top-k, source info and ``sched`` as in
    ep_dispatch."""
    R, T, K, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.hidden
    cap = _rows(recv_x, "recv_x")
    S = 0 if x_scales is None else x_scales.shape[-1]
    rc = lib().ep_dispatch_fp8(
        ctypes.byref(shape), _t(x, torch.uint8, (R, T, H), "x"),
        _t(x_scales, torch.float32, (R, T, S), "x_scales", nullable=True), _i32(S),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx", nullable=True),
        _t(topk_w, torch.float32, (R, T, K), "topk_w", nullable=True),
        _t(send_pos, torch.int32, (R, T, R), "send_pos"),
        _t(recv_base, torch.int64, (R + 1,), "recv_base"), _i64(cap),
        _t(recv_x, torch.uint8, (cap, H), "recv_x"),
        _t(recv_x_scales, torch.float32, (cap, S), "recv_x_scales", nullable=True),
        _t(recv_topk_idx, torch.int64, (cap, K), "recv_topk_idx", nullable=True),
        _t(recv_topk_w, torch.float32, (cap, K), "recv_topk_w", nullable=True),
        _t(recv_src_info, torch.int32, (cap, 2), "recv_src_info", nullable=True),
        _t(status, torch.int32, (1,), "status"), _sched(sched), _stream(stream))
    _check("ep_dispatch_fp8", rc)


def ep_combine(shape: EpShape, y, y_w, send_pos, recv_base, combined_x, combined_w, status,
               stream=None) -> None:
    R, T, K, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.hidden
    rows = _rows(y, "y")
    rc = lib().ep_combine(
        ctypes.byref(shape), _t(y, torch.bfloat16, (rows, H), "y"),
        _t(y_w, torch.float32, (rows, K), "y_w", nullable=True), _i64(rows),
        _t(send_pos, torch.int32, (R, T, R), "send_pos"),
        _t(recv_base, torch.int64, (R + 1,), "recv_base"),
        _t(combined_x, torch.bfloat16, (R, T, H), "combined_x"),
        _t(combined_w, torch.float32, (R, T, K), "combined_w", nullable=True),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_combine", rc)


def ep_ll_layout(shape: EpShape, topk_idx, num_tokens_per_expert, expert_capacity: int, slot_pos,
                 layout_range, count, status, stream=None) -> None:
    """Low-latency (per-expert packed) layout: row of each slot in its expert's buffer.
    ``num_tokens_per_expert`` may be None: the kernel then counts for itself (R <= 16)."""
    R, T, K, E = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts
    rc = lib().ep_ll_layout(
        ctypes.byref(shape), _t(topk_idx, torch.int64, (R, T, K), "topk_idx"),
        _t(num_tokens_per_expert, torch.int32, (R, E), "num_tokens_per_expert", nullable=True),
        _i32(expert_capacity),
        _t(slot_pos, torch.int32, (R, T, K), "slot_pos"), _t(layout_range, torch.int32, (E, R, 2), "layout_range"),
        _t(count, torch.int32, (E,), "count"), _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_ll_layout", rc)


def ep_ll_dispatch(shape: EpShape, x, topk_idx, slot_pos, expert_capacity: int, recv_x, recv_src_info,
                   status, stream=None, sched=None) -> None:
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    cap = expert_capacity
    rc = lib().ep_ll_dispatch(
        ctypes.byref(shape), _t(x, torch.bfloat16, (R, T, H), "x"),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(slot_pos, torch.int32, (R, T, K), "slot_pos"),
        _i32(cap), _t(recv_x, torch.bfloat16, (E, cap, H), "recv_x"),
        _t(recv_src_info, torch.int32, (E, cap, 2), "recv_src_info", nullable=True),
        _t(status, torch.int32, (1,), "status"), _sched(sched), _stream(stream))
    _check("ep_ll_dispatch", rc)


def ep_ll_combine(shape: EpShape, y, expert_capacity: int, topk_idx, topk_w, slot_pos, combined_x, status,
                  stream=None) -> None:
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    cap = expert_capacity
    rc = lib().ep_ll_combine(
        ctypes.byref(shape), _t(y, torch.bfloat16, (E, cap, H), "y"), _i32(cap),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(topk_w, torch.float32, (R, T, K), "topk_w"),
        _t(slot_pos, torch.int32, (R, T, K), "slot_pos"), _t(combined_x, torch.bfloat16, (R, T, H), "combined_x"),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_ll_combine", rc)


def ep_check_route(shape: EpShape, route: EpRoute) -> int:
    return lib().ep_check_route(ctypes.byref(shape), ctypes.byref(route))


def _logits(logits, shape: EpShape, name="logits"):
    if logits is not None and logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    dtype = torch.float32 if logits is None else logits.dtype
    return _t(logits, dtype, (shape.num_ranks, shape.num_tokens, shape.num_experts), name), dtype


def ep_route(shape: EpShape, route: EpRoute, logits, bias, topk_idx, topk_w, status, stream=None) -> None:
    """Router: ``logits`` [R, T, E] (fp32 or bf16) to the top-k map and weights the other
    calls take; ``bias`` [E] fp32 (or None) is added to the scores for the selection only."""
    R, T, K, E = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts
    lp, dtype = _logits(logits, shape)
    rc = lib().ep_route(
        ctypes.byref(shape), ctypes.byref(route), lp, _i32(int(dtype == torch.bfloat16)),
        _t(bias, torch.float32, (E,), "bias", nullable=True), _t(topk_idx, torch.int64, (R, T, K), "topk_idx"),
        _t(topk_w, torch.float32, (R, T, K), "topk_w"), _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_route", rc)


def ep_route_backward(shape: EpShape, route: EpRoute, logits, topk_idx, grad_topk_w, grad_logits, status,
                      stream=None) -> None:
    """Gradient of :func:`ep_route`'s weights with respect to the logits
    (``grad_logits`` has the logits' type; every element is written)."""
    R, T, K = shape.num_ranks, shape.num_tokens, shape.num_topk
    lp, dtype = _logits(logits, shape)
    rc = lib().ep_route_backward(
        ctypes.byref(shape), ctypes.byref(route), lp, _i32(int(dtype == torch.bfloat16)),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(grad_topk_w, torch.float32, (R, T, K), "grad_topk_w"),
        _t(grad_logits, dtype, (R, T, shape.num_experts), "grad_logits"), _t(status, torch.int32, (1,), "status"),
        _stream(stream))
    _check("ep_route_backward", rc)


def ep_ll_dispatch_fp8(shape: EpShape, x, topk_idx, slot_pos, expert_capacity: int, recv_x, recv_x_scales,
                       recv_src_info, status, stream=None) -> None:
    """:func:`ep_ll_dispatch` with the rows cast to e4m3 (uint8 bytes), one fp32 scale per
    128 columns ([E, capacity, ceil(H / 128)])."""
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    cap = expert_capacity
    rc = lib().ep_ll_dispatch_fp8(
        ctypes.byref(shape), _t(x, torch.bfloat16, (R, T, H), "x"),
        _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(slot_pos, torch.int32, (R, T, K), "slot_pos"),
        _i32(cap), _t(recv_x, torch.uint8, (E, cap, H), "recv_x"),
        _t(recv_x_scales, torch.float32, (E, cap, scale_blocks(H)), "recv_x_scales"),
        _t(recv_src_info, torch.int32, (E, cap, 2), "recv_src_info", nullable=True),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_ll_dispatch_fp8", rc)


def scale_blocks(n: int) -> int:
    """Scales of ``n`` columns: one per 128."""
    return -(-n // 128)


def ep_check_gemm_shape(shape: EpGemmShape) -> int:
    return lib().ep_check_gemm_shape(ctypes.byref(shape))


def _gemm_dims(a, w, w_dims: int):
    for t, dims, name in ((a, 3, "a"), (w, w_dims, "w")):
        if t is None or t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions")
    return a.shape[0], a.shape[1], w.shape[-2], a.shape[2]


def ep_ll_gemm_fp8(a, a_scales, w, w_scales, count, y, status, stream=None) -> None:
    """Experts' product: ``a`` [E, capacity, k] and ``w`` [E, n, k] e4m3 (uint8 bytes) with
    their 128-column and 128 x 128 block scales, ``count`` [E] rows per expert ->
    ``y`` [E, capacity, n] bf16."""
    E, cap, n, k = _gemm_dims(a, w, 3)
    rc = lib().ep_ll_gemm_fp8(
        ctypes.byref(EpGemmShape(E, cap, n, k)), _t(a, torch.uint8, (E, cap, k), "a"),
        _t(a_scales, torch.float32, (E, cap, scale_blocks(k)), "a_scales"), _t(w, torch.uint8, (E, n, k), "w"),
        _t(w_scales, torch.float32, (E, scale_blocks(n), scale_blocks(k)), "w_scales"),
        _t(count, torch.int32, (E,), "count"), _t(y, torch.bfloat16, (E, cap, n), "y"),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_ll_gemm_fp8", rc)


def ep_ll_gemm_swiglu_fp8(a, a_scales, w, w_scales, count, y, y_scales, status, stream=None) -> None:
    """Gate and up products, silu(gate) * up and its cast in one launch: ``w`` [E, 2, n, k]
    (gate, up) -> ``y`` [E, capacity, n] e4m3 (uint8 bytes), ``y_scales`` per 128 columns."""
    E, cap, n, k = _gemm_dims(a, w, 4)
    rc = lib().ep_ll_gemm_swiglu_fp8(
        ctypes.byref(EpGemmShape(E, cap, n, k)), _t(a, torch.uint8, (E, cap, k), "a"),
        _t(a_scales, torch.float32, (E, cap, scale_blocks(k)), "a_scales"), _t(w, torch.uint8, (E, 2, n, k), "w"),
        _t(w_scales, torch.float32, (E, 2, scale_blocks(n), scale_blocks(k)), "w_scales"),
        _t(count, torch.int32, (E,), "count"), _t(y, torch.uint8, (E, cap, n), "y"),
        _t(y_scales, torch.float32, (E, cap, scale_blocks(n)), "y_scales"),
        _t(status, torch.int32, (1,), "status"), _stream(stream))
    _check("ep_ll_gemm_swiglu_fp8", rc)


def ep_debug_ll_gemm_fp8_stall(a, a_scales, w, w_scales, count, y, y_scales, status, stall_cta: int, stall_tile: int,
                               wait_limit_us: int, stream=None) -> None:
    """Testing hook: :func:`ep_ll_gemm_swiglu_fp8` (:func:`ep_ll_gemm_fp8` where ``y_scales`` is None) with
    one CTA or pair of CTAs fed no products from its tile ``stall_tile`` on and every device wait
    bounded by ``wait_limit_us``; the status word then reports a timeout and the context stays usable."""
    gated = y_scales is not None
    E, cap, n, k = _gemm_dims(a, w, 4 if gated else 3)
    nb, kb, two = scale_blocks(n), scale_blocks(k), (2,) if gated else ()
    rc = lib().ep_debug_ll_gemm_fp8_stall(
        ctypes.byref(EpGemmShape(E, cap, n, k)), _t(a, torch.uint8, (E, cap, k), "a"),
        _t(a_scales, torch.float32, (E, cap, kb), "a_scales"), _t(w, torch.uint8, (E, *two, n, k), "w"),
        _t(w_scales, torch.float32, (E, *two, nb, kb), "w_scales"), _t(count, torch.int32, (E,), "count"),
        _t(y, torch.uint8 if gated else torch.bfloat16, (E, cap, n), "y"),
        _t(y_scales, torch.float32, (E, cap, nb), "y_scales", nullable=True), _t(status, torch.int32, (1,), "status"),
        _i32(stall_cta), _i32(stall_tile), _i32(wait_limit_us), _stream(stream))
    _check("ep_debug_ll_gemm_fp8_stall", rc)


def _here(status, *tensors) -> None:
    """Refuses tensors of another device than the current one, whose stream the call runs on."""
    device = torch.cuda.current_device()
    for t in (status, *tensors):
        if t is not None and t.is_cuda and t.get_device() != device:
            raise ValueError(f"tensors must be on the current device (cuda:{device}), got {t.device}")


def ep_ll_combine_backward(shape: EpShape, grad_combined, y, expert_capacity: int, topk_idx, topk_w, slot_pos, grad_y,
                           grad_topk_w, status, stream=None) -> None:
    """Gradient of :func:`ep_ll_combine`: ``grad_combined`` [R, T, H] bf16 and the expert outputs
    ``y`` -> ``grad_y`` [E, capacity, H] bf16 (rows without a slot are left as they are) and
    ``grad_topk_w`` [R, T, K] fp32 (every element written)."""
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    cap = expert_capacity
    args = (_t(grad_combined, torch.bfloat16, (R, T, H), "grad_combined"), _t(y, torch.bfloat16, (E, cap, H), "y"),
            _i32(cap), _t(topk_idx, torch.int64, (R, T, K), "topk_idx"), _t(topk_w, torch.float32, (R, T, K), "topk_w"),
            _t(slot_pos, torch.int32, (R, T, K), "slot_pos"), _t(grad_y, torch.bfloat16, (E, cap, H), "grad_y"),
            _t(grad_topk_w, torch.float32, (R, T, K), "grad_topk_w"), _t(status, torch.int32, (1,), "status"))
    _here(status, grad_combined, y, topk_idx, topk_w, slot_pos, grad_y, grad_topk_w)
    _check("ep_ll_combine_backward", lib().ep_ll_combine_backward(ctypes.byref(shape), *args, _stream(stream)))


def ep_check_gemm_shape_bf16(shape: EpGemmShape) -> int:
    return lib().ep_check_gemm_shape_bf16(ctypes.byref(shape))


def ep_ll_gemm_bf16(a, w, count, y, status, stream=None) -> None:
    """Experts' product in bf16: ``a`` [E, capacity, k] and ``w`` [E, n, k] with ``count`` [E]
    rows per expert -> ``y`` [E, capacity, n]."""
    E, cap, n, k = _gemm_dims(a, w, 3)
    bf16 = torch.bfloat16
    args = (_t(a, bf16, (E, cap, k), "a"), _t(w, bf16, (E, n, k), "w"), _t(count, torch.int32, (E,), "count"),
            _t(y, bf16, (E, cap, n), "y"), _t(status, torch.int32, (1,), "status"))
    _here(status, a, w, count, y)
    _check("ep_ll_gemm_bf16", lib().ep_ll_gemm_bf16(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_ll_gemm_swiglu_bf16(a, w, count, y, gate_up, status, stream=None) -> None:
    """Gate and up products and silu(gate) * up in one launch: ``w`` [E, 2, n, k] (gate, up) ->
    ``y`` [E, capacity, n] bf16, and where ``gate_up`` [E, capacity, 2, n] is given (not None)
    both products, which the gradient starts from."""
    E, cap, n, k = _gemm_dims(a, w, 4)
    bf16 = torch.bfloat16
    args = (_t(a, bf16, (E, cap, k), "a"), _t(w, bf16, (E, 2, n, k), "w"), _t(count, torch.int32, (E,), "count"),
            _t(y, bf16, (E, cap, n), "y"), _t(gate_up, bf16, (E, cap, 2, n), "gate_up", nullable=True),
            _t(status, torch.int32, (1,), "status"))
    _here(status, a, w, count, y, gate_up)
    _check("ep_ll_gemm_swiglu_bf16",
           lib().ep_ll_gemm_swiglu_bf16(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def _grad_dims(grad_y, w):
    for t, name in ((grad_y, "grad_y"), (w, "w")):
        if t is None or t.dim() != 3:
            raise ValueError(f"{name} must have 3 dimensions")
    return grad_y.shape[0], grad_y.shape[1], grad_y.shape[2], w.shape[2]


def ep_ll_gemm_dgrad_bf16(grad_y, w, count, grad_a, status, stream=None) -> None:
    """Gradient of a product's rows: ``grad_y`` [E, capacity, n] and ``w`` [E, n, k] ->
    ``grad_a`` [E, capacity, k] (the gated product's: ``grad_gate_up`` and ``w`` viewed with 2 n)."""
    E, cap, n, k = _grad_dims(grad_y, w)
    bf16 = torch.bfloat16
    args = (_t(grad_y, bf16, (E, cap, n), "grad_y"), _t(w, bf16, (E, n, k), "w"), _t(count, torch.int32, (E,), "count"),
            _t(grad_a, bf16, (E, cap, k), "grad_a"), _t(status, torch.int32, (1,), "status"))
    _here(status, grad_y, w, count, grad_a)
    _check("ep_ll_gemm_dgrad_bf16",
           lib().ep_ll_gemm_dgrad_bf16(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_ll_gemm_dswiglu_bf16(grad_y, w, gate_up, count, grad_gate_up, status, stream=None) -> None:
    """Gradient of the last product's rows carried through the gated activation: ``grad_y``
    [E, capacity, n], ``w`` [E, n, k] and the kept ``gate_up`` [E, capacity, 2, k] ->
    ``grad_gate_up`` [E, capacity, 2, k]."""
    E, cap, n, k = _grad_dims(grad_y, w)
    bf16 = torch.bfloat16
    args = (_t(grad_y, bf16, (E, cap, n), "grad_y"), _t(w, bf16, (E, n, k), "w"),
            _t(gate_up, bf16, (E, cap, 2, k), "gate_up"), _t(count, torch.int32, (E,), "count"),
            _t(grad_gate_up, bf16, (E, cap, 2, k), "grad_gate_up"), _t(status, torch.int32, (1,), "status"))
    _here(status, grad_y, w, gate_up, count, grad_gate_up)
    _check("ep_ll_gemm_dswiglu_bf16",
           lib().ep_ll_gemm_dswiglu_bf16(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_ll_gemm_wgrad_bf16(grad_y, a, count, grad_w, status, stream=None) -> None:
    """Gradient of a product's weights: ``grad_y`` [E, capacity, n] and ``a`` [E, capacity, k] ->
    ``grad_w`` [E, n, k], fp32 or bf16, every element written."""
    E, cap, n, k = _grad_dims(grad_y, a)
    if grad_w is not None and grad_w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"grad_w must be torch.float32 or torch.bfloat16, got {grad_w.dtype}")
    gt = torch.float32 if grad_w is None else grad_w.dtype
    args = (_t(grad_y, torch.bfloat16, (E, cap, n), "grad_y"), _t(a, torch.bfloat16, (E, cap, k), "a"),
            _t(count, torch.int32, (E,), "count"), _t(grad_w, gt, (E, n, k), "grad_w"), _i32(int(gt == torch.bfloat16)),
            _t(status, torch.int32, (1,), "status"))
    _here(status, grad_y, a, count, grad_w)
    _check("ep_ll_gemm_wgrad_bf16",
           lib().ep_ll_gemm_wgrad_bf16(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_ll_dispatch_int8(shape: EpShape, x, topk_idx, slot_pos, expert_capacity: int, recv_x, recv_x_scales,
                        recv_src_info, status, stream=None) -> None:
    """:func:`ep_ll_dispatch` with the rows cast to int8, one fp32 scale per row ([E, capacity])."""
    R, T, K, E, H = shape.num_ranks, shape.num_tokens, shape.num_topk, shape.num_experts, shape.hidden
    cap = expert_capacity
    args = (_t(x, torch.bfloat16, (R, T, H), "x"), _t(topk_idx, torch.int64, (R, T, K), "topk_idx"),
            _t(slot_pos, torch.int32, (R, T, K), "slot_pos"), _i32(cap), _t(recv_x, torch.int8, (E, cap, H), "recv_x"),
            _t(recv_x_scales, torch.float32, (E, cap), "recv_x_scales"),
            _t(recv_src_info, torch.int32, (E, cap, 2), "recv_src_info", nullable=True),
            _t(status, torch.int32, (1,), "status"))
    _here(status, x, topk_idx, slot_pos, recv_x, recv_x_scales, recv_src_info)
    _check("ep_ll_dispatch_int8", lib().ep_ll_dispatch_int8(ctypes.byref(shape), *args, _stream(stream)))


def ep_ll_gemm_int8(a, a_scales, w, w_scales, count, y, status, stream=None) -> None:
    """Experts' product in int8: ``a`` [E, capacity, k] with a scale per row ([E, capacity]), ``w``
    [E, n, k] with a scale per output column ([E, n]), ``count`` [E] -> ``y`` [E, capacity, n] bf16."""
    E, cap, n, k = _gemm_dims(a, w, 3)
    args = (_t(a, torch.int8, (E, cap, k), "a"), _t(a_scales, torch.float32, (E, cap), "a_scales"),
            _t(w, torch.int8, (E, n, k), "w"), _t(w_scales, torch.float32, (E, n), "w_scales"),
            _t(count, torch.int32, (E,), "count"), _t(y, torch.bfloat16, (E, cap, n), "y"),
            _t(status, torch.int32, (1,), "status"))
    _here(status, a, a_scales, w, w_scales, count, y)
    _check("ep_ll_gemm_int8", lib().ep_ll_gemm_int8(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_ll_gemm_swiglu_int8_workspace_bytes(shape: EpGemmShape) -> int:
    return int(lib().ep_ll_gemm_swiglu_int8_workspace_bytes(ctypes.byref(shape)))


def ep_ll_gemm_swiglu_int8(a, a_scales, w, w_scales, count, y, y_scales, workspace, status, stream=None) -> None:
    """Gate and up products in int8, silu(gate) * up and its cast by rows: ``w`` [E, 2, n, k] with
    ``w_scales`` [E, 2, n] -> ``y`` [E, capacity, n] int8, ``y_scales`` [E, capacity]; ``workspace``
    of :func:`ep_ll_gemm_swiglu_int8_workspace_bytes` bytes."""
    E, cap, n, k = _gemm_dims(a, w, 4)
    shape = EpGemmShape(E, cap, n, k)
    args = (_t(a, torch.int8, (E, cap, k), "a"), _t(a_scales, torch.float32, (E, cap), "a_scales"),
            _t(w, torch.int8, (E, 2, n, k), "w"), _t(w_scales, torch.float32, (E, 2, n), "w_scales"),
            _t(count, torch.int32, (E,), "count"), _t(y, torch.int8, (E, cap, n), "y"),
            _t(y_scales, torch.float32, (E, cap), "y_scales"))
    ws, nws = _workspace(workspace, ep_ll_gemm_swiglu_int8_workspace_bytes(shape))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _here(status, a, a_scales, w, w_scales, count, y, y_scales, workspace)
    _check("ep_ll_gemm_swiglu_int8",
           lib().ep_ll_gemm_swiglu_int8(ctypes.byref(shape), *args, ws, nws, _t(status, torch.int32, (1,), "status"),
                                        _stream(stream)))


def ep_debug_ll_gemm_bf16_stall(form: int, n: int, k: int, rows, other, gate_up, count, out, gate_up_out, status,
                                stall_pair: int, stall_tile: int, wait_limit_us: int, stream=None) -> None:
    """Testing hook: the bf16 product of ``form`` (0 plain, 1 gated, 2 rows' gradient, 3 gradient
    through the activation, 4 and 5 weights' gradient in fp32 and bf16) of weights [n, k] with one
    pair of CTAs fed no products from its tile ``stall_tile`` on and every device wait bounded by
    ``wait_limit_us``; the status word then reports a timeout and the context stays usable."""
    bf16 = torch.bfloat16
    E, cap = rows.shape[:2]
    wgrad, halves = form in (4, 5), form == 3
    out_dim = {0: n, 1: n, 2: k, 3: k}.get(form)
    other_shape = (E, cap, k) if wgrad else (E, 2, n, k) if form == 1 else (E, n, k)
    out_shape = (E, n, k) if wgrad else (E, cap, 2, out_dim) if halves else (E, cap, out_dim)
    args = (_i32(form), _t(rows, bf16, (E, cap, k if form < 2 else n), "rows"), _t(other, bf16, other_shape, "other"),
            _t(gate_up, bf16, (E, cap, 2, k), "gate_up", nullable=not halves), _t(count, torch.int32, (E,), "count"),
            _t(out, torch.float32 if form == 4 else bf16, out_shape, "out"),
            _t(gate_up_out, bf16, (E, cap, 2, n), "gate_up_out", nullable=True), _t(status, torch.int32, (1,), "status"),
            _i32(stall_pair), _i32(stall_tile), _i32(wait_limit_us))
    _check("ep_debug_ll_gemm_bf16_stall",
           lib().ep_debug_ll_gemm_bf16_stall(ctypes.byref(EpGemmShape(E, cap, n, k)), *args, _stream(stream)))


def ep_debug_ll_gemm_int8_stall(a, a_scales, w, w_scales, count, y, y_scales, workspace, status, stall_pair: int,
                                stall_tile: int, wait_limit_us: int, stream=None) -> None:
    """Testing hook: :func:`ep_ll_gemm_swiglu_int8` (:func:`ep_ll_gemm_int8` where ``y_scales`` is
    None) stalled as in :func:`ep_debug_ll_gemm_bf16_stall`."""
    gated = y_scales is not None
    E, cap, n, k = _gemm_dims(a, w, 4 if gated else 3)
    two = (2,) if gated else ()
    shape = EpGemmShape(E, cap, n, k)
    ws, nws = _workspace(workspace, ep_ll_gemm_swiglu_int8_workspace_bytes(shape)) if gated else (None, _sz(0))
    rc = lib().ep_debug_ll_gemm_int8_stall(
        ctypes.byref(shape), _t(a, torch.int8, (E, cap, k), "a"), _t(a_scales, torch.float32, (E, cap), "a_scales"),
        _t(w, torch.int8, (E, *two, n, k), "w"), _t(w_scales, torch.float32, (E, *two, n), "w_scales"),
        _t(count, torch.int32, (E,), "count"), _t(y, torch.int8 if gated else torch.bfloat16, (E, cap, n), "y"),
        _t(y_scales, torch.float32, (E, cap), "y_scales", nullable=True), ws, nws, _t(status, torch.int32, (1,), "status"),
        _i32(stall_pair), _i32(stall_tile), _i32(wait_limit_us), _stream(stream))
    _check("ep_debug_ll_gemm_int8_stall", rc)


def ep_sync_status(status, stream=None) -> int:
    """Wait for the stream and return the status code the device word maps to."""
    return int(lib().ep_sync_status(_t(status, torch.int32, (1,), "status"), _stream(stream)))


# --------------------------------------------------------------------------- allocation
def alloc_layout(shape: EpShape, device="cuda") -> dict:
    R, T, E, N = shape.num_ranks, shape.num_tokens, shape.num_experts, shape.N
    z = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device=device)  # noqa: E731
    return dict(num_tokens_per_rank=z(R, R), num_tokens_per_rdma_rank=z(R, N),
                num_tokens_per_expert=z(R, E), is_token_in_rank=z(R, T, R, dt=torch.uint8))


def alloc_notify(shape: EpShape, device="cuda") -> dict:
    outs = {k: torch.empty(s, dtype=dt, device=device) for k, (s, dt) in notify_shapes(shape).items()}
    ws = ep_notify_workspace_bytes(shape)
    # zeroed once here; every notify call leaves it ready for the next one
    outs["workspace"] = torch.zeros((ws + 15) // 16 * 16, dtype=torch.uint8, device=device)
    return outs


def alloc_layout_notify_workspace(shape: EpShape, device="cuda", nbytes: int | None = None) -> torch.Tensor:
    """Zeroed workspace for :func:`ep_layout_notify` (every call leaves it ready
    for the next one); ``nbytes`` overrides the size (e.g. for several shapes)."""
    n = ep_layout_notify_workspace_bytes(shape) if nbytes is None else nbytes
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def alloc_dispatch(shape: EpShape, capacity_rows: int, device="cuda") -> dict:
    H, K = shape.hidden, shape.num_topk
    return dict(recv_x=torch.empty(capacity_rows, H, dtype=torch.bfloat16, device=device),
                recv_topk_idx=torch.empty(capacity_rows, K, dtype=torch.int64, device=device),
                recv_topk_w=torch.empty(capacity_rows, K, dtype=torch.float32, device=device),
                recv_src_info=torch.empty(capacity_rows, 2, dtype=torch.int32, device=device))


def alloc_combine(shape: EpShape, device="cuda") -> dict:
    R, T, H, K = shape.num_ranks, shape.num_tokens, shape.hidden, shape.num_topk
    return dict(combined_x=torch.empty(R, T, H, dtype=torch.bfloat16, device=device),
                combined_w=torch.empty(R, T, K, dtype=torch.float32, device=device))


@dataclass
class Pipeline:
    """Buffers for one shape plus the four steps in order (identity expert by
    default).  Allocates once; :meth:`run` launches layout + notify (one call,
    :func:`ep_layout_notify`), dispatch and combine on the current stream
    without synchronising."""

    shape: EpShape
    capacity_rows: int
    device: str = "cuda"

    def __post_init__(self):
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        # dispatch's unit counter: zeroed once here, every call leaves it zero
        self.sched = torch.zeros(1, dtype=torch.int64, device=self.device)
        self.layout = alloc_layout(self.shape, self.device)
        self.notify = alloc_notify(self.shape, self.device)
        self.ln_workspace = alloc_layout_notify_workspace(self.shape, self.device)
        self.dispatch = alloc_dispatch(self.shape, self.capacity_rows, self.device)
        self.combine = alloc_combine(self.shape, self.device)

    def run(self, x, topk_idx, topk_w, y=None, y_w=None, stream=None, host_num_recv_tokens=None):
        sh, L, Nt, D, C = self.shape, self.layout, self.notify, self.dispatch, self.combine
        ep_layout_notify(sh, topk_idx, L, Nt, self.ln_workspace, self.status, host_num_recv_tokens, stream)
        ep_dispatch(sh, x, topk_idx, topk_w, Nt["send_pos"], Nt["recv_base"], D["recv_x"],
                    D["recv_topk_idx"], D["recv_topk_w"], D["recv_src_info"], self.status, stream, self.sched)
        ep_combine(sh, D["recv_x"] if y is None else y, D["recv_topk_w"] if y_w is None else y_w,
                   Nt["send_pos"], Nt["recv_base"], C["combined_x"], C["combined_w"], self.status,
                   stream)
        return C["combined_x"], C["combined_w"]

    def run_cached(self, x, y=None, stream=None):
        """Cached mode: dispatch and combine only, reusing the handle (send_pos,
        recv_base) of the last :meth:`run`; the top-k is not dispatched and the
        combined weights are not produced."""
        sh, Nt, D, C = self.shape, self.notify, self.dispatch, self.combine
        ep_dispatch(sh, x, None, None, Nt["send_pos"], Nt["recv_base"], D["recv_x"], None, None, None,
                    self.status, stream, self.sched)
        ep_combine(sh, D["recv_x"] if y is None else y, None, Nt["send_pos"], Nt["recv_base"],
                   C["combined_x"], None, self.status, stream)
        return C["combined_x"]


def cast_weight_blocks(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Weights [..., n, k] as the experts' products take them: e4m3 bytes (uint8) and one
    fp32 scale per 128 x 128 block ([..., ceil(n / 128), ceil(k / 128)]), the block's largest
    magnitude over 448.  Plain torch, for use once when weights are loaded."""
    n, k = w.shape[-2:]
    nb, kb = scale_blocks(n), scale_blocks(k)
    blocks = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n))
    blocks = blocks.unflatten(-1, (kb, 128)).unflatten(-3, (nb, 128))
    scales = (blocks.abs().amax((-3, -1)).clamp(min=2.0 ** -100) / 448.0).contiguous()
    q = (blocks / scales.unsqueeze(-1).unsqueeze(-3)).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-4, -3).flatten(-2)[..., :n, :k].contiguous(), scales


def cast_weight_channels(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Weights [..., n, k] as the experts' int8 products take them: int8 and one fp32 scale per
    output column ([..., n]), the row's largest magnitude by 1 / 127.  Plain torch, for use once
    when weights are loaded."""
    w = w.float()
    scales = (w.abs().amax(-1).clamp(min=2.0 ** -100) * (1.0 / 127.0)).contiguous()
    return torch.round(w / scales.unsqueeze(-1)).to(torch.int8).contiguous(), scales


def _route_and_place(layer, logits, bias, stream) -> None:
    """Router and low-latency layout of a layer: fills its topk_idx, topk_w, slot_pos,
    layout_range and count."""
    sh = layer.shape
    ep_route(sh, layer.route, logits, bias, layer.topk_idx, layer.topk_w, layer.status, stream)
    counts = None
    if layer.layout is not None:
        L = layer.layout
        ep_get_dispatch_layout(sh, layer.topk_idx, L["num_tokens_per_rank"], L["num_tokens_per_rdma_rank"],
                               L["num_tokens_per_expert"], L["is_token_in_rank"], layer.status, stream)
        counts = L["num_tokens_per_expert"]
    ep_ll_layout(sh, layer.topk_idx, counts, layer.expert_capacity, layer.slot_pos, layer.layout_range, layer.count,
                 layer.status, stream)


@dataclass
class MoELayer:
    """A mixture-of-experts layer on the low-latency layout: router, layout, casting
    dispatch, gated e4m3 or int8 experts, weighted combine.  Owns every buffer; :meth:`run`
    launches the calls on the current stream without synchronising.

    ``ffn`` is the experts' inner size; ``expert_capacity`` bounds the rows of an expert
    (slots beyond it are dropped and reported as EP_ERR_CAPACITY).  ``weights`` is "fp8" (e4m3
    with 128 x 128 block scales) or "int8" (a scale for each token and output column)."""

    shape: EpShape
    route: EpRoute
    ffn: int
    expert_capacity: int
    device: str = "cuda"
    weights: str = "fp8"

    def __post_init__(self):
        if self.weights not in ("fp8", "int8"):
            raise ValueError(f"weights must be 'fp8' or 'int8', got {self.weights!r}")
        sh, cap, F, dev = self.shape, self.expert_capacity, self.ffn, self.device
        R, T, K, E, H = sh.num_ranks, sh.num_tokens, sh.num_topk, sh.num_experts, sh.hidden
        z = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.topk_idx, self.topk_w = z(R, T, K, dt=torch.int64), z(R, T, K, dt=torch.float32)
        # the layout counts for itself where one cluster of R CTAs can; else the counts come from the layout step
        self.layout = None if R <= 16 and R * E <= 16384 else alloc_layout(sh, dev)
        self.slot_pos, self.layout_range, self.count = z(R, T, K), z(E, R, 2), z(E)
        if self.weights == "int8":
            self.rows, self.row_scales = z(E, cap, H, dt=torch.int8), z(E, cap, dt=torch.float32)
            self.inner, self.inner_scales = z(E, cap, F, dt=torch.int8), z(E, cap, dt=torch.float32)
            self.workspace = z(ep_ll_gemm_swiglu_int8_workspace_bytes(EpGemmShape(E, cap, F, H)), dt=torch.uint8)
        else:
            self.rows = z(E, cap, H, dt=torch.uint8)
            self.row_scales = z(E, cap, scale_blocks(H), dt=torch.float32)
            self.inner = z(E, cap, F, dt=torch.uint8)
            self.inner_scales = z(E, cap, scale_blocks(F), dt=torch.float32)
        self.y = z(E, cap, H, dt=torch.bfloat16)
        self.combined_x = z(R, T, H, dt=torch.bfloat16)

    def run(self, x, logits, bias, w13, w13_scales, w2, w2_scales, stream=None):
        """``x`` [R, T, H] bf16 and router ``logits`` [R, T, E] -> combined_x [R, T, H] bf16.
        Weights as :func:`cast_weight_blocks` (int8: :func:`cast_weight_channels`) makes them:
        ``w13`` [E, 2, ffn, H] (gate, up) and ``w2`` [E, H, ffn]; ``bias`` [E] of the selection, or None."""
        sh, cap = self.shape, self.expert_capacity
        _route_and_place(self, logits, bias, stream)
        if self.weights == "int8":
            ep_ll_dispatch_int8(sh, x, self.topk_idx, self.slot_pos, cap, self.rows, self.row_scales, None, self.status,
                                stream)
            ep_ll_gemm_swiglu_int8(self.rows, self.row_scales, w13, w13_scales, self.count, self.inner,
                                   self.inner_scales, self.workspace, self.status, stream)
            ep_ll_gemm_int8(self.inner, self.inner_scales, w2, w2_scales, self.count, self.y, self.status, stream)
        else:
            ep_ll_dispatch_fp8(sh, x, self.topk_idx, self.slot_pos, cap, self.rows, self.row_scales, None, self.status,
                               stream)
            ep_ll_gemm_swiglu_fp8(self.rows, self.row_scales, w13, w13_scales, self.count, self.inner,
                                  self.inner_scales, self.status, stream)
            ep_ll_gemm_fp8(self.inner, self.inner_scales, w2, w2_scales, self.count, self.y, self.status, stream)
        ep_ll_combine(sh, self.y, cap, self.topk_idx, self.topk_w, self.slot_pos, self.combined_x, self.status, stream)
        return self.combined_x


@dataclass
class MoETrainLayer:
    """A mixture-of-experts layer that trains, on the low-latency layout in bf16: router, layout,
    dispatch, gated experts, weighted combine, and in :meth:`backward` all of their gradients.
    Owns every buffer; both methods launch their calls on the current stream without
    synchronising, and either can be captured in a CUDA graph.

    ``ffn`` is the experts' inner size; ``expert_capacity`` bounds the rows of an expert
    (slots beyond it are dropped and reported as EP_ERR_CAPACITY; they have no gradient).
    :meth:`backward` reads what the last :meth:`run` left in the buffers."""

    shape: EpShape
    route: EpRoute
    ffn: int
    expert_capacity: int
    device: str = "cuda"

    def __post_init__(self):
        sh, cap, F, dev = self.shape, self.expert_capacity, self.ffn, self.device
        R, T, K, E, H = sh.num_ranks, sh.num_tokens, sh.num_topk, sh.num_experts, sh.hidden
        z = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=dev)  # noqa: E731
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        # dispatch's unit counter: zeroed once here, every call leaves it zero
        self.sched = torch.zeros(1, dtype=torch.int64, device=dev)
        self.topk_idx, self.topk_w = z(R, T, K, dt=torch.int64), z(R, T, K, dt=torch.float32)
        # the layout counts for itself where one cluster of R CTAs can; else the counts come from the layout step
        self.layout = None if R <= 16 and R * E <= 16384 else alloc_layout(sh, dev)
        self.slot_pos, self.layout_range = z(R, T, K, dt=torch.int32), z(E, R, 2, dt=torch.int32)
        self.count = z(E, dt=torch.int32)
        self.rows, self.gate_up, self.inner = z(E, cap, H), z(E, cap, 2, F), z(E, cap, F)
        self.y, self.combined_x = z(E, cap, H), z(R, T, H)
        self.grad_y, self.grad_topk_w = z(E, cap, H), z(R, T, K, dt=torch.float32)
        self.grad_gate_up, self.grad_rows, self.grad_x = z(E, cap, 2, F), z(E, cap, H), z(R, T, H)
        self.ones = torch.ones(R, T, K, device=dev)  # the dispatch's gradient is a combine with these weights

    def run(self, x, logits, bias, w13, w2, stream=None):
        """``x`` [R, T, H] bf16 and router ``logits`` [R, T, E] -> combined_x [R, T, H] bf16, with
        ``w13`` [E, 2, ffn, H] (gate, up) and ``w2`` [E, H, ffn] bf16; ``bias`` [E] of the
        selection, or None."""
        sh, cap = self.shape, self.expert_capacity
        _route_and_place(self, logits, bias, stream)
        ep_ll_dispatch(sh, x, self.topk_idx, self.slot_pos, cap, self.rows, None, self.status, stream, self.sched)
        ep_ll_gemm_swiglu_bf16(self.rows, w13, self.count, self.inner, self.gate_up, self.status, stream)
        ep_ll_gemm_bf16(self.inner, w2, self.count, self.y, self.status, stream)
        ep_ll_combine(sh, self.y, cap, self.topk_idx, self.topk_w, self.slot_pos, self.combined_x, self.status, stream)
        return self.combined_x

    def backward(self, grad_out, logits, w13, w2, grad_logits, grad_w13, grad_w2, stream=None):
        """``grad_out`` [R, T, H] bf16, and the last run's ``logits`` and weights -> grad_x
        [R, T, H] bf16; writes ``grad_logits`` (the logits' type), ``grad_w13`` and ``grad_w2``
        (fp32 or bf16, the weights' shapes), every element of them."""
        sh, cap, F = self.shape, self.expert_capacity, self.ffn
        E, H = sh.num_experts, sh.hidden
        # views with another order of the same sizes would hide a wrong shape from the calls; and nothing is launched for one
        bf16 = torch.bfloat16
        _t(w13, bf16, (E, 2, F, H), "w13")
        _t(w2, bf16, (E, H, F), "w2")
        for t, shape, name in ((grad_w13, (E, 2, F, H), "grad_w13"), (grad_w2, (E, H, F), "grad_w2")):
            _t(t, bf16 if t is not None and t.dtype == bf16 else torch.float32, shape, name)
        ep_ll_combine_backward(sh, grad_out, self.y, cap, self.topk_idx, self.topk_w, self.slot_pos, self.grad_y,
                               self.grad_topk_w, self.status, stream)
        ep_route_backward(sh, self.route, logits, self.topk_idx, self.grad_topk_w, grad_logits, self.status, stream)
        ep_ll_gemm_dswiglu_bf16(self.grad_y, w2, self.gate_up, self.count, self.grad_gate_up, self.status, stream)
        flat = self.grad_gate_up.view(E, cap, 2 * F)
        ep_ll_gemm_dgrad_bf16(flat, w13.view(E, 2 * F, H), self.count, self.grad_rows, self.status, stream)
        ep_ll_combine(sh, self.grad_rows, cap, self.topk_idx, self.ones, self.slot_pos, self.grad_x, self.status, stream)
        ep_ll_gemm_wgrad_bf16(flat, self.rows, self.count, grad_w13.view(E, 2 * F, H), self.status, stream)
        ep_ll_gemm_wgrad_bf16(self.grad_y, self.inner, self.count, grad_w2, self.status, stream)
        return self.grad_x
