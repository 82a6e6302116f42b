"""WBMM (Windowed Batch Matrix Multiplication) for AMD MI355X (gfx950).

Thin Python binding over the C ABI of ``libwbmm.so`` (declared in ``include/wbmm.h``). Each
function here has the C entry point's name and only marshals arguments: PyTorch supplies device
memory and the current stream, every step of the operator runs in the library's HIP kernels.
There is no CPU fallback: if the library is missing or cannot load, calls raise ``WbmmError``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import Optional

__all__ = [
    "WbmmError", "lib_path", "load_library", "abi_version",
    "wbmm_build_index", "wbmm_build_matrix", "wbmm_fold_hier",
    "wbmm_forward", "wbmm_forward_workspace_bytes",
    "wbmm_backward", "wbmm_backward_workspace_bytes", "wbmm_set_launch_events",
    "wbmm_forward_hier", "wbmm_forward_hier_workspace_bytes",
    "wbmm_backward_hier", "wbmm_backward_hier_workspace_bytes", "wbmm_dwconv_forward",
    "wbmm_forward_shifted", "wbmm_forward_shifted_workspace_bytes", "wbmm_backward_shifted",
    "wbmm_backward_shifted_workspace_bytes", "wbmm_probe_mfma", "wbmm_backward_bf16",
    "wbmm_backward_bf16_workspace_bytes", "wbmm_backward_noalloc", "WBMM_NOALLOC_SCRATCH_BYTES",
    "wbmm_ckpt_pack", "wbmm_ckpt_unpack", "wbmm_backward_ckpt",
    "wbmm_backward_ckpt_workspace_bytes", "wbmm_scan_forward", "wbmm_scan_backward",
    "wbmm_scan_forward_workspace_bytes", "wbmm_scan_backward_workspace_bytes", "WBMM_CKPT_GROUP", "WBMM_SCAN_CHUNK",
    "WBMM_OK", "WBMM_E_INVALID", "WBMM_E_UNSUPPORTED", "WBMM_E_WORKSPACE", "WBMM_E_HIP",
]

WBMM_OK, WBMM_E_INVALID, WBMM_E_UNSUPPORTED, WBMM_E_WORKSPACE, WBMM_E_HIP = range(5)
WBMM_F32, WBMM_BF16 = 0, 1
WBMM_NCHW, WBMM_NHWC = 0, 1
WBMM_CKPT_INT8, WBMM_CKPT_E4M3 = 0, 1
WBMM_CKPT_GROUP = 32   # elements per scale of an 8-bit checkpoint
WBMM_SCAN_CHUNK = 32   # steps between two states that the recurrence's forward keeps
WBMM_NOALLOC_SCRATCH_BYTES = 32 << 20  # the library's fixed scratch for wbmm_backward_noalloc

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_LOCK = threading.Lock()


class WbmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"wbmm status {status}: {message}")
        self.status = status


def lib_path() -> str:
    return os.path.join(_PKG_DIR, "libwbmm.so")


def _declare(lib):
    c_int, c_size, vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    c_i64 = ctypes.c_int64
    sigs = {
        "wbmm_abi_version": (c_int, []),
        "wbmm_last_error": (ctypes.c_char_p, []),
        "wbmm_build_index": (c_int, [c_int, vp, vp]),
        "wbmm_build_matrix": (c_int, [vp, c_int, c_int, c_int, vp, vp]),
        "wbmm_fold_hier": (c_int, [vp, vp, c_int, c_int, c_int, c_int, vp, vp]),
        "wbmm_forward_workspace_bytes": (c_size, [c_int] * 8),
        "wbmm_forward": (c_int, [c_int] * 8 + [vp] * 7 + [c_size, vp]),
        "wbmm_backward_workspace_bytes": (c_size, [c_int] * 7),
        "wbmm_backward": (c_int, [c_int] * 6 + [vp] * 10 + [c_size, vp]),
        "wbmm_set_launch_events": (c_int, [vp, vp]),
        "wbmm_forward_hier_workspace_bytes": (c_size, [c_int] * 9),
        "wbmm_forward_hier": (c_int, [c_int] * 7 + [vp] * 7 + [c_size, vp]),
        "wbmm_backward_hier_workspace_bytes": (c_size, [c_int] * 8),
        "wbmm_backward_hier": (c_int, [c_int] * 7 + [vp] * 11 + [c_size, vp]),
        "wbmm_dwconv_forward": (c_int, [c_int] * 5 + [vp] * 4),
        "wbmm_probe_mfma_flops": (ctypes.c_double, [c_int] * 3),
        "wbmm_backward_bf16_workspace_bytes": (c_size, [c_int] * 7),
        "wbmm_backward_bf16": (c_int, [c_int] * 6 + [vp] * 9 + [c_size, vp]),
        "wbmm_probe_mfma": (c_int, [c_int] * 3 + [vp, vp]),
        "wbmm_forward_shifted_workspace_bytes": (c_size, [c_int] * 10),
        "wbmm_forward_shifted": (c_int, [c_int] * 10 + [vp] * 7 + [c_size, vp]),
        "wbmm_backward_shifted_workspace_bytes": (c_size, [c_int] * 9),
        "wbmm_backward_shifted": (c_int, [c_int] * 8 + [vp] * 10 + [c_size, vp]),
        "wbmm_backward_noalloc": (c_int, [c_int] * 6 + [vp] * 10),
        "wbmm_ckpt_pack": (c_int, [vp, c_i64, c_int, c_int, vp, vp, vp]),
        "wbmm_ckpt_unpack": (c_int, [vp, vp, c_i64, c_int, c_int, vp, vp]),
        "wbmm_backward_ckpt_workspace_bytes": (c_size, [c_int] * 8),
        "wbmm_backward_ckpt": (c_int, [c_int] * 8 + [vp] * 11 + [c_size, vp]),
        "wbmm_scan_forward_workspace_bytes": (c_size, [c_i64] * 3),
        "wbmm_scan_backward_workspace_bytes": (c_size, [c_i64] * 3 + [c_int]),
        "wbmm_scan_forward": (c_int, [c_i64] * 3 + [c_int] * 2 + [vp] * 4 + [c_i64] + [vp] * 4 +
                              [c_size, vp]),
        "wbmm_scan_backward": (c_int, [c_i64] * 3 + [c_int] * 3 + [vp] * 8 + [c_i64] + [vp] * 4 +
                               [c_size, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load_library(path: Optional[str] = None):
    """Load libwbmm.so (built in-tree by ``receptive_field_spatial_amd.build``)."""
    global _LIB
    with _LOCK:
        if _LIB is None or path is not None:
            p = path or lib_path()
            if not os.path.exists(p):
                raise WbmmError(WBMM_E_UNSUPPORTED,
                                f"{p} is missing: build it with `python -m receptive_field_spatial_amd.build`")
            _LIB = _declare(ctypes.CDLL(p))
        return _LIB


def _lib():
    return _LIB if _LIB is not None else load_library()


def abi_version() -> int:
    return _lib().wbmm_abi_version()


def _check(status: int):
    if status != WBMM_OK:
        raise WbmmError(status, _lib().wbmm_last_error().decode(errors="replace"))


# ----------------------------------------------------------------------------- torch plumbing
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise WbmmError(WBMM_E_INVALID, "tensors must be on the GPU")
    if not t.is_contiguous():
        raise WbmmError(WBMM_E_INVALID, "tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.float32:
        return WBMM_F32
    if dt == torch.bfloat16:
        return WBMM_BF16
    raise WbmmError(WBMM_E_INVALID, f"unsupported dtype {dt}")


def _layout_code(layout: str) -> int:
    if layout.upper() == "NCHW":
        return WBMM_NCHW
    if layout.upper() == "NHWC":
        return WBMM_NHWC
    raise WbmmError(WBMM_E_INVALID, f"unknown layout {layout}")


def _bchw(x, layout: str):
    if x.dim() != 4:
        raise WbmmError(WBMM_E_INVALID, "feature maps are 4-D")
    if _layout_code(layout) == WBMM_NCHW:
        B, C, H, W = x.shape
    else:
        B, H, W, C = x.shape
    return int(B), int(C), int(H), int(W)


# ----------------------------------------------------------------------------- entry points
def wbmm_build_index(w: int, out=None, stream=None):
    """int32 (d, d) relative-position index of one w x w window."""
    torch = _torch()
    d = w * w
    if out is None:
        out = torch.empty((d, d), dtype=torch.int32, device="cuda")
    _check(_lib().wbmm_build_index(int(w), _ptr(out), _stream(stream)))
    return out


def wbmm_build_matrix(T, w: int, out=None, stream=None):
    """Cached matrices M (C, d, d) gathered from the tables T (C, 2w-1, 2w-1)."""
    torch = _torch()
    C = int(T.shape[0])
    d = w * w
    if out is None:
        out = torch.empty((C, d, d), dtype=T.dtype, device=T.device)
    _check(_lib().wbmm_build_matrix(_ptr(T), C, int(w), _dtype_code(T.dtype), _ptr(out),
                                    _stream(stream)))
    return out


def wbmm_fold_hier(M_in, T_sub, w: int, s: int, out=None, stream=None):
    """Fold the s x s sub-window tables T_sub (C, 2s-1, 2s-1) into M_in (C, d, d)."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(M_in)
    _check(_lib().wbmm_fold_hier(_ptr(M_in), _ptr(T_sub), int(M_in.shape[0]), int(w), int(s),
                                 _dtype_code(M_in.dtype), _ptr(out), _stream(stream)))
    return out


def wbmm_forward_workspace_bytes(B, C, H, W, w, layout="NCHW", has_mix=False, has_z_save=False) -> int:
    return int(_lib().wbmm_forward_workspace_bytes(B, C, H, W, w, _layout_code(layout),
                                                   int(bool(has_mix)), int(bool(has_z_save))))


def wbmm_forward(x, w: int, T=None, M=None, mix_w=None, *, layout: str = "NCHW", out_dtype=None,
                 y=None, z_save=None, workspace=None, stream=None):
    """Layer forward. Returns y (and z_save, when given, holds the pre-mix output)."""
    return _forward(x, w, None, T, M, mix_w, layout, out_dtype, y, z_save, workspace, stream)


def wbmm_forward_shifted_workspace_bytes(B, C, H, W, w, oy, ox, layout="NCHW", has_mix=False,
                                         has_z_save=False) -> int:
    return int(_lib().wbmm_forward_shifted_workspace_bytes(B, C, H, W, int(w), int(oy), int(ox),
                                                           _layout_code(layout),
                                                           int(bool(has_mix)),
                                                           int(bool(has_z_save))))


def wbmm_forward_shifted(x, w: int, oy: int, ox: int, T=None, M=None, mix_w=None, *,
                         layout: str = "NCHW", out_dtype=None, y=None, z_save=None,
                         workspace=None, stream=None):
    """Layer forward on the window grid offset by (oy, ox) (interleaved windows). Returns y."""
    return _forward(x, w, (int(oy), int(ox)), T, M, mix_w, layout, out_dtype, y, z_save,
                    workspace, stream)


def _forward(x, w, shift, T, M, mix_w, layout, out_dtype, y, z_save, workspace, stream):
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    out_dtype = out_dtype or x.dtype
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    if shift is None:
        need = wbmm_forward_workspace_bytes(B, C, H, W, w, layout, mix_w is not None,
                                            z_save is not None)
    else:
        need = wbmm_forward_shifted_workspace_bytes(B, C, H, W, w, shift[0], shift[1], layout,
                                                    mix_w is not None, z_save is not None)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_layout_code(layout), _dtype_code(x.dtype), _dtype_code(out_dtype), _ptr(x), _ptr(T),
            _ptr(M), _ptr(mix_w), _ptr(z_save), _ptr(y), _ptr(workspace), ws_bytes,
            _stream(stream))
    if shift is None:
        _check(_lib().wbmm_forward(B, C, H, W, int(w), *args))
    else:
        _check(_lib().wbmm_forward_shifted(B, C, H, W, int(w), shift[0], shift[1], *args))
    return y


def wbmm_backward_workspace_bytes(B, C, H, W, w, layout="NCHW", has_mix=False) -> int:
    return int(_lib().wbmm_backward_workspace_bytes(B, C, H, W, w, _layout_code(layout),
                                                    int(bool(has_mix))))


def wbmm_backward(x, dy, w: int, T=None, M=None, mix_w=None, z_saved=None, *, layout: str = "NCHW",
                  dx=True, dT=True, dmix_w=True, workspace=None, stream=None):
    """Layer backward (fp32). Returns (dx, dT, dmix_w); an output passed as False is skipped.

    ``workspace`` (uint8, at least wbmm_backward_workspace_bytes); one is allocated when None.
    """
    return _backward(x, dy, w, None, T, M, mix_w, z_saved, layout, dx, dT, dmix_w, workspace,
                     stream)


def wbmm_backward_noalloc(x, dy, w: int, T=None, M=None, mix_w=None, z_saved=None, *,
                          layout: str = "NCHW", dx=True, dT=True, dmix_w=True, stream=None):
    """wbmm_backward without a workspace: the library's own fixed scratch (one per GPU,
    WBMM_NOALLOC_SCRATCH_BYTES) holds what the backward needs, and the C call allocates nothing.
    Outputs passed as tensors are written in place (pass them all to keep the whole call free of
    allocations); True allocates one here, False skips it. Returns (dx, dT, dmix_w)."""
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    L = 2 * w - 1
    dev = x.device
    dx_t = torch.empty_like(x) if dx is True else (dx if dx is not False else None)
    dT_t = torch.empty((C, L, L), dtype=torch.float32, device=dev) if dT is True else (dT if dT is not False else None)
    if mix_w is None:
        dW_t = None
    else:
        dW_t = torch.empty((C, 3, 3), dtype=torch.float32, device=dev) if dmix_w is True else (dmix_w if dmix_w is not False else None)
    _check(_lib().wbmm_backward_noalloc(B, C, H, W, int(w), _layout_code(layout), _ptr(x), _ptr(T),
                                        _ptr(M), _ptr(mix_w), _ptr(z_saved), _ptr(dy), _ptr(dx_t),
                                        _ptr(dT_t), _ptr(dW_t), _stream(stream)))
    return dx_t, dT_t, dW_t


def wbmm_backward_shifted_workspace_bytes(B, C, H, W, w, oy, ox, layout="NCHW",
                                          has_mix=False) -> int:
    return int(_lib().wbmm_backward_shifted_workspace_bytes(B, C, H, W, int(w), int(oy), int(ox),
                                                            _layout_code(layout),
                                                            int(bool(has_mix))))


def wbmm_backward_shifted(x, dy, w: int, oy: int, ox: int, T=None, M=None, mix_w=None,
                          z_saved=None, *, layout: str = "NCHW", dx=True, dT=True, dmix_w=True,
                          workspace=None, stream=None):
    """Backward of wbmm_forward_shifted (fp32). Returns (dx, dT, dmix_w)."""
    return _backward(x, dy, w, (int(oy), int(ox)), T, M, mix_w, z_saved, layout, dx, dT, dmix_w,
                     workspace, stream)


def _backward(x, dy, w, shift, T, M, mix_w, z_saved, layout, dx, dT, dmix_w, workspace, stream):
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    L = 2 * w - 1
    dev = x.device
    dx_t = torch.empty_like(x) if dx is True else (dx if dx is not False else None)
    dT_t = torch.empty((C, L, L), dtype=torch.float32, device=dev) if dT is True else (dT if dT is not False else None)
    if mix_w is None:
        dW_t = None
    else:
        dW_t = torch.empty((C, 3, 3), dtype=torch.float32, device=dev) if dmix_w is True else (dmix_w if dmix_w is not False else None)
    if shift is None:
        need = wbmm_backward_workspace_bytes(B, C, H, W, w, layout, mix_w is not None)
    else:
        need = wbmm_backward_shifted_workspace_bytes(B, C, H, W, w, shift[0], shift[1], layout,
                                                     mix_w is not None)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_layout_code(layout), _ptr(x), _ptr(T), _ptr(M), _ptr(mix_w), _ptr(z_saved), _ptr(dy),
            _ptr(dx_t), _ptr(dT_t), _ptr(dW_t), _ptr(workspace), ws_bytes, _stream(stream))
    if shift is None:
        _check(_lib().wbmm_backward(B, C, H, W, int(w), *args))
    else:
        _check(_lib().wbmm_backward_shifted(B, C, H, W, int(w), shift[0], shift[1], *args))
    return dx_t, dT_t, dW_t


def wbmm_forward_hier_workspace_bytes(B, C, H, W, w, s, layout="NCHW", has_mix=False,
                                      has_z_save=False) -> int:
    return int(_lib().wbmm_forward_hier_workspace_bytes(B, C, H, W, int(w), int(s),
                                                        _layout_code(layout), int(bool(has_mix)),
                                                        int(bool(has_z_save))))


def wbmm_forward_hier(x, w: int, s: int, T, T_sub, mix_w=None, *, layout: str = "NCHW", y=None,
                      z_save=None, workspace=None, stream=None):
    """Layer forward (fp32) with the s x s sub-window tables T_sub (C, 2s-1, 2s-1) folded into
    the matrix (s divides w and s < w; on chip for the quadrants, w = 2s <= 16, otherwise into a
    matrix in the workspace). Returns y (and z_save, when given, holds the pre-mix output)."""
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    if y is None:
        y = torch.empty_like(x)
    need = wbmm_forward_hier_workspace_bytes(B, C, H, W, w, s, layout, mix_w is not None,
                                             z_save is not None)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().wbmm_forward_hier(B, C, H, W, int(w), int(s), _layout_code(layout), _ptr(x),
                                    _ptr(T), _ptr(T_sub), _ptr(mix_w), _ptr(z_save), _ptr(y),
                                    _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def wbmm_backward_hier_workspace_bytes(B, C, H, W, w, s, layout="NCHW", has_mix=False) -> int:
    return int(_lib().wbmm_backward_hier_workspace_bytes(B, C, H, W, int(w), int(s),
                                                         _layout_code(layout), int(bool(has_mix))))


def wbmm_backward_hier(x, dy, w: int, s: int, T, T_sub, mix_w=None, z_saved=None, *,
                       layout: str = "NCHW", dx=True, dT=True, dT_sub=True, dmix_w=True,
                       workspace=None, stream=None):
    """Backward of wbmm_forward_hier (fp32). Returns (dx, dT, dT_sub, dmix_w); an output passed as
    False is skipped."""
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    L, Ls = 2 * w - 1, 2 * s - 1
    dev = x.device

    def out(v, shape):
        return torch.empty(shape, dtype=torch.float32, device=dev) if v is True else (v if v is not False else None)

    dx_t = out(dx, tuple(x.shape))
    dT_t = out(dT, (C, L, L))
    dTs_t = out(dT_sub, (C, Ls, Ls))
    dW_t = None if mix_w is None else out(dmix_w, (C, 3, 3))
    need = wbmm_backward_hier_workspace_bytes(B, C, H, W, w, s, layout, mix_w is not None)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().wbmm_backward_hier(B, C, H, W, int(w), int(s), _layout_code(layout), _ptr(x),
                                     _ptr(T), _ptr(T_sub), _ptr(mix_w), _ptr(z_saved), _ptr(dy),
                                     _ptr(dx_t), _ptr(dT_t), _ptr(dTs_t), _ptr(dW_t),
                                     _ptr(workspace), ws_bytes, _stream(stream)))
    return dx_t, dT_t, dTs_t, dW_t


def wbmm_set_launch_events(before, after):
    """Attach two HIP events (raw handles) to the dispatch of the next forward/backward call's
    main kernel: their elapsed time is that kernel's execution."""
    _check(_lib().wbmm_set_launch_events(before, after))


def wbmm_dwconv_forward(x, w_dw, *, y=None, stream=None):
    """k x k depthwise convolution (DW-Std, the pages' comparison operator): fp32 NCHW x
    (B, C, H, W), weights w_dw (C, k, k), zero padding k // 2, stride 1. Returns y."""
    torch = _torch()
    B, C, H, W = _bchw(x, "NCHW")
    k = int(w_dw.shape[-1])
    if tuple(w_dw.shape) != (C, k, k):
        raise WbmmError(WBMM_E_INVALID, f"w_dw must be (C, k, k), got {tuple(w_dw.shape)}")
    if x.dtype != torch.float32 or w_dw.dtype != torch.float32:
        raise WbmmError(WBMM_E_INVALID, "the depthwise convolution is fp32")
    if y is None:
        y = torch.empty_like(x)
    _check(_lib().wbmm_dwconv_forward(B, C, H, W, k, _ptr(x), _ptr(w_dw), _ptr(y),
                                      _stream(stream)))
    return y


def wbmm_probe_mfma(dtype, blocks: int, iters: int, *, out=None, stream=None) -> float:
    """Matrix-core peak probe (measurement aid): launches it and returns the launch's flops.
    dtype: torch.float32 or torch.bfloat16 (the MFMA operand type)."""
    torch = _torch()
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device="cuda")
    code = _dtype_code(dtype)
    _check(_lib().wbmm_probe_mfma(code, int(blocks), int(iters), _ptr(out), _stream(stream)))
    return float(_lib().wbmm_probe_mfma_flops(code, int(blocks), int(iters)))


def wbmm_backward_bf16_workspace_bytes(B, C, H, W, w, layout="NCHW", has_mix=False) -> int:
    return int(_lib().wbmm_backward_bf16_workspace_bytes(B, C, H, W, int(w), _layout_code(layout),
                                                         int(bool(has_mix))))


def wbmm_backward_bf16(x, dy, w: int, T, mix_w=None, z_saved=None, *, layout: str = "NCHW",
                       dx=True, dT=True, dmix_w=True, workspace=None, stream=None):
    """Layer backward with bf16 maps (x, dy, z_saved bf16; T bf16). Returns (dx bf16, dT fp32,
    dmix_w fp32); an output passed as False is skipped."""
    torch = _torch()
    B, C, H, W = _bchw(x, layout)
    L = 2 * w - 1
    dev = x.device
    dx_t = torch.empty_like(x) if dx is True else (dx if dx is not False else None)
    dT_t = torch.empty((C, L, L), dtype=torch.float32, device=dev) if dT is True else (dT if dT is not False else None)
    if mix_w is None:
        dW_t = None
    else:
        dW_t = torch.empty((C, 3, 3), dtype=torch.float32, device=dev) if dmix_w is True else (dmix_w if dmix_w is not False else None)
    need = wbmm_backward_bf16_workspace_bytes(B, C, H, W, w, layout, mix_w is not None)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib().wbmm_backward_bf16(B, C, H, W, int(w), _layout_code(layout), _ptr(x), _ptr(T),
                                     _ptr(mix_w),
                                     _ptr(z_saved), _ptr(dy), _ptr(dx_t), _ptr(dT_t), _ptr(dW_t),
                                     _ptr(workspace), ws_bytes, _stream(stream)))
    return dx_t, dT_t, dW_t


# ----------------------------------------------------------------------------- 8-bit checkpoints
def _fmt_code(fmt: str) -> int:
    if fmt == "int8":
        return WBMM_CKPT_INT8
    if fmt == "e4m3":
        return WBMM_CKPT_E4M3
    raise WbmmError(WBMM_E_INVALID, f"unknown checkpoint format {fmt!r} (int8 or e4m3)")


# Per-call host time counts in a one-step call, so the checks below take one pass over each tensor
# and hand back its address.
def _device(name, t) -> int:
    """The device of a call, from one of its tensors: the current one."""
    idx = -1 if t is None else t.get_device()
    if idx < 0 or idx != _torch()._C._cuda_getDevice():
        why = ("is required" if t is None else "must be on the GPU" if idx < 0 else
               f"is on {t.device}, which is not the current device")
        raise WbmmError(WBMM_E_INVALID, f"{name} {why}")
    return idx


def _need(name, t, shape, dtype, idx):
    """Address of a tensor argument of this shape and dtype, dense, on device idx."""
    if (t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != idx
            or not t.is_contiguous()):
        why = ("is required" if t is None else
               f"must have shape {tuple(shape)}, got {tuple(t.shape)}" if t.shape != shape else
               f"must be {dtype}, got {t.dtype}" if t.dtype is not dtype else
               f"is on {t.device}, not on GPU {idx}" if t.get_device() != idx else
               "must be contiguous")
        raise WbmmError(WBMM_E_INVALID, f"{name} {why}")
    return t.data_ptr()


def _opt(name, t, shape, dtype, idx):
    return None if t is None else _need(name, t, shape, dtype, idx)


def _out(name, v, shape, dtype, idx, like=None):
    """An output argument: True allocates it (like a dense tensor of its shape and dtype, where there
    is one: the cheaper call), False or None skips it, a tensor is written. Returns the tensor and
    its address."""
    if v is True:
        torch = _torch()
        v = torch.empty(shape, dtype=dtype, device=idx) if like is None else torch.empty_like(like)
        return v, v.data_ptr()
    if v is False or v is None:
        return None, None
    return v, _need(name, v, shape, dtype, idx)


def _current_stream(idx) -> int:
    return _torch()._C._cuda_getCurrentRawStream(idx)


def _on_stream(stream, name, t):
    """Makes the call's stream the current one, so that what it allocates belongs to that stream."""
    idx, cuda = _device(name, t), _torch().cuda
    if not isinstance(stream, cuda.Stream):
        raw = _stream(stream)
        stream = cuda.ExternalStream(raw, device=idx) if raw else cuda.default_stream(idx)
    return cuda.stream(stream)


def _workspace(need, workspace, idx):
    """A caller's workspace when it is given (the library checks its size), else a new one; its
    address and size."""
    if workspace is not None:
        if workspace.get_device() != idx or not workspace.is_contiguous():
            raise WbmmError(WBMM_E_INVALID, f"workspace must be contiguous and on GPU {idx}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    workspace = _torch().empty(need, dtype=_torch().uint8, device=idx)
    return workspace, workspace.data_ptr(), need


def _ckpt_scales(n: int) -> int:
    return -(-n // WBMM_CKPT_GROUP)


def wbmm_ckpt_pack(x, *, fmt: str = "int8", codes=None, scales=None, stream=None):
    """Packs x (fp32 or bf16, any shape) into an 8-bit checkpoint: (codes, scales), codes uint8 in
    x's shape, scales uint8 with one entry per WBMM_CKPT_GROUP elements in memory order."""
    if stream is not None:
        with _on_stream(stream, "x", x):
            return wbmm_ckpt_pack(x, fmt=fmt, codes=codes, scales=scales)
    u8 = _torch().uint8
    code, dt, idx = _fmt_code(fmt), _dtype_code(x.dtype), _device("x", x)
    xp, n = _need("x", x, x.shape, x.dtype, idx), x.numel()
    codes, cp = _out("codes", True if codes is None else codes, x.shape, u8, idx)
    scales, sp = _out("scales", True if scales is None else scales, (_ckpt_scales(n),), u8, idx)
    _check(_lib().wbmm_ckpt_pack(xp, n, dt, code, cp, sp, _current_stream(idx)))
    return codes, scales


def wbmm_ckpt_unpack(codes, scales, *, fmt: str = "int8", dtype=None, out=None, stream=None):
    """The values of a checkpoint in `dtype` (fp32 by default, or out's)."""
    if stream is not None:
        with _on_stream(stream, "codes", codes):
            return wbmm_ckpt_unpack(codes, scales, fmt=fmt, dtype=dtype, out=out)
    torch = _torch()
    code, idx = _fmt_code(fmt), _device("codes", codes)
    dtype = dtype or (torch.float32 if out is None else out.dtype)
    dt, n = _dtype_code(dtype), codes.numel()
    cp = _need("codes", codes, codes.shape, torch.uint8, idx)
    sp = _need("scales", scales, (_ckpt_scales(n),), torch.uint8, idx)
    out, xp = _out("out", True if out is None else out, codes.shape, dtype, idx)
    _check(_lib().wbmm_ckpt_unpack(cp, sp, n, dt, code, xp, _current_stream(idx)))
    return out


@functools.lru_cache(maxsize=256)
def _backward_ckpt_bytes(*sizes) -> int:
    return int(_lib().wbmm_backward_ckpt_workspace_bytes(*sizes))


def wbmm_backward_ckpt_workspace_bytes(B, C, H, W, w, layout="NCHW", dtype=None,
                                       has_mix=False) -> int:
    code = WBMM_F32 if dtype is None else _dtype_code(dtype)
    return _backward_ckpt_bytes(int(B), int(C), int(H), int(W), int(w), _layout_code(layout), code,
                                int(bool(has_mix)))


def wbmm_backward_ckpt(x_ckpt, dy, w: int, T, mix_w=None, z_ckpt=None, *, fmt: str = "int8",
                       layout: str = "NCHW", dx=True, dT=True, dmix_w=True, workspace=None,
                       stream=None):
    """Layer backward with x and z kept as 8-bit checkpoints: x_ckpt and z_ckpt are the (codes,
    scales) that wbmm_ckpt_pack returned for the maps (z_ckpt exactly with mix_w). dy and T are
    both fp32 or both bf16. Returns (dx in dy's dtype, dT fp32, dmix_w fp32); an output passed as
    False is skipped."""
    if stream is not None:
        with _on_stream(stream, "dy", dy):
            return wbmm_backward_ckpt(x_ckpt, dy, w, T, mix_w, z_ckpt, fmt=fmt, layout=layout, dx=dx,
                                      dT=dT, dmix_w=dmix_w, workspace=workspace)
    torch = _torch()
    idx = _device("dy", dy)
    B, C, H, W = _bchw(dy, layout)
    w, n, shape = int(w), dy.numel(), dy.shape
    lay, fcode, dt = _layout_code(layout), _fmt_code(fmt), _dtype_code(dy.dtype)
    L = 2 * w - 1
    if (mix_w is None) != (z_ckpt is None):
        raise WbmmError(WBMM_E_INVALID, "z_ckpt is required exactly when mix_w is given")
    u8, f32, scales = torch.uint8, torch.float32, (_ckpt_scales(n),)
    dyp = _need("dy", dy, shape, dy.dtype, idx)
    xc, xs = _need("x codes", x_ckpt[0], shape, u8, idx), _need("x scales", x_ckpt[1], scales, u8, idx)
    Tp = _need("T", T, (C, L, L), dy.dtype, idx)
    mp = zc = zs = None
    if mix_w is not None:
        mp = _need("mix_w", mix_w, (C, 3, 3), f32, idx)
        zc = _need("z codes", z_ckpt[0], shape, u8, idx)
        zs = _need("z scales", z_ckpt[1], scales, u8, idx)
    dx, dxp = _out("dx", dx, shape, dy.dtype, idx, dy)
    dT, dTp = _out("dT", dT, (C, L, L), f32, idx)
    dmix_w, dWp = (None, None) if mix_w is None else _out("dmix_w", dmix_w, (C, 3, 3), f32, idx)
    ws, wp, wb = _workspace(_backward_ckpt_bytes(B, C, H, W, w, lay, dt, int(mix_w is not None)),
                            workspace, idx)
    _check(_lib().wbmm_backward_ckpt(B, C, H, W, w, lay, dt, fcode, xc, xs, Tp, mp, zc, zs, dyp,
                                     dxp, dTp, dWp, wp, wb, _current_stream(idx)))
    return dx, dT, dmix_w


# ----------------------------------------------------------------------------- recurrence
@functools.lru_cache(maxsize=256)
def wbmm_scan_forward_workspace_bytes(outer: int, length: int, inner: int) -> int:
    return int(_lib().wbmm_scan_forward_workspace_bytes(int(outer), int(length), int(inner)))


@functools.lru_cache(maxsize=256)
def wbmm_scan_backward_workspace_bytes(outer: int, length: int, inner: int,
                                       has_states: bool = True) -> int:
    return int(_lib().wbmm_scan_backward_workspace_bytes(int(outer), int(length), int(inner),
                                                         int(bool(has_states))))


@functools.lru_cache(maxsize=256)
def _scan_sizes(shape, dim: int):
    """(outer, len, inner) of a tensor's shape, and the shapes of h0 / h_last and of states."""
    if not -len(shape) <= dim < len(shape):
        raise WbmmError(WBMM_E_INVALID, f"dim={dim} is no dimension of a tensor of {len(shape)}")
    dim %= len(shape)
    lead, tail, length = tuple(shape[:dim]), tuple(shape[dim + 1:]), shape[dim]
    return (math.prod(lead), length, math.prod(tail), lead + tail,
            lead + (-(-length // WBMM_SCAN_CHUNK),) + tail)


def _scan_lens(lens, idx):
    if lens is None:
        return None, 0
    n = lens.numel()
    if n == 0:
        raise WbmmError(WBMM_E_INVALID, "lens is empty")
    return _need("lens", lens, (n,), _torch().int32, idx), n


def wbmm_scan_forward(g, u, dim: int, *, h0=None, lens=None, reverse: bool = False, h=None,
                      h_last=False, states=False, workspace=None, stream=None):
    """Gated linear recurrence along dimension `dim` of g and u (same shape, fp32 or bf16, dense):
    h_t = a_t h_{t-1} + (1 - a_t) u_t with a_t = sigmoid(g_t).

    h0: fp32 state in g's shape without `dim`, or None for zeros. lens: int32 lengths (1-D, on the
    GPU), one for each of the leading dimensions' sequences or for each equal run of them; h is 0
    past a sequence's end. reverse: from each sequence's last position to its first. h_last and
    states: True allocates them, a tensor is written (h_last may be h0), False skips them; states
    (fp32, `dim` divided by WBMM_SCAN_CHUNK and rounded up) is what wbmm_scan_backward starts
    from. Returns (h, h_last, states)."""
    if stream is not None:
        with _on_stream(stream, "g", g):
            return wbmm_scan_forward(g, u, dim, h0=h0, lens=lens, reverse=reverse, h=h,
                                     h_last=h_last, states=states, workspace=workspace)
    f32, dtype, shape = _torch().float32, g.dtype, g.shape
    dt, idx = _dtype_code(dtype), _device("g", g)
    outer, length, inner, flat, kept = _scan_sizes(shape, dim)
    gp, up = _need("g", g, shape, dtype, idx), _need("u", u, shape, dtype, idx)
    h0p = _opt("h0", h0, flat, f32, idx)
    lp, n_lens = _scan_lens(lens, idx)
    h, hp = _out("h", True if h is None else h, shape, dtype, idx, g)
    h_last, hlp = _out("h_last", h_last, flat, f32, idx, h0)
    states, sp = _out("states", states, kept, f32, idx)
    ws, wp, wb = _workspace(wbmm_scan_forward_workspace_bytes(outer, length, inner), workspace,
                            idx)
    _check(_lib().wbmm_scan_forward(outer, length, inner, dt, int(bool(reverse)), gp, up, h0p,
                                    lp, n_lens, hp, hlp, sp, wp, wb, _current_stream(idx)))
    return h, h_last, states


def wbmm_scan_backward(g, states, dh, dim: int, *, u=None, u_ckpt=None, fmt: str = "int8",
                       h0=None, dh_last=None, lens=None, reverse: bool = False, dg=None, du=None,
                       dh0=True, workspace=None, stream=None):
    """Gradients of wbmm_scan_forward (same g, dim, lens and reverse; states as it wrote them).
    Without states (None) they are formed again from h0 (fp32, or None for zeros) and the u given.
    u: the forward's u, or u_ckpt: its checkpoint (codes, scales) in `fmt`. dh: gradient of h;
    dh_last: fp32 gradient of h_last, or None. Returns (dg, du, dh0), dg and du in g's dtype and 0
    past a sequence's end, dh0 fp32 (False skips it)."""
    if stream is not None:
        with _on_stream(stream, "g", g):
            return wbmm_scan_backward(g, states, dh, dim, u=u, u_ckpt=u_ckpt, fmt=fmt, h0=h0,
                                      dh_last=dh_last, lens=lens, reverse=reverse, dg=dg, du=du,
                                      dh0=dh0, workspace=workspace)
    torch = _torch()
    f32, dtype, shape = torch.float32, g.dtype, g.shape
    dt, idx = _dtype_code(dtype), _device("g", g)
    outer, length, inner, flat, kept = _scan_sizes(shape, dim)
    if (u is None) == (u_ckpt is None):
        raise WbmmError(WBMM_E_INVALID, "exactly one of u and u_ckpt must be given")
    gp, dhp = _need("g", g, shape, dtype, idx), _need("dh", dh, shape, dtype, idx)
    if u_ckpt is None:
        up, us, fcode = _need("u", u, shape, dtype, idx), None, 0
    else:
        fcode = _fmt_code(fmt)
        up = _need("u codes", u_ckpt[0], shape, torch.uint8, idx)
        us = _need("u scales", u_ckpt[1], (_ckpt_scales(g.numel()),), torch.uint8, idx)
    sp, h0p = _opt("states", states, kept, f32, idx), _opt("h0", h0, flat, f32, idx)
    dlp = _opt("dh_last", dh_last, flat, f32, idx)
    lp, n_lens = _scan_lens(lens, idx)
    dg, dgp = _out("dg", True if dg is None else dg, shape, dtype, idx, g)
    du, dup = _out("du", True if du is None else du, shape, dtype, idx, g)
    dh0, d0p = _out("dh0", dh0, flat, f32, idx, dh_last)
    need = wbmm_scan_backward_workspace_bytes(outer, length, inner, states is not None)
    ws, wp, wb = _workspace(need, workspace, idx)
    _check(_lib().wbmm_scan_backward(outer, length, inner, dt, int(bool(reverse)), fcode, gp,
                                     up, us, sp, h0p, dhp, dlp, lp, n_lens, dgp, dup, d0p, wp,
                                     wb, _current_stream(idx)))
    return dg, du, dh0
