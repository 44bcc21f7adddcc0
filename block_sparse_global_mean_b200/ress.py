"""Python binding of the C ABI in ``include/ress.h`` (ctypes).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libress.so``.  PyTorch supplies device memory and the current stream.  If
the library is missing, importing this module raises ImportError; there is no
fallback implementation.
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
from typing import NamedTuple, Optional, Tuple

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libress.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m block_sparse_global_mean_b200.build` "
        "(this package has no CPU fallback)")

lib = ctypes.CDLL(LIB_PATH)

RESS_OK = 0
RESS_ERR_INVALID_ARG = 1
RESS_ERR_UNSUPPORTED = 2
RESS_ERR_WORKSPACE = 3
RESS_ERR_CUDA = 4
RESS_ERR_TIMEOUT = 5
RESS_ERR_BAD_INDEX = 6

RESS_BF16 = 0
RESS_F32 = 1


class ress_shape(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class ress_layout(ctypes.Structure):
    _fields_ = [("tokens_per_view", ctypes.c_int32), ("real_tokens", ctypes.c_int32),
                ("special_tokens", ctypes.c_int32)]


class ress_cross_shape(ctypes.Structure):
    _fields_ = [("nq", ctypes.c_int64), ("nk", ctypes.c_int64), ("seqs", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


class ress_cache_shape(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("requests", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SIZE = ctypes.c_size_t
_SHAPE = ctypes.POINTER(ress_shape)

lib.ress_version.restype = ctypes.c_int
lib.ress_version.argtypes = []
lib.ress_status_string.restype = ctypes.c_char_p
lib.ress_status_string.argtypes = [ctypes.c_int]
lib.ress_select_workspace_bytes.restype = ctypes.c_size_t
lib.ress_select_workspace_bytes.argtypes = [_SHAPE, ctypes.c_float]
lib.ress_select_blocks.restype = ctypes.c_int
lib.ress_select_blocks.argtypes = [_SHAPE, _P, _P, _P, ctypes.c_int32, ctypes.c_float, _P, _P,
                                   ctypes.c_size_t, _P]
lib.ress_attn_workspace_bytes.restype = ctypes.c_size_t
lib.ress_attn_workspace_bytes.argtypes = [_SHAPE]
lib.ress_block_sparse_attn.restype = ctypes.c_int
lib.ress_block_sparse_attn.argtypes = [_SHAPE, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_int32,
                                       _P, _P, ctypes.c_size_t, _P]
lib.ress_block_drift.restype = ctypes.c_int
lib.ress_block_drift.argtypes = [_SHAPE, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P,
                                 ctypes.c_size_t, _P]
lib.ress_select_blocks_noalloc.restype = ctypes.c_int
lib.ress_select_blocks_noalloc.argtypes = [_SHAPE, _P, _P, _P, ctypes.c_int32, ctypes.c_float, _P, _P]
lib.ress_select_blocks_cdf.restype = ctypes.c_int
lib.ress_select_blocks_cdf.argtypes = [_SHAPE, _P, _P, ctypes.c_float, ctypes.c_int32, _P, _P, _P,
                                         ctypes.c_size_t, _P]
lib.ress_last_cuda_error.restype = ctypes.c_char_p
lib.ress_last_cuda_error.argtypes = []
lib.ress_test_exp2.restype = ctypes.c_int
lib.ress_test_exp2.argtypes = [_P, _P, ctypes.c_int32, _P]
_LAYOUT = ctypes.POINTER(ress_layout)
lib.ress_select_blocks_layout.restype = ctypes.c_int
lib.ress_select_blocks_layout.argtypes = [_SHAPE, _LAYOUT, _P, _P, ctypes.c_int32, _P, _P,
                                          ctypes.c_size_t, _P]
lib.ress_attn_layout_workspace_bytes.restype = ctypes.c_size_t
lib.ress_attn_layout_workspace_bytes.argtypes = [_SHAPE, _LAYOUT, ctypes.c_int32]
lib.ress_block_sparse_attn_layout.restype = ctypes.c_int
lib.ress_block_sparse_attn_layout.argtypes = [_SHAPE, _LAYOUT, _P, _P, _P, ctypes.c_int32, _P, _P,
                                              ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]
lib.ress_block_drift_layout.restype = ctypes.c_int
lib.ress_block_drift_layout.argtypes = [_SHAPE, _LAYOUT, _P, _P, _P, ctypes.c_int32, _P, _P, _P,
                                        _P, _P, ctypes.c_size_t, _P]
lib.ress_restore_workspace_bytes.restype = ctypes.c_size_t
lib.ress_restore_workspace_bytes.argtypes = [_SHAPE]
lib.ress_select_blocks_restore.restype = ctypes.c_int
lib.ress_select_blocks_restore.argtypes = [_SHAPE, _P, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, _P, _P, _P, _P, ctypes.c_size_t, _P]
lib.ress_vasc_workspace_bytes.restype = ctypes.c_size_t
lib.ress_vasc_workspace_bytes.argtypes = [_SHAPE]
lib.ress_select_blocks_vasc.restype = ctypes.c_int
lib.ress_select_blocks_vasc.argtypes = [_SHAPE, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
lib.ress_validate_idx.restype = ctypes.c_int
lib.ress_validate_idx.argtypes = [_SHAPE, ctypes.c_int32, _P, _P]
_CROSS = ctypes.POINTER(ress_cross_shape)
lib.ress_cross_workspace_bytes.restype = _SIZE
lib.ress_cross_workspace_bytes.argtypes = [_CROSS]
lib.ress_cross_bwd_workspace_bytes.restype = _SIZE
lib.ress_cross_bwd_workspace_bytes.argtypes = [_CROSS]
lib.ress_cross_attn.restype = ctypes.c_int
lib.ress_cross_attn.argtypes = [_CROSS] + [_P] * 10 + [_SIZE, _P]
lib.ress_cross_attn_bwd.restype = ctypes.c_int
lib.ress_cross_attn_bwd.argtypes = [_CROSS] + [_P] * 14 + [_SIZE, _P]
_CACHE = ctypes.POINTER(ress_cache_shape)
lib.ress_cache_plan.restype = ctypes.c_int
lib.ress_cache_plan.argtypes = [_CACHE, _P, _P, _P, _P, _I32, _P, _I32, _P, _P, _P, _P, _P]
lib.ress_cache_append.restype = ctypes.c_int
lib.ress_cache_append.argtypes = [_CACHE, _P, _P, _I32, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P]
lib.ress_cache_attn_workspace_bytes.restype = _SIZE
lib.ress_cache_attn_workspace_bytes.argtypes = [_CACHE, _I32, _I32]
lib.ress_cache_attn.restype = ctypes.c_int
lib.ress_cache_attn.argtypes = ([_CACHE, _I32, _I32, _P, _I64] + [_P] * 7 + [_I32] + [_P] * 3
                                + [_SIZE, _P])
lib.ress_check_device_errors.restype = ctypes.c_int
lib.ress_check_device_errors.argtypes = [_P, ctypes.POINTER(ctypes.c_int32)]


class RessError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.ress_status_string(status).decode()
        if status == RESS_ERR_CUDA:
            msg += f" [{lib.ress_last_cuda_error().decode()}]"
        super().__init__(f"{where}: {msg} (status {status})")


def _check(status: int, where: str) -> None:
    if status != RESS_OK:
        raise RessError(status, where)


def _on(device: torch.device, fn, *args) -> int:
    """Calls ``fn(*args)`` with ``device`` current: the library looks up its
    per-device state (error flag, fixed scratch) on the current device."""
    with torch.cuda.device(device):
        return fn(*args)


def make_shape(n: int, heads: int, block: int, dtype: torch.dtype, head_dim: int = 64) -> ress_shape:
    if dtype == torch.bfloat16:
        code = RESS_BF16
    elif dtype == torch.float32:
        code = RESS_F32
    else:
        raise TypeError(f"unsupported dtype {dtype}")
    return ress_shape(n, heads, head_dim, block, code)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_ptr(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _shape_of(q: torch.Tensor, block: int) -> ress_shape:
    if q.dim() != 3:
        raise ValueError("q, k, v must be [N, H, d]")
    n, h, d = q.shape
    return make_shape(n, h, block, q.dtype, d)


def _check_inputs(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor] = None) -> None:
    """k and v must match q in shape, dtype and device (the library reads all
    three with q's shape)."""
    if q.dim() != 3:
        raise ValueError("q, k, v must be [N, H, d]")
    for name, t in (("k", k), ("v", v)):
        if t is None:
            continue
        if tuple(t.shape) != tuple(q.shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, q has {tuple(q.shape)}")
        if t.dtype != q.dtype:
            raise TypeError(f"{name} is {t.dtype}, q is {q.dtype}")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")


def _check_buffer(t: torch.Tensor, shape, dtype: torch.dtype, device: torch.device,
                  name: str) -> None:
    """A caller-provided buffer must have exactly the shape, dtype and device
    the library writes or reads."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_workspace(ws: Optional[torch.Tensor], device: torch.device) -> None:
    if ws is not None:
        _check_buffer(ws, (ws.numel(),), torch.uint8, device, "workspace")


def _check_idx(idx: torch.Tensor, h: int, nb: int, device: torch.device) -> int:
    """idx must be int32 [H, nb, budget]; returns budget."""
    if idx.dim() != 3:
        raise ValueError(f"idx must be [H, nb, budget], got {tuple(idx.shape)}")
    _check_buffer(idx, (h, nb, idx.shape[2]), torch.int32, device, "idx")
    return int(idx.shape[2])


def select_workspace_bytes(n: int, heads: int, block: int, dtype: torch.dtype, lam: float) -> int:
    sh = make_shape(n, heads, block, dtype)
    return int(lib.ress_select_workspace_bytes(ctypes.byref(sh), ctypes.c_float(lam)))


def vasc_workspace_bytes(n: int, heads: int, block: int, dtype: torch.dtype) -> int:
    sh = make_shape(n, heads, block, dtype)
    return int(lib.ress_vasc_workspace_bytes(ctypes.byref(sh)))


def attn_workspace_bytes(n: int, heads: int, block: int, dtype: torch.dtype) -> int:
    sh = make_shape(n, heads, block, dtype)
    return int(lib.ress_attn_workspace_bytes(ctypes.byref(sh)))


def ress_select_blocks(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor], budget: int,
                       lam: float, block: int, idx: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Stage 1: returns idx [H, nb, budget] int32 (ascending kept blocks per row)."""
    _check_inputs(q, k, v if lam else None)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    if idx is None:
        idx = torch.empty((h, nb, budget), dtype=torch.int32, device=q.device)
    _check_buffer(idx, (h, nb, budget), torch.int32, q.device, "idx")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_select_workspace_bytes(ctypes.byref(sh), ctypes.c_float(lam)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_select_blocks, ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), int(budget),
                                    ctypes.c_float(lam), _ptr(idx), _ptr(workspace),
                                    workspace.numel(), _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks")
    return idx


def ress_select_blocks_cdf(q: torch.Tensor, k: torch.Tensor, tau: float, block: int,
                           capacity: Optional[int] = None, counts: Optional[torch.Tensor] = None,
                           idx: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None
                           ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Stage 1 with the cumulative (CDF) threshold: returns (counts [H, nb]
    int32, idx [H, nb, capacity] int32); capacity defaults to nb."""
    _check_inputs(q, k)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    cap = nb if capacity is None else int(capacity)
    if counts is None:
        counts = torch.empty((h, nb), dtype=torch.int32, device=q.device)
    if idx is None:
        idx = torch.empty((h, nb, max(cap, 1)), dtype=torch.int32, device=q.device)
    _check_buffer(counts, (h, nb), torch.int32, q.device, "counts")
    _check_buffer(idx, (h, nb, max(cap, 1)), torch.int32, q.device, "idx")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_select_workspace_bytes(ctypes.byref(sh), ctypes.c_float(0.0)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_select_blocks_cdf, ctypes.byref(sh), _ptr(q), _ptr(k), ctypes.c_float(tau),
                                        cap, _ptr(counts), _ptr(idx), _ptr(workspace),
                                        workspace.numel(), _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks_cdf")
    return counts, idx


def ress_select_blocks_noalloc(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                               budget: int, lam: float, block: int,
                               idx: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Stage 1 with the library's fixed scratch array instead of a workspace
    (for callers that cannot allocate device memory); see include/ress.h."""
    _check_inputs(q, k, v if lam else None)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    if idx is None:
        idx = torch.empty((h, n // block, budget), dtype=torch.int32, device=q.device)
    _check_buffer(idx, (h, n // block, budget), torch.int32, q.device, "idx")
    status = _on(q.device, lib.ress_select_blocks_noalloc, ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), int(budget),
                                            ctypes.c_float(lam), _ptr(idx),
                                            _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks_noalloc")
    return idx


def ress_block_sparse_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor,
                           block: int, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                           workspace: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None,
                           out_dtype: Optional[torch.dtype] = None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Stage 2: returns (out [N, H, 64], lse [H, N] float32 or None).

    The output dtype is ``out.dtype`` if ``out`` is given, else ``out_dtype``,
    else the input dtype."""
    _check_inputs(q, k, v)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    budget = _check_idx(idx, h, n // block, q.device)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    out_code = RESS_F32 if out.dtype == torch.float32 else (
        RESS_BF16 if out.dtype == torch.bfloat16 else None)
    if out_code is None:
        raise TypeError(f"unsupported output dtype {out.dtype}")
    _check_buffer(out, q.shape, out.dtype, q.device, "out")
    if lse is None and want_lse:
        lse = torch.empty((h, n), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_buffer(lse, (h, n), torch.float32, q.device, "lse")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_attn_workspace_bytes(ctypes.byref(sh)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_block_sparse_attn, ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), int(budget),
                                        _ptr(idx), _ptr(out), out_code, _ptr(lse), _ptr(workspace),
                                        0 if workspace is None else workspace.numel(),
                                        _stream_ptr(stream, q.device))
    _check(status, "ress_block_sparse_attn")
    return out, lse


def ress_block_drift(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor,
                     lse: torch.Tensor, block: int, drift: Optional[torch.Tensor] = None,
                     set_drift: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Stage 3: returns (drift [H, nb, nb - budget], set_drift [H, nb]) float32."""
    _check_inputs(q, k, v)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    budget = _check_idx(idx, h, nb, q.device)
    _check_buffer(lse, (h, n), torch.float32, q.device, "lse")
    if drift is None:
        drift = torch.empty((h, nb, max(nb - budget, 0)), dtype=torch.float32, device=q.device)
    if set_drift is None:
        set_drift = torch.empty((h, nb), dtype=torch.float32, device=q.device)
    _check_buffer(drift, (h, nb, max(nb - budget, 0)), torch.float32, q.device, "drift")
    _check_buffer(set_drift, (h, nb), torch.float32, q.device, "set_drift")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_attn_workspace_bytes(ctypes.byref(sh)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_block_drift, ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), int(budget),
                                  _ptr(idx), _ptr(lse), _ptr(drift) if drift.numel() else None,
                                  _ptr(set_drift), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(),
                                  _stream_ptr(stream, q.device))
    _check(status, "ress_block_drift")
    return drift, set_drift


def _layout(layout) -> ress_layout:
    """(tokens_per_view, real_tokens, special_tokens) -> ress_layout."""
    t, r, sp = (int(x) for x in layout)
    return ress_layout(t, r, sp)


def ress_select_blocks_layout(q: torch.Tensor, k: torch.Tensor, budget: int, block: int, layout,
                              idx: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Stage 1 with a per-view layout (tokens_per_view, real_tokens,
    special_tokens): returns idx [H, nb, budget] int32."""
    _check_inputs(q, k)
    sh = _shape_of(q, block)
    lay = _layout(layout)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    if idx is None:
        idx = torch.empty((h, nb, budget), dtype=torch.int32, device=q.device)
    _check_buffer(idx, (h, nb, budget), torch.int32, q.device, "idx")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_select_workspace_bytes(ctypes.byref(sh), ctypes.c_float(0.0)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_select_blocks_layout, ctypes.byref(sh), ctypes.byref(lay),
                 _ptr(q), _ptr(k), int(budget), _ptr(idx), _ptr(workspace), workspace.numel(),
                 _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks_layout")
    return idx


def ress_block_sparse_attn_layout(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  idx: torch.Tensor, block: int, layout,
                                  out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                                  workspace: Optional[torch.Tensor] = None,
                                  stream: Optional[torch.cuda.Stream] = None,
                                  out_dtype: Optional[torch.dtype] = None
                                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Stage 2 with a per-view layout: returns (out [N, H, 64], lse [H, N])."""
    _check_inputs(q, k, v)
    sh = _shape_of(q, block)
    lay = _layout(layout)
    n, h = q.shape[0], q.shape[1]
    budget = _check_idx(idx, h, n // block, q.device)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    out_code = RESS_F32 if out.dtype == torch.float32 else (
        RESS_BF16 if out.dtype == torch.bfloat16 else None)
    if out_code is None:
        raise TypeError(f"unsupported output dtype {out.dtype}")
    _check_buffer(out, q.shape, out.dtype, q.device, "out")
    if lse is None and want_lse:
        lse = torch.empty((h, n), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_buffer(lse, (h, n), torch.float32, q.device, "lse")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_attn_layout_workspace_bytes(ctypes.byref(sh), ctypes.byref(lay), out_code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_block_sparse_attn_layout, ctypes.byref(sh), ctypes.byref(lay),
                 _ptr(q), _ptr(k), _ptr(v), int(budget), _ptr(idx), _ptr(out), out_code,
                 _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                 _stream_ptr(stream, q.device))
    _check(status, "ress_block_sparse_attn_layout")
    return out, lse


def ress_block_drift_layout(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor,
                            lse: torch.Tensor, block: int, layout,
                            drift: Optional[torch.Tensor] = None,
                            set_drift: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Stage 3 with a per-view layout: returns (drift [H, nb, nb - budget], set_drift [H, nb])."""
    _check_inputs(q, k, v)
    sh = _shape_of(q, block)
    lay = _layout(layout)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    budget = _check_idx(idx, h, nb, q.device)
    _check_buffer(lse, (h, n), torch.float32, q.device, "lse")
    if drift is None:
        drift = torch.empty((h, nb, max(nb - budget, 0)), dtype=torch.float32, device=q.device)
    if set_drift is None:
        set_drift = torch.empty((h, nb), dtype=torch.float32, device=q.device)
    _check_buffer(drift, (h, nb, max(nb - budget, 0)), torch.float32, q.device, "drift")
    _check_buffer(set_drift, (h, nb), torch.float32, q.device, "set_drift")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_attn_workspace_bytes(ctypes.byref(sh)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_block_drift_layout, ctypes.byref(sh), ctypes.byref(lay),
                 _ptr(q), _ptr(k), _ptr(v), int(budget), _ptr(idx), _ptr(lse),
                 _ptr(drift) if drift.numel() else None, _ptr(set_drift), _ptr(workspace),
                 0 if workspace is None else workspace.numel(), _stream_ptr(stream, q.device))
    _check(status, "ress_block_drift_layout")
    return drift, set_drift


def ress_select_blocks_restore(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, budget: int,
                               block: int, rounds: int = 4, candidates: int = 8,
                               idx: Optional[torch.Tensor] = None,
                               drift_init: Optional[torch.Tensor] = None,
                               drift_final: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               stream: Optional[torch.cuda.Stream] = None
                               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Stage 1 by drift with restoration: returns (idx [H, nb, budget] int32,
    drift of the initial drop set [H, nb], drift of the result [H, nb])."""
    _check_inputs(q, k, v)
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    if idx is None:
        idx = torch.empty((h, nb, budget), dtype=torch.int32, device=q.device)
    if drift_init is None:
        drift_init = torch.empty((h, nb), dtype=torch.float32, device=q.device)
    if drift_final is None:
        drift_final = torch.empty((h, nb), dtype=torch.float32, device=q.device)
    _check_buffer(idx, (h, nb, budget), torch.int32, q.device, "idx")
    _check_buffer(drift_init, (h, nb), torch.float32, q.device, "drift_init")
    _check_buffer(drift_final, (h, nb), torch.float32, q.device, "drift_final")
    _check_workspace(workspace, q.device)
    need = int(lib.ress_restore_workspace_bytes(ctypes.byref(sh)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    status = _on(q.device, lib.ress_select_blocks_restore, ctypes.byref(sh), _ptr(q), _ptr(k),
                 _ptr(v), int(budget), int(rounds), int(candidates), _ptr(idx), _ptr(drift_init),
                 _ptr(drift_final), _ptr(workspace), workspace.numel(),
                 _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks_restore")
    return idx, drift_init, drift_final


def vasc_pairs(nb: int) -> int:
    """Memory entries per head of the VASC selection: one per fixed pair of
    neighbouring key blocks, the last a singleton when nb is odd."""
    return (nb + 1) // 2


def ress_select_blocks_vasc(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
                            budgets, block: int, capacity: Optional[int] = None,
                            memory: Optional[torch.Tensor] = None, value_aware: bool = True,
                            reset: Optional[bool] = None, idx: Optional[torch.Tensor] = None,
                            demand: Optional[torch.Tensor] = None,
                            service: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor],
                                       Optional[torch.Tensor]]:
    """VASC selection of one global layer: returns (idx [H, nb, capacity]
    int32, memory [H, pairs] float32 settled in place, demand, service).

    ``budgets`` holds c_h for every head (an int applies to all); capacity
    defaults to the largest.  Without ``memory`` a zeroed one is made and
    ``reset`` defaults to True (the first global layer); with one, ``reset``
    defaults to False.  ``demand`` / ``service`` ([H, pairs] float32) are
    filled when given.
    """
    _check_inputs(q, k, v)
    if value_aware and v is None:
        raise ValueError("the value contrast needs v (or value_aware=False)")
    sh = _shape_of(q, block)
    n, h = q.shape[0], q.shape[1]
    nb = n // block
    pairs = vasc_pairs(nb)
    per_head = [int(budgets)] * h if isinstance(budgets, int) else [int(b) for b in budgets]
    if len(per_head) != h:
        raise ValueError(f"budgets needs {h} entries, got {len(per_head)}")
    cap = max(per_head) if capacity is None else int(capacity)
    if memory is None:
        memory = torch.zeros((h, pairs), dtype=torch.float32, device=q.device)
        reset = True if reset is None else reset
    reset = False if reset is None else reset
    if idx is None:
        idx = torch.empty((h, nb, max(cap, 1)), dtype=torch.int32, device=q.device)
    _check_buffer(memory, (h, pairs), torch.float32, q.device, "memory")
    _check_buffer(idx, (h, nb, max(cap, 1)), torch.int32, q.device, "idx")
    for name, t in (("demand", demand), ("service", service)):
        if t is not None:
            _check_buffer(t, (h, pairs), torch.float32, q.device, name)
    _check_workspace(workspace, q.device)
    need = int(lib.ress_vasc_workspace_bytes(ctypes.byref(sh)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    host_budgets = (ctypes.c_int32 * h)(*per_head)
    status = _on(q.device, lib.ress_select_blocks_vasc, ctypes.byref(sh), _ptr(q), _ptr(k),
                 _ptr(v), ctypes.cast(host_budgets, _P), cap, int(bool(value_aware)),
                 int(bool(reset)), _ptr(memory), _ptr(idx), _ptr(demand), _ptr(service),
                 _ptr(workspace), workspace.numel(), _stream_ptr(stream, q.device))
    _check(status, "ress_select_blocks_vasc")
    return idx, memory, demand, service


def ress_validate_idx(idx: torch.Tensor, n: int, block: int,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Checks idx [H, nb, budget] on the device (in range, strictly ascending
    rows); a bad row shows up in ress_check_device_errors (RESS_ERR_BAD_INDEX,
    detail 80 out of range, 81 repeated block, 82 not ascending)."""
    if idx.dim() != 3:
        raise ValueError(f"idx must be [H, nb, budget], got {tuple(idx.shape)}")
    h = idx.shape[0]
    _check_idx(idx, h, n // block, idx.device)
    sh = make_shape(n, h, block, torch.bfloat16)
    status = _on(idx.device, lib.ress_validate_idx, ctypes.byref(sh), int(idx.shape[2]), _ptr(idx),
                 _stream_ptr(stream, idx.device))
    _check(status, "ress_validate_idx")


# --------------------------------------------------------------------------------------------
# Keys of another length, and the 8-bit cache
# --------------------------------------------------------------------------------------------
try:   # the common calls in C++ (csrc/ress_call.cpp); without it all of them are made below
    from . import _ress_call as _call
    from .build import call_tag
    _call.init(LIB_PATH, call_tag())
except ImportError:
    _call = None


def _int32(**numbers) -> None:
    """ctypes cuts integers to their low 32 bits without a word."""
    for name, x in numbers.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name} must fit in 32 bits, got {x}")


@functools.lru_cache(maxsize=1024)
def _cross_shape(nq: int, nk: int, seqs: int, heads: int, kv_heads: int, head_dim: int,
                 q_stride: int, k_stride: int, v_stride: int):
    _int32(sequences=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    sh = ctypes.byref(ress_cross_shape(nq, nk, seqs, heads, kv_heads, head_dim, RESS_BF16,
                                       q_stride, k_stride, v_stride))
    return (sh, int(lib.ress_cross_workspace_bytes(sh)),
            int(lib.ress_cross_bwd_workspace_bytes(sh)))


@functools.lru_cache(maxsize=1024)
def _cache_shape(pages: int, page: int, kv_heads: int, head_dim: int, requests: int,
                 max_pages: int):
    _int32(pages=pages, page=page, kv_heads=kv_heads, head_dim=head_dim, requests=requests,
           max_pages=max_pages)
    return ctypes.byref(ress_cache_shape(pages, page, kv_heads, head_dim, requests, max_pages))


@functools.lru_cache(maxsize=1024)
def _cache_attn_bytes(pages: int, page: int, kv_heads: int, head_dim: int, requests: int,
                      max_pages: int, heads: int, tokens: int) -> int:
    _int32(heads=heads, tokens=tokens)
    sh = _cache_shape(pages, page, kv_heads, head_dim, requests, max_pages)
    return int(lib.ress_cache_attn_workspace_bytes(sh, heads, tokens))


def _run_on(device: torch.device, stream: Optional[torch.cuda.Stream], fn, *args) -> int:
    """``_on`` with the stream as the last argument, without a device switch
    where ``device`` is current already."""
    raw = (torch._C._cuda_getCurrentRawStream(device.index) if stream is None
           else stream.cuda_stream)
    if device.index == torch._C._cuda_getDevice():
        return fn(*args, raw)
    with torch.cuda.device(device):
        return fn(*args, raw)


def _new(shape, dtype: torch.dtype, like: torch.Tensor,
         stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new tensor on the device of ``like`` for a call on ``stream``: allocated
    on that stream, so that the caching allocator hands its memory to no one
    before the call is done."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _expect(t: torch.Tensor, shape, dtype: torch.dtype, device: torch.device, name: str) -> int:
    """``_check_buffer`` and ``_ptr`` in one, for calls that take microseconds
    (``device`` is known to be a CUDA device, or the checks below say so)."""
    if (t.shape != shape or t.dtype is not dtype or t.device != device
            or not t.is_contiguous() or device.type != "cuda"):
        _check_buffer(t, shape, dtype, device, name)
        return _ptr(t)
    return t.data_ptr()


def _scratch(workspace: Optional[torch.Tensor], need: int, like: torch.Tensor,
             stream: Optional[torch.cuda.Stream]) -> Tuple[Optional[int], int, object]:
    """(pointer, bytes, owner) of a call's workspace."""
    if workspace is not None:
        _check_workspace(workspace, like.device)
        return _ptr(workspace), workspace.numel(), workspace
    if need == 0:
        return None, 0, None
    ws = _new((need,), torch.uint8, like, stream)
    return ws.data_ptr(), need, ws


def _token_rows(t: torch.Tensor, name: str) -> int:
    """Elements between the token rows of [n, heads, d] (0: dense).  Rows may
    be slices of wider ones; the values of a row stand together."""
    if t.is_contiguous():
        return 0
    s0, s1, s2 = t.stride()
    _, h, d = t.shape
    if s2 != 1 or (h > 1 and s1 != d) or s0 < h * d:
        raise ValueError(f"{name}: the heads of a token must stand together")
    return s0


def _check_rows(t: torch.Tensor, name: str, device: torch.device, heads: Optional[int] = None,
                dtypes=(torch.bfloat16,)) -> None:
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, d]")
    if heads is not None and t.shape[1] != heads:
        raise ValueError(f"{name} has {t.shape[1]} heads, expected {heads}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")


def _seq_arrays(q_offsets, kv_offsets, q_lens, kv_lens, device: torch.device):
    """Checks the arrays of a packed batch; returns the number of sequences and
    the four pointers."""
    if (q_offsets is None) != (kv_offsets is None):
        raise ValueError("q_offsets and kv_offsets come together")
    seqs, i32, qo, ko, ql, kl = 1, torch.int32, None, None, None, None
    if q_offsets is not None:
        if q_offsets.dim() != 1 or q_offsets.shape[0] < 2:
            raise ValueError("q_offsets must be [sequences + 1]")
        seqs = q_offsets.shape[0] - 1
        qo = _expect(q_offsets, (seqs + 1,), i32, device, "q_offsets")
        ko = _expect(kv_offsets, (seqs + 1,), i32, device, "kv_offsets")
    if q_lens is not None:
        ql = _expect(q_lens, (seqs,), i32, device, "q_lens")
    if kv_lens is not None:
        kl = _expect(kv_lens, (seqs,), i32, device, "kv_lens")
    return seqs, qo, ko, ql, kl


def _cross_inputs(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens):
    """(shape and workspace sizes, pointers of q to kv_lens)."""
    device = q.device
    _check_rows(q, "q", device)
    _check_rows(k, "k", device)
    if v.shape != k.shape:
        raise ValueError(f"v has shape {tuple(v.shape)}, k has {tuple(k.shape)}")
    _check_rows(v, "v", device)
    nq, h, d = q.shape
    nk, hk, dk = k.shape
    if dk != d:
        raise ValueError(f"k has head dim {dk}, q has {d}")
    seqs, *arrays = _seq_arrays(q_offsets, kv_offsets, q_lens, kv_lens, device)
    return (_cross_shape(nq, nk, seqs, h, hk, d, _token_rows(q, "q"), _token_rows(k, "k"),
                         _token_rows(v, "v")),
            (q.data_ptr(), k.data_ptr(), v.data_ptr()), arrays)


def ress_cross_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q_offsets: Optional[torch.Tensor] = None,
                    kv_offsets: Optional[torch.Tensor] = None,
                    q_lens: Optional[torch.Tensor] = None, kv_lens: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of q [nq, H, 64] over k, v [nk, Hk, 64] (bf16, Hk divides H):
    returns (out [nq, H, 64], lse [H, nq] float32 or None).

    ``q_offsets`` / ``kv_offsets`` ([sequences + 1] int32) pack several
    sequences; ``q_lens`` / ``kv_lens`` ([sequences] int32) mark the rows of
    each that are not padding.  Token rows of q, k and v may be slices of
    wider rows.  Rows of no sequence are left as they were (undefined in a
    tensor that this call allocates).  Nothing is recorded for autograd, whatever
    the inputs ask for: ress_cross_attn_bwd gives the gradients.  See
    include/ress.h."""
    if _call is not None and out is lse is workspace is stream is None:
        done = _call.cross_attn(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens, bool(want_lse))
        if done is not None:
            return done
    (sh, need, _), qkv, arrays = _cross_inputs(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens)
    device, (nq, h, _) = q.device, q.shape
    out, out_ptr, lse, lse_ptr = _attn_outputs(q, out, lse, want_lse, stream)
    ws, size, owner = _scratch(workspace, need, q, stream)
    _check(_run_on(device, stream, lib.ress_cross_attn, sh, *qkv, *arrays, out_ptr, lse_ptr, ws,
                   size), "ress_cross_attn")
    return out, lse


def _attn_outputs(q, out, lse, want_lse, stream):
    """The output tensors of an attention call over q and their pointers."""
    nq, h, _ = q.shape
    if out is None:
        out = (torch.empty_like(q) if stream is None and q.is_contiguous()
               else _new(q.shape, q.dtype, q, stream))
        out_ptr = out.data_ptr()
    else:
        out_ptr = _expect(out, q.shape, q.dtype, q.device, "out")
    if lse is not None:
        return out, out_ptr, lse, _expect(lse, (h, nq), torch.float32, q.device, "lse")
    if not want_lse:
        return out, out_ptr, None, None
    lse = _new((h, nq), torch.float32, q, stream)
    return out, out_ptr, lse, lse.data_ptr()


def ress_cross_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                        lse: torch.Tensor, dout: torch.Tensor,
                        q_offsets: Optional[torch.Tensor] = None,
                        kv_offsets: Optional[torch.Tensor] = None,
                        q_lens: Optional[torch.Tensor] = None,
                        kv_lens: Optional[torch.Tensor] = None,
                        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                        dv: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of ress_cross_attn: returns (dq, dk, dv) in the shapes of q,
    k and v, from what the forward call returned and dout [nq, H, 64]."""
    if _call is not None and dq is dk is dv is workspace is stream is None:
        done = _call.cross_attn_bwd(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens, out, lse, dout)
        if done is not None:
            return done
    (sh, _, need), qkv, arrays = _cross_inputs(q, k, v, q_offsets, kv_offsets, q_lens, kv_lens)
    device, (nq, h, _) = q.device, q.shape
    saved = (_expect(out, q.shape, q.dtype, device, "out"),
             _expect(lse, (h, nq), torch.float32, device, "lse"),
             _expect(dout, q.shape, q.dtype, device, "dout"))
    grads, ptrs = [], []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, k)):
        if t is None:
            t = _new(like.shape, like.dtype, q, stream)
            ptrs.append(t.data_ptr())
        else:
            ptrs.append(_expect(t, like.shape, like.dtype, device, name))
        grads.append(t)
    ws, size, owner = _scratch(workspace, need, q, stream)
    _check(_run_on(device, stream, lib.ress_cross_attn_bwd, sh, *qkv, *saved, *arrays, *ptrs, ws,
                   size), "ress_cross_attn_bwd")
    return grads[0], grads[1], grads[2]


class ress_cache(NamedTuple):
    """A paged 8-bit cache: codes [pages, Hk, page, 64] float8_e4m3fn and
    scales [pages, Hk] float32 of the keys and the values."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def make_cache(pages: int, kv_heads: int, page: int, device="cuda") -> ress_cache:
    """An empty pool of ``pages`` pages of ``page`` (64 or 128) tokens."""
    codes = [torch.zeros((pages, kv_heads, page, 64), dtype=torch.float8_e4m3fn, device=device)
             for _ in range(2)]
    return ress_cache(*codes, *(torch.zeros((pages, kv_heads), dtype=torch.float32, device=device)
                                for _ in range(2)))


def _check_cache(cache: ress_cache, device: torch.device):
    """(pages, page, kv_heads, head_dim) of a cache whose parts fit together, and
    the pointers of its parts."""
    k, v, k_scale, v_scale = cache
    if k.dim() != 4:
        raise ValueError("cache.k must be [pages, heads, page, d]")
    shape = k.shape
    pages, heads, page, d = shape
    return (pages, page, heads, d), (
        _expect(k, shape, torch.float8_e4m3fn, device, "cache.k"),
        _expect(v, shape, torch.float8_e4m3fn, device, "cache.v"),
        _expect(k_scale, (pages, heads), torch.float32, device, "cache.k_scale"),
        _expect(v_scale, (pages, heads), torch.float32, device, "cache.v_scale"))


def ress_cache_plan(added: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                    free_pages: torch.Tensor, cursor: torch.Tensor, page: int, tokens: int,
                    pages: Optional[int] = None, offsets: Optional[torch.Tensor] = None,
                    slots: Optional[torch.Tensor] = None,
                    new_lengths: Optional[torch.Tensor] = None,
                    new_cursor: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Block tables and slot maps for ``added`` [R] tokens behind ``lengths``
    [R] cached ones: extends ``table`` [R, max_pages] in place from
    ``free_pages[cursor:]`` and returns (offsets [R + 1], slots [tokens],
    new_lengths [R], new_cursor [1]), all int32 (parts of one allocation unless
    any is passed in).  ``tokens`` is the length of the slot map (at least the sum of ``added``); ``pages`` bounds the page ids
    (default: the largest pool).  See include/ress.h."""
    if _call is not None and offsets is slots is new_lengths is new_cursor is stream is None:
        done = _call.cache_plan(added, lengths, table, free_pages, cursor, page, tokens, pages)
        if done is not None:
            return done
    device, i32 = added.device, torch.int32
    if added.dim() != 1 or table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("added must be [R], table [R, max_pages], free_pages [n]")
    (r, width), page, tokens = table.shape, operator.index(page), operator.index(tokens)
    limit = (2 ** 31 - 1) // max(page, 1) if pages is None else operator.index(pages)
    _int32(page=page, pages=limit, tokens=tokens, free_pages=free_pages.shape[0])
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    ins = (_expect(added, (r,), i32, device, "added"),
           _expect(lengths, (r,), i32, device, "lengths"),
           _expect(table, (r, width), i32, device, "table"),
           _expect(free_pages, free_pages.shape, i32, device, "free_pages"),
           free_pages.shape[0], _expect(cursor, (1,), i32, device, "cursor"))
    sizes = (r + 1, tokens, r, 1)
    if offsets is slots is new_lengths is new_cursor is None:
        made = _new((sum(sizes),), i32, added, stream).split_with_sizes(sizes)
        ptrs = [t.data_ptr() for t in made]
    else:
        made, ptrs = [], []
        for name, t, n in zip(("offsets", "slots", "new_lengths", "new_cursor"),
                              (offsets, slots, new_lengths, new_cursor), sizes):
            made.append(_new((n,), i32, added, stream) if t is None else t)
            ptrs.append(_expect(made[-1], (n,), i32, device, name))
    _check(_run_on(device, stream, lib.ress_cache_plan,
                   _cache_shape(limit, page, 1, 64, r, width), *ins, tokens, *ptrs),
           "ress_cache_plan")
    return made[0], made[1], made[2], made[3]


def ress_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: ress_cache,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Writes the tokens k, v [tokens, Hk, 64] (bf16 or float32; rows may be
    slices of wider ones) into the cells ``slots`` [tokens] int32 of ``cache``,
    in place; negative slots skip their token.  See include/ress.h."""
    if _call is not None and stream is None and _call.cache_append(k, v, slots, *cache):
        return
    device = k.device
    (pages, page, heads, d), parts = _check_cache(cache, device)
    _check_rows(k, "k", device, heads, (torch.bfloat16, torch.float32))
    if v.shape != k.shape or k.shape[2] != d:
        raise ValueError(f"k and v must be [tokens, {heads}, {d}], got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    _check_rows(v, "v", device, heads, (k.dtype,))
    n = k.shape[0]
    _int32(tokens=n)
    _check(_run_on(device, stream, lib.ress_cache_append,
                   _cache_shape(pages, page, heads, d, 1, 1), k.data_ptr(), v.data_ptr(),
                   RESS_F32 if k.dtype is torch.float32 else RESS_BF16, _token_rows(k, "k"),
                   _token_rows(v, "v"), _expect(slots, (n,), torch.int32, device, "slots"), n,
                   *parts), "ress_cache_append")


def ress_cache_attn(q: torch.Tensor, cache: ress_cache, table: torch.Tensor,
                    lengths: torch.Tensor, offsets: torch.Tensor, step: int = 0,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of the newest tokens q [T, H, 64] (bf16) of every request over
    its cached tokens: returns (out [T, H, 64], lse [H, T] float32 or None).

    ``offsets`` [R + 1] packs the query rows of the requests, ``lengths`` [R]
    counts their cached tokens (the queries' own among them), ``table`` [R,
    max_pages] names their pages.  ``step`` 0: every query sees all of its
    request; 1: causal; n: groups of n tokens see themselves and the earlier
    groups.  See include/ress.h."""
    if _call is not None and out is lse is workspace is stream is None:
        done = _call.cache_attn(q, *cache, table, lengths, offsets, step, bool(want_lse))
        if done is not None:
            return done
    device, i32 = q.device, torch.int32
    (pages, page, heads, d), parts = _check_cache(cache, device)
    _check_rows(q, "q", device)
    n, h, dq = q.shape
    if dq != d:
        raise ValueError(f"q has head dim {dq}, the cache {d}")
    if table.dim() != 2:
        raise ValueError("table must be [requests, max_pages]")
    (r, width), step = table.shape, operator.index(step)
    _int32(step=step)
    arrays = (_expect(table, (r, width), i32, device, "table"),
              _expect(lengths, (r,), i32, device, "lengths"),
              _expect(offsets, (r + 1,), i32, device, "offsets"))
    out, out_ptr, lse, lse_ptr = _attn_outputs(q, out, lse, want_lse, stream)
    ws, size, owner = _scratch(workspace, _cache_attn_bytes(pages, page, heads, d, r, width, h, n),
                               q, stream)
    _check(_run_on(device, stream, lib.ress_cache_attn,
                   _cache_shape(pages, page, heads, d, r, width), h, n, q.data_ptr(),
                   _token_rows(q, "q"), *parts, *arrays, step, out_ptr, lse_ptr, ws, size),
           "ress_cache_attn")
    return out, lse


def ress_check_device_errors(stream: Optional[torch.cuda.Stream] = None,
                             device: Optional[torch.device] = None) -> Tuple[int, int]:
    """Synchronise and return (status, detail) of the device error flag (cleared)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    detail = ctypes.c_int32(0)
    status = _on(dev, lib.ress_check_device_errors, _stream_ptr(stream, dev), ctypes.byref(detail))
    return int(status), int(detail.value)
