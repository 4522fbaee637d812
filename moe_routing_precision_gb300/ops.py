"""Thin Python binding of ``include/moe_route.h`` (argument marshalling only).

Every function checks dtype, device, shape and contiguity, allocates any
output the caller did not pass (PyTorch is the memory manager), and calls the
C ABI with raw device pointers and the current CUDA stream.  All computation
happens in the CUDA kernels of ``libmoe_route.so``; there is no fallback: if
the library is missing or the tensors are not on a CUDA device, the call
raises.

``stream`` (a torch.cuda.Stream or a raw handle; None: the current one) is where
a call's kernels run.  What the call allocates belongs to that stream; tensors
that the caller passes are the caller's to order and to keep.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from ._build import lib_path

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_DEVICE = range(5)
MOE_WEIGHTS_NONE, MOE_WEIGHTS_SOFTMAX_TOPK = 0, 1
MOE_OUT_BF16, MOE_OUT_F32 = 0, 1
MOE_DEVERR_EXPERT_RANGE, MOE_DEVERR_POS_RANGE, MOE_DEVERR_DUPLICATE_EXPERT = 0x1, 0x2, 0x4
MOE_DEVERR_ROWS_SHORT, MOE_DEVERR_TIMEOUT, MOE_DEVERR_BOUNDS = 0x8, 0x10, 0x20
GROUP = 128
SF_COLMAJOR, SF_POW2, SF_UE8M0 = 0x1, 0x2, 0x4

# Every symbol declared in include/moe_route.h, with its ctypes signature.
_P = ctypes.c_void_p
_i64, _i32, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
SIGNATURES = {
    "moe_topk_gate": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _i32, _P]),
    "moe_route_map_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "moe_route_map": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _P, _P, _P, _sz, _P]),
    "moe_route_map_noalloc": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _P, _P, _P]),
    "moe_expand_cast_fp8": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _i64, _P, _P, _i32, _P]),
    "moe_route_map_aligned": (ctypes.c_int, [_P, _i64, _i32, _i32, _i32, _i64, _P, _P, _P, _P,
                                             _P, _sz, _P]),
    "moe_expand_cast_fp8_padded": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _i64, _P, _P,
                                                  _i32, _P]),
    "swiglu_cast_fp8": (ctypes.c_int, [_P, _i64, _i32, _P, _P, _i32, _P]),
    "moe_expand_cast_fp8_ex": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _i64, _P, _P,
                                              ctypes.c_uint32, _i64, _P, ctypes.c_size_t, _i32,
                                              _P]),
    "moe_expand_cast_fp8_ex_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, ctypes.c_uint32]),
    "moe_expand_cast_fp4": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _P, _i64, _P, _P,
                                           ctypes.c_uint32, _i64, _P, ctypes.c_size_t, _i32, _P]),
    "moe_expand_cast_fp4_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, _i32,
                                                              ctypes.c_uint32]),
    "swiglu_cast_fp4": (ctypes.c_int, [_P, _i64, _i32, _P, _P, ctypes.c_uint32, _i64, _i32,
                                       ctypes.c_float, _P, _P, _i32, _P]),
    "moe_route_expand_cast_fp8": (ctypes.c_int, [_P, _i64, _i32, _i32, _P, _i32, _P, _P, _P, _P,
                                                 _P, _P, _P, _P, _P, ctypes.c_size_t, _i32, _i32,
                                                 _P]),
    "moe_route_expand_cast_fp8_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, _i32]),
    "moe_debug_set": (ctypes.c_int, [_i32, _i64]),
    "moe_debug_cvt": (ctypes.c_int, [_i32, _P, _P, _i64, _P]),
    "swiglu_cast_fp8_ex": (ctypes.c_int, [_P, _i64, _i32, _P, _P, ctypes.c_uint32, _i64, _i32,
                                          ctypes.c_float, _P, _P, _i32, _P]),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, _i64, _i32, _i32, _i64, _P, _i32, _P]),
    "moe_block_norm": (ctypes.c_int, [_P, _i32, _P, _i32, _i64, _i32, _P, _P, _i32, _i32,
                                      ctypes.c_float, _P, ctypes.c_float, _P, _P, _P, _P, _P]),
    "moe_block_norm_backward": (ctypes.c_int, [_P, _P, _P, _i32, _P, _i32, _i64, _i32, _P, _P,
                                               _i32, _i32, ctypes.c_float, _P, _P, _P, _P, _P, _P,
                                               _P, _P, _P, _sz, _P]),
    "moe_block_norm_backward_workspace_bytes": (_sz, [_i64, _i32]),
    "moe_balance_loss": (ctypes.c_int, [_P, _P, _i64, _i32, _i32, _i32, _P, _i32, _P, _P, _P, _P,
                                        _P, _P, _P, _sz, _P]),
    "moe_balance_loss_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "moe_balance_loss_backward": (ctypes.c_int, [_P, _i64, _i32, _i32, _i32, _P, _i32, _P, _P, _P,
                                                 _P, _P, _P, _P, _P, _P, _P]),
    "moe_combine_backward": (ctypes.c_int, [_P, _i32, _P, _P, _P, _P, _i64, _i32, _i32, _i64, _P,
                                            _P, _P]),
    "moe_expert_matvec_fp4": (ctypes.c_int, [_P, _i64, _P, _P, _i32, _i32, _P, _P, _i32, _i32,
                                             _i64, _i32, _i32, _i32, _P, _i32, _P]),
    "moe_peak_copy": (ctypes.c_int, [_P, _P, _sz, _P]),
    "moe_get_device_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_cuda_error_string": (ctypes.c_char_p, []),
    "moe_abi_version": (ctypes.c_int32, []),
    "moe_kernel_launch_count": (ctypes.c_uint64, []),
    "moe_debug_bounds_enabled": (ctypes.c_int32, []),
    "moe_debug_bounds_selftest": (ctypes.c_int, [_P]),
}

_lock = threading.Lock()
_lib = None


def load_library(path: str) -> ctypes.CDLL:
    """Load a build of the library at `path` and set every signature."""
    L = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib() -> ctypes.CDLL:
    """The loaded ``libmoe_route.so``, or ``libmoe_route_debug.so`` when the
    environment variable MOE_DEBUG_BOUNDS is 1 at the first call (raises if
    it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = lib_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with moe_routing_precision_gb300.build() "
                    "(nvcc, sm_103a); there is no CPU fallback")
            _lib = load_library(path)
    return _lib



class MoeError(RuntimeError):
    def __init__(self, rc: int, what: str):
        L = lib()
        msg = L.moe_status_string(rc).decode()
        if rc == MOE_ERR_CUDA:
            msg += f" ({L.moe_last_cuda_error_string().decode()})"
        super().__init__(f"{what}: {msg}")
        self.rc = rc


def _check(rc: int, what: str):
    if rc != MOE_OK:
        raise MoeError(rc, what)


# The current stream's handle without building a Stream object around it (2.9
# against 0.1 us per call on a Grace host), where this PyTorch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cuda_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and _cuda_device is not None:
            return _raw_stream(_cuda_device()) or None
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _dev(t: torch.Tensor, name: str, dtype, shape=None):
    if (type(t) is torch.Tensor and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device (no CPU path), got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t):
    return None if t is None else (t.data_ptr() or None)


def _on(stream, alloc):
    """`alloc` (torch.empty, ...) for a call whose kernels run on `stream`.

    On another stream than the current one a tensor is allocated as that stream's
    own: taken from the current stream's memory, its last user there might still
    be running, and a workspace or an output that the caller drops would go back
    to the current stream while the kernels are yet to write it.  The current
    stream is recorded on it, for the work the caller gives it there."""
    if stream is None:
        return alloc
    here = torch.cuda.current_stream()
    handle = _stream(stream) or 0
    if handle == here.cuda_stream:
        return alloc
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()

    def there(*args, **kwargs):
        with torch.cuda.stream(stream):
            t = alloc(*args, **kwargs)
        t.record_stream(here)
        return t
    return there


def _empty(shape, dtype, like, stream=None):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _on(stream, torch.empty)(shape, dtype=dtype, device=like.device)


# --------------------------------------------------------------------------

def topk_gate(scores: torch.Tensor, k: int, weights: bool = True, *, out_idx=None, out_w=None,
              stream=None):
    """Top-k experts per token (ties -> lower index) and softmax top-k weights.

    scores [T, E] float32 -> (idx [T, k] int32, w [T, k] float32 or None)."""
    _dev(scores, "scores", torch.float32)
    T, E = scores.shape
    idx = out_idx if out_idx is not None else _empty((T, k), torch.int32, scores, stream)
    _dev(idx, "out_idx", torch.int32, (T, k))
    w = None
    if weights:
        w = out_w if out_w is not None else _empty((T, k), torch.float32, scores, stream)
        _dev(w, "out_w", torch.float32, (T, k))
    rc = lib().moe_topk_gate(_ptr(scores), T, E, k, _ptr(idx), _ptr(w),
                             MOE_WEIGHTS_SOFTMAX_TOPK if weights else MOE_WEIGHTS_NONE,
                             _stream(stream))
    _check(rc, "moe_topk_gate")
    return idx, w


def route_map_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(lib().moe_route_map_workspace_bytes(T, E, k))


def route_map(topk_idx: torch.Tensor, num_experts: int, *, workspace=None, out=None, stream=None):
    """Stable token -> expert mapping.

    topk_idx [T, k] int32 -> (counts [E], offsets [E+1], pos [T, k],
    sorted_src [T*k]), all int32.  ``workspace`` (uint8, at least
    route_map_workspace_bytes bytes) is allocated when not given."""
    _dev(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    E = int(num_experts)
    if out is None:
        counts = _empty((E,), torch.int32, topk_idx, stream)
        offsets = _empty((E + 1,), torch.int32, topk_idx, stream)
        pos = _empty((T, k), torch.int32, topk_idx, stream)
        src = _empty((T * k,), torch.int32, topk_idx, stream)
    else:
        counts, offsets, pos, src = out
    _dev(counts, "counts", torch.int32, (E,))
    _dev(offsets, "offsets", torch.int32, (E + 1,))
    _dev(pos, "pos", torch.int32, (T, k))
    _dev(src, "sorted_src", torch.int32, (T * k,))
    need = route_map_workspace_bytes(T, E, k)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, topk_idx, stream)
    _dev(workspace, "workspace", torch.uint8)
    rc = lib().moe_route_map(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(pos),
                             _ptr(src), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "moe_route_map")
    return counts, offsets, pos, src


def route_map_aligned(topk_idx: torch.Tensor, num_experts: int, align: int,
                      num_rows: int | None = None, *, workspace=None, stream=None):
    """Route map into a padded layout: each expert's segment rounded up to a
    multiple of `align` rows.  num_rows defaults to T*k + E*(align-1), which
    always suffices.  -> (counts [E], offsets [E+1] padded, pos [T, k],
    sorted_src [num_rows], -1 on padding rows), all int32."""
    _dev(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    E = int(num_experts)
    R = T * k + E * (align - 1) if num_rows is None else int(num_rows)
    counts = _empty((E,), torch.int32, topk_idx, stream)
    offsets = _empty((E + 1,), torch.int32, topk_idx, stream)
    pos = _empty((T, k), torch.int32, topk_idx, stream)
    src = _empty((R,), torch.int32, topk_idx, stream)
    need = route_map_workspace_bytes(T, E, k)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, topk_idx, stream)
    _dev(workspace, "workspace", torch.uint8)
    rc = lib().moe_route_map_aligned(_ptr(topk_idx), T, E, k, int(align), R, _ptr(counts),
                                     _ptr(offsets), _ptr(pos), _ptr(src), _ptr(workspace),
                                     workspace.numel(), _stream(stream))
    _check(rc, "moe_route_map_aligned")
    return counts, offsets, pos, src


def expand_cast_fp8_padded(x: torch.Tensor, pos: torch.Tensor, sorted_src: torch.Tensor, *,
                           out=None, out_sf=None, stream=None):
    """expand_cast_fp8 into a padded layout of len(sorted_src) rows, zeroing
    (codes and scales) every row whose sorted_src entry is negative."""
    _dev(x, "x", torch.bfloat16)
    _dev(pos, "pos", torch.int32)
    _dev(sorted_src, "sorted_src", torch.int32)
    T, H = x.shape
    k = pos.shape[1]
    R = sorted_src.shape[0]
    q = out if out is not None else _empty((R, H), torch.uint8, x, stream)
    sf = out_sf if out_sf is not None else _empty((R, H // GROUP), torch.float32, x, stream)
    _dev(q, "out", torch.uint8, (R, H))
    _dev(sf, "out_sf", torch.float32, (R, H // GROUP))
    rc = lib().moe_expand_cast_fp8_padded(_ptr(x), T, H, k, _ptr(pos), _ptr(sorted_src), R,
                                          _ptr(q), _ptr(sf), GROUP, _stream(stream))
    _check(rc, "moe_expand_cast_fp8_padded")
    return q, sf


def sf_empty(rows: int, G: int, flags: int, ld: int | None, like: torch.Tensor, stream=None):
    """Scale buffer of the layout `flags` names: f32 [rows, G] or [G, ld];
    uint8 [rows, G]; or packed words as uint8 [ceil(G/4), ld, 4]."""
    ld = rows if ld is None else ld
    if flags & SF_UE8M0:
        if flags & SF_COLMAJOR:
            return _empty(((G + 3) // 4, ld, 4), torch.uint8, like, stream), ld
        return _empty((rows, G), torch.uint8, like, stream), ld
    if flags & SF_COLMAJOR:
        return _empty((G, ld), torch.float32, like, stream), ld
    return _empty((rows, G), torch.float32, like, stream), ld


PATH_AUTO, PATH_FUSED, PATH_SEPARATE, PATH_REPLICATED, PATH_CHAINED = 0, 1, 2, 3, 4
DEBUG_WAIT_TIMEOUT_NS, DEBUG_SKIP_ROUTE_SIGNAL = 1, 2


def route_expand_cast_workspace(T: int, E: int, k: int, like: torch.Tensor,
                                stream=None) -> torch.Tensor:
    """A zero-filled workspace for route_expand_cast_fp8 (its first 256 bytes
    are the fused path's control words, which must start at zero)."""
    n = int(lib().moe_route_expand_cast_fp8_workspace_bytes(T, E, k))
    return _on(stream, torch.zeros)(max(n, 256), dtype=torch.uint8, device=like.device)


def route_expand_cast_fp8(scores: torch.Tensor, x: torch.Tensor, k: int, *, mode: int = PATH_AUTO,
                          workspace=None, out=None, stream=None):
    """topk_gate + route_map + expand_cast_fp8 in one call; mode PATH_AUTO,
    PATH_SEPARATE, PATH_FUSED (one cooperative launch), PATH_REPLICATED (one
    launch, routing repeated per block) or PATH_CHAINED (top-k with chunk
    ranks, a scan, the expand placing its own copies).  -> (topk_idx, topk_w,
    counts, offsets, pos, sorted_src, q, sf)."""
    _dev(scores, "scores", torch.float32)
    _dev(x, "x", torch.bfloat16)
    T, E = scores.shape
    H = x.shape[1]
    R = T * k
    idx, w = _empty((T, k), torch.int32, x, stream), _empty((T, k), torch.float32, x, stream)
    counts = _empty((E,), torch.int32, x, stream)
    offsets = _empty((E + 1,), torch.int32, x, stream)
    pos, src = _empty((T, k), torch.int32, x, stream), _empty((R,), torch.int32, x, stream)
    q, sf = (out if out is not None else
             (_empty((R, H), torch.uint8, x, stream),
              _empty((R, H // GROUP), torch.float32, x, stream)))
    if workspace is None:
        workspace = route_expand_cast_workspace(T, E, k, x, stream)
    rc = lib().moe_route_expand_cast_fp8(_ptr(scores), T, E, k, _ptr(x), H, _ptr(idx), _ptr(w),
                                         _ptr(counts), _ptr(offsets), _ptr(pos), _ptr(src),
                                         _ptr(q), _ptr(sf), _ptr(workspace), workspace.numel(),
                                         mode, GROUP, _stream(stream))
    _check(rc, "moe_route_expand_cast_fp8")
    return idx, w, counts, offsets, pos, src, q, sf


CVT_E4M3, CVT_E2M1 = 0, 1


def debug_cvt(values: torch.Tensor, fmt: int, out=None, stream=None) -> torch.Tensor:
    """The device's f32 -> E4M3 / E2M1 conversion of every value (one code
    per byte), as the cast kernels convert; for tests."""
    _dev(values, "values", torch.float32)
    out = out if out is not None else _empty(values.shape, torch.uint8, values, stream)
    _check(lib().moe_debug_cvt(fmt, _ptr(values), _ptr(out), values.numel(), _stream(stream)),
           "moe_debug_cvt")
    return out


def debug_set(key: int, value: int) -> None:
    _check(lib().moe_debug_set(key, int(value)), "moe_debug_set")


def expand_cast_fp8_ex_workspace_bytes(T: int, H: int, sf_flags: int) -> int:
    return int(lib().moe_expand_cast_fp8_ex_workspace_bytes(T, H, sf_flags))


def expand_cast_fp8_ex(x: torch.Tensor, pos: torch.Tensor, num_rows: int | None = None, *,
                       sorted_src=None, sf_flags: int = 0, sf_ld: int | None = None, out=None,
                       out_sf=None, workspace=None, stream=None):
    """expand_cast_fp8 with scale options (SF_COLMAJOR, SF_POW2, SF_UE8M0) and
    an optional zero-fill of the rows whose sorted_src entry is negative.
    workspace: None (direct scale stores), True (allocate one), or a uint8
    CUDA tensor; used with a column-major layout and sorted_src to write the
    scales in whole lines (sorted_src must be pos's inverse)."""
    _dev(x, "x", torch.bfloat16)
    _dev(pos, "pos", torch.int32)
    T, H = x.shape
    k = pos.shape[1]
    if sorted_src is not None:
        _dev(sorted_src, "sorted_src", torch.int32)
    R = (T * k if sorted_src is None else sorted_src.shape[0]) if num_rows is None else int(num_rows)
    if sf_ld is None and (sf_flags & SF_COLMAJOR):
        sf_ld = (R + 3) // 4 * 4
    q = out if out is not None else _empty((R, H), torch.uint8, x, stream)
    _dev(q, "out", torch.uint8, (R, H))
    if out_sf is None:
        out_sf, sf_ld = sf_empty(R, H // GROUP, sf_flags, sf_ld, x, stream)
    elif out_sf.device.type != "cuda" or not out_sf.is_contiguous():
        raise ValueError("out_sf must be a contiguous CUDA tensor")
    if workspace is True:
        n = expand_cast_fp8_ex_workspace_bytes(T, H, sf_flags)
        workspace = _empty((n,), torch.uint8, x, stream) if n > 0 else None
    ws_bytes = 0 if workspace is None else workspace.numel()
    rc = lib().moe_expand_cast_fp8_ex(_ptr(x), T, H, k, _ptr(pos), _ptr(sorted_src), R, _ptr(q),
                                      _ptr(out_sf), sf_flags, int(sf_ld or R), _ptr(workspace),
                                      ws_bytes, GROUP, _stream(stream))
    _check(rc, "moe_expand_cast_fp8_ex")
    return q, out_sf


def expand_cast_fp4(x: torch.Tensor, pos: torch.Tensor, num_rows: int | None = None, *,
                    group: int = 32, sorted_src=None, sf_flags: int = 0, sf_ld: int | None = None,
                    out=None, out_sf=None, workspace=None, stream=None):
    """Expand + per-group FP4 E2M1 cast -> (q [R, H/2] packed uint8, scales in
    the flagged layout).  workspace: None, True (allocate) or a uint8 CUDA
    tensor, for column-major scales written from sorted_src."""
    _dev(x, "x", torch.bfloat16)
    _dev(pos, "pos", torch.int32)
    T, H = x.shape
    k = pos.shape[1]
    if sorted_src is not None:
        _dev(sorted_src, "sorted_src", torch.int32)
    R = (T * k if sorted_src is None else sorted_src.shape[0]) if num_rows is None else int(num_rows)
    if sf_ld is None and (sf_flags & SF_COLMAJOR):
        sf_ld = (R + 3) // 4 * 4
    q = out if out is not None else _empty((R, H // 2), torch.uint8, x, stream)
    _dev(q, "out", torch.uint8, (R, H // 2))
    if out_sf is None:
        out_sf, sf_ld = sf_empty(R, H // group, sf_flags, sf_ld, x, stream)
    if workspace is True:
        n = int(lib().moe_expand_cast_fp4_workspace_bytes(T, H, group, sf_flags))
        workspace = _empty((n,), torch.uint8, x, stream) if n > 0 else None
    ws_bytes = 0 if workspace is None else workspace.numel()
    rc = lib().moe_expand_cast_fp4(_ptr(x), T, H, k, _ptr(pos), _ptr(sorted_src), R, _ptr(q),
                                   _ptr(out_sf), sf_flags, int(sf_ld or R), _ptr(workspace),
                                   ws_bytes, group, _stream(stream))
    _check(rc, "moe_expand_cast_fp4")
    return q, out_sf


def swiglu_cast_fp4(x: torch.Tensor, *, group: int = 32, clamp: float | None = None, weights=None,
                    clamp_count=None, sf_flags: int = 0, sf_ld: int | None = None, out=None,
                    out_sf=None, stream=None):
    """SwiGLU (optional clamp, per-row weight, clamp counter) then the
    per-group FP4 E2M1 cast -> (q [M, N/2] packed uint8, scales)."""
    _dev(x, "x", torch.bfloat16)
    M, N2 = x.shape
    N = N2 // 2
    if weights is not None:
        _dev(weights, "weights", torch.float32, (M,))
    if clamp_count is not None:
        _dev(clamp_count, "clamp_count", torch.int64, (1,))
    if sf_ld is None and (sf_flags & SF_COLMAJOR):
        sf_ld = (M + 3) // 4 * 4
    q = out if out is not None else _empty((M, N // 2), torch.uint8, x, stream)
    _dev(q, "out", torch.uint8, (M, N // 2))
    if out_sf is None:
        out_sf, sf_ld = sf_empty(M, N // group, sf_flags, sf_ld, x, stream)
    rc = lib().swiglu_cast_fp4(_ptr(x), M, N, _ptr(q), _ptr(out_sf), sf_flags, int(sf_ld or M),
                               int(clamp is not None), float(clamp or 0.0), _ptr(weights),
                               _ptr(clamp_count), group, _stream(stream))
    _check(rc, "swiglu_cast_fp4")
    return q, out_sf


def swiglu_cast_fp8_ex(x: torch.Tensor, *, clamp: float | None = None, weights=None,
                       clamp_count=None, sf_flags: int = 0, sf_ld: int | None = None, out=None,
                       out_sf=None, stream=None):
    """SwiGLU with optional clamp, per-row weight and clamp counter (an int64
    CUDA tensor of one element, added to), then the cast with scale options."""
    _dev(x, "x", torch.bfloat16)
    M, N2 = x.shape
    N = N2 // 2
    if weights is not None:
        _dev(weights, "weights", torch.float32, (M,))
    if clamp_count is not None:
        _dev(clamp_count, "clamp_count", torch.int64, (1,))
    if sf_ld is None and (sf_flags & SF_COLMAJOR):
        sf_ld = (M + 3) // 4 * 4
    q = out if out is not None else _empty((M, N), torch.uint8, x, stream)
    _dev(q, "out", torch.uint8, (M, N))
    if out_sf is None:
        out_sf, sf_ld = sf_empty(M, N // GROUP, sf_flags, sf_ld, x, stream)
    rc = lib().swiglu_cast_fp8_ex(_ptr(x), M, N, _ptr(q), _ptr(out_sf), sf_flags, int(sf_ld or M),
                                  int(clamp is not None), float(clamp or 0.0), _ptr(weights),
                                  _ptr(clamp_count), GROUP, _stream(stream))
    _check(rc, "swiglu_cast_fp8_ex")
    return q, out_sf


def expand_cast_fp8(x: torch.Tensor, pos: torch.Tensor, num_rows: int | None = None, *,
                    out=None, out_sf=None, stream=None):
    """Per-token E4M3 cast (one fp32 scale per 128 channels) written to the
    rows pos[t, j] of the expert-sorted buffers.

    x [T, H] bfloat16, pos [T, k] int32 -> (out [R, H] uint8 E4M3 codes,
    out_sf [R, H/128] float32); R = num_rows (default T*k)."""
    _dev(x, "x", torch.bfloat16)
    _dev(pos, "pos", torch.int32)
    T, H = x.shape
    k = pos.shape[1]
    if pos.shape[0] != T:
        raise ValueError("pos must have one row per token")
    R = T * k if num_rows is None else int(num_rows)
    q = out if out is not None else _empty((R, H), torch.uint8, x, stream)
    sf = out_sf if out_sf is not None else _empty((R, H // GROUP), torch.float32, x, stream)
    _dev(q, "out", torch.uint8, (R, H))
    _dev(sf, "out_sf", torch.float32, (R, H // GROUP))
    rc = lib().moe_expand_cast_fp8(_ptr(x), T, H, k, _ptr(pos), R, _ptr(q), _ptr(sf), GROUP,
                                   _stream(stream))
    _check(rc, "moe_expand_cast_fp8")
    return q, sf


def swiglu_cast_fp8(x: torch.Tensor, *, out=None, out_sf=None, stream=None):
    """silu(gate) * up in fp32, then the per-128-channel E4M3 cast.

    x [M, 2N] bfloat16 (gate | up) -> (out [M, N] uint8, out_sf [M, N/128] f32)."""
    _dev(x, "x", torch.bfloat16)
    M, N2 = x.shape
    N = N2 // 2
    q = out if out is not None else _empty((M, N), torch.uint8, x, stream)
    sf = out_sf if out_sf is not None else _empty((M, N // GROUP), torch.float32, x, stream)
    _dev(q, "out", torch.uint8, (M, N))
    _dev(sf, "out_sf", torch.float32, (M, N // GROUP))
    rc = lib().swiglu_cast_fp8(_ptr(x), M, N, _ptr(q), _ptr(sf), GROUP, _stream(stream))
    _check(rc, "swiglu_cast_fp8")
    return q, sf


def combine(y: torch.Tensor, topk_weights: torch.Tensor, pos: torch.Tensor,
            out_dtype=torch.bfloat16, *, out=None, stream=None):
    """out[t] = sum_j w[t, j] * y[pos[t, j]], fp32 accumulation in slot order.

    y [R, H] bfloat16, w [T, k] float32, pos [T, k] int32 ->
    out [T, H] bfloat16 (or float32)."""
    _dev(y, "y", torch.bfloat16)
    _dev(topk_weights, "topk_weights", torch.float32)
    _dev(pos, "pos", torch.int32, tuple(topk_weights.shape))
    R, H = y.shape
    T, k = pos.shape
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    o = out if out is not None else _empty((T, H), out_dtype, y, stream)
    _dev(o, "out", out_dtype, (T, H))
    rc = lib().moe_combine(_ptr(y), _ptr(topk_weights), _ptr(pos), T, H, k, R, _ptr(o),
                           MOE_OUT_F32 if out_dtype == torch.float32 else MOE_OUT_BF16,
                           _stream(stream))
    _check(rc, "moe_combine")
    return o


# --------------------------------------------------------------------------
# The operators around the routed experts.

DT_BF16, DT_F32 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_ELEMENT = range(4)
_GATE_ACT = {"none": 0, "sigmoid": 1}
_SCORE_FUNC = {"softmax": 0, "sigmoid": 1}
WSF_F32, WSF_UE8M0 = 0, 1


def _dt(t: torch.Tensor, name: str) -> int:
    """MOE_DT_* of a bfloat16 or float32 tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == torch.bfloat16:
        return DT_BF16
    if t.dtype == torch.float32:
        return DT_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _choice(value: str, table: dict, name: str) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _gate_kind(gate, T: int, H: int, block_dtype) -> int:
    """MOE_GATE_* from the gate's shape: [H] float32, [T, 1] float32, or
    [T, H] in the block's type."""
    if gate is None:
        return GATE_NONE
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dim() == 1:
        _dev(gate, "gate", torch.float32, (H,))
        return GATE_CHANNEL
    if gate.dim() == 2 and gate.shape[1] == 1 and gate.dtype == torch.float32:
        _dev(gate, "gate", torch.float32, (T, 1))
        return GATE_TOKEN
    _dev(gate, "gate", block_dtype, (T, H))
    return GATE_ELEMENT


def block_norm(residual: torch.Tensor, y: torch.Tensor | None = None, *, post_weight=None,
               gate=None, gate_act: str = "none", scale: float = 1.0, pre_weight=None,
               eps: float = 1e-6, block_dtype=None, out=None, stream=None):
    """The norms before and after a block, with its gate and residual scale:

        z = y * rstd_post * post_weight          (post_weight None: z = y)
        h = residual + scale * g * z             (y None: h is residual)
        n = h * rstd_pre * pre_weight            (pre_weight None: no n)

    with rstd = 1 / sqrt(mean(row^2) + eps) and g the gate: None, [H] or [T, 1]
    float32, or [T, H] in y's type; gate_act "none" or "sigmoid".  residual and
    h are [T, H] bfloat16 or float32, y and n [T, H] bfloat16 or float32
    (block_dtype, y's own by default, else bfloat16); weights are [H] float32.
    out: None or (h, n), where h may be residual itself (without y h is residual and
    out[0] is not used).
    -> (h, n, rstd_post, rstd_pre), None for what there is not."""
    sd = _dt(residual, "residual")
    T, H = _dev(residual, "residual", residual.dtype).shape
    if block_dtype is None:
        block_dtype = torch.bfloat16 if y is None else y.dtype
    if block_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("block_dtype must be bfloat16 or float32")
    if y is not None:
        _dev(y, "y", block_dtype, (T, H))
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need y")
    elif pre_weight is None:
        raise ValueError("nothing to do: neither y nor pre_weight given")
    if post_weight is not None:
        _dev(post_weight, "post_weight", torch.float32, (H,))
    if pre_weight is not None:
        _dev(pre_weight, "pre_weight", torch.float32, (H,))
    kind = GATE_NONE if gate is None else _gate_kind(gate, T, H, block_dtype)
    empty, empty_like = _on(stream, torch.empty), _on(stream, torch.empty_like)
    h, n = out if out is not None else (None, None)
    if y is None:
        h = residual
    elif h is None:
        h = empty_like(residual)
    else:
        _dev(h, "out[0]", residual.dtype, (T, H))
    if pre_weight is None:
        n = None
    elif n is None:
        n = (empty_like(y) if y is not None else
             empty((T, H), dtype=block_dtype, device=residual.device))
    else:
        _dev(n, "out[1]", block_dtype, (T, H))
    rp = rn = None
    if post_weight is not None:
        rp = empty((T,), dtype=torch.float32, device=residual.device)
    if pre_weight is not None:
        rn = empty((T,), dtype=torch.float32, device=residual.device)
    rc = lib().moe_block_norm(_ptr(residual), sd, _ptr(y),
                              DT_F32 if block_dtype == torch.float32 else DT_BF16, T, H,
                              _ptr(post_weight), _ptr(gate), kind,
                              _choice(gate_act, _GATE_ACT, "gate_act"), scale, _ptr(pre_weight),
                              eps, _ptr(h), _ptr(n), _ptr(rp), _ptr(rn), _stream(stream))
    _check(rc, "moe_block_norm")
    return h, n, rp, rn


@functools.lru_cache(maxsize=256)
def block_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(lib().moe_block_norm_backward_workspace_bytes(T, H))


def block_norm_backward(grad_h, grad_n, h: torch.Tensor, *, y=None, post_weight=None, gate=None,
                        gate_act: str = "none", scale: float = 1.0, pre_weight=None,
                        rstd_post=None, rstd_pre=None, workspace=None, stream=None):
    """Gradients of block_norm for grad_h (of h, or None) and grad_n (of n, or
    None without pre_weight), from the saved h, y and inverse norms.
    -> (grad_residual, grad_y, grad_post_weight, grad_gate, grad_pre_weight),
    None for what there is not; each in its tensor's type and shape."""
    sd = _dt(h, "h")
    T, H = _dev(h, "h", h.dtype).shape
    if grad_h is not None:
        _dev(grad_h, "grad_h", h.dtype, (T, H))
    if (pre_weight is None) != (grad_n is None) or (pre_weight is None) != (rstd_pre is None):
        raise ValueError("pre_weight, grad_n and rstd_pre go together")
    if (post_weight is None) != (rstd_post is None):
        raise ValueError("post_weight and rstd_post go together")
    block = y if y is not None else grad_n
    if block is None:
        raise ValueError("nothing to do: neither y nor grad_n given")
    bd = _dt(block, "y or grad_n")
    if y is not None:
        _dev(y, "y", block.dtype, (T, H))
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need y")
    if grad_n is not None:
        _dev(grad_n, "grad_n", block.dtype, (T, H))
    if post_weight is not None:
        _dev(post_weight, "post_weight", torch.float32, (H,))
        _dev(rstd_post, "rstd_post", torch.float32, (T,))
    if pre_weight is not None:
        _dev(pre_weight, "pre_weight", torch.float32, (H,))
        _dev(rstd_pre, "rstd_pre", torch.float32, (T,))
    kind = GATE_NONE if gate is None else _gate_kind(gate, T, H, block.dtype)
    empty_like = _on(stream, torch.empty_like)
    gr = empty_like(h)
    gy = None if y is None else empty_like(y)
    gpw = None if post_weight is None else empty_like(post_weight)
    gg = None if gate is None else empty_like(gate)
    gnw = None if pre_weight is None else empty_like(pre_weight)
    ws_bytes = block_norm_backward_workspace_bytes(T, H)
    if workspace is None:
        workspace = _empty((ws_bytes,), torch.uint8, h, stream)
    else:
        ws_bytes = _dev(workspace, "workspace", torch.uint8).numel()
    rc = lib().moe_block_norm_backward(
        _ptr(grad_h), _ptr(grad_n), _ptr(h), sd, _ptr(y), bd, T, H, _ptr(post_weight), _ptr(gate),
        kind, _choice(gate_act, _GATE_ACT, "gate_act"), scale, _ptr(pre_weight), _ptr(rstd_post),
        _ptr(rstd_pre), _ptr(gr), _ptr(gy), _ptr(gpw), _ptr(gg), _ptr(gnw), _ptr(workspace),
        ws_bytes, _stream(stream))
    _check(rc, "moe_block_norm_backward")
    return gr, gy, gpw, gg, gnw


def _sequences(seq_offsets, token_mask, T: int) -> int:
    """Checks of what the balance loss and its backward share; the sequences."""
    if seq_offsets is not None:
        _dev(seq_offsets, "seq_offsets", torch.int32)
        if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
            raise ValueError("seq_offsets must be [S + 1] with S >= 1")
    if token_mask is not None:
        if not isinstance(token_mask, torch.Tensor) or token_mask.dtype not in (torch.bool,
                                                                                torch.uint8):
            raise TypeError("token_mask must be a bool or uint8 tensor")
        _dev(token_mask, "token_mask", token_mask.dtype, (T,))
    return 1 if seq_offsets is None else seq_offsets.numel() - 1


@functools.lru_cache(maxsize=256)
def balance_loss_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return int(lib().moe_balance_loss_workspace_bytes(T, E, S))


def balance_loss(scores: torch.Tensor, topk_idx: torch.Tensor, *, score_func: str = "softmax",
                 seq_offsets=None, token_mask=None, workspace=None, stream=None):
    """Per-expert counts, balance loss and z-loss of the router per sequence.

    scores [T, E] float32 (-inf allowed), topk_idx [T, k] int32; seq_offsets
    [S+1] int32 (None: one sequence of all T tokens); token_mask [T] bool or
    uint8, zero where a token does not count (nor does one whose scores are all
    -inf or hold a NaN).  With p = softmax(scores), or
    sigmoid(scores) over its row sum:
        balance[i] = sum_e E counts[i,e] / (k n_i) * probs[i,e],  probs = mean p
        z[i]       = mean of logsumexp(scores)^2
    -> (balance [S], z [S], counts [S, E] int32, probs [S, E], tokens [S] int32)."""
    _dev(scores, "scores", torch.float32)
    T, E = scores.shape
    k = topk_idx.shape[1]
    _dev(topk_idx, "topk_idx", torch.int32, (T, k))
    S = _sequences(seq_offsets, token_mask, T)
    empty, dev = _on(stream, torch.empty), scores.device
    bal = empty((S,), dtype=torch.float32, device=dev)
    z = empty((S,), dtype=torch.float32, device=dev)
    counts = empty((S, E), dtype=torch.int32, device=dev)
    probs = empty((S, E), dtype=torch.float32, device=dev)
    tokens = empty((S,), dtype=torch.int32, device=dev)
    ws_bytes = balance_loss_workspace_bytes(T, E, S)
    if workspace is None and ws_bytes:
        workspace = _empty((ws_bytes,), torch.uint8, scores, stream)
    if workspace is not None:
        ws_bytes = _dev(workspace, "workspace", torch.uint8).numel()
    rc = lib().moe_balance_loss(_ptr(scores), _ptr(topk_idx), T, E, k,
                                _choice(score_func, _SCORE_FUNC, "score_func"), _ptr(seq_offsets),
                                S, _ptr(token_mask), _ptr(bal), _ptr(z), _ptr(counts),
                                _ptr(probs), _ptr(tokens), _ptr(workspace), ws_bytes,
                                _stream(stream))
    _check(rc, "moe_balance_loss")
    return bal, z, counts, probs, tokens


def balance_loss_backward(scores: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor,
                          grad_balance=None, grad_z=None, *, k: int | None = None,
                          score_func: str = "softmax", seq_offsets=None, token_mask=None,
                          topk_idx=None, topk_weights=None, grad_topk_weights=None, out=None,
                          stream=None):
    """The router's score gradient [T, E] float32: of balance_loss's two losses
    (grad_balance, grad_z [S] float32, or None) and, with grad_topk_weights
    [T, k], of topk_gate's softmax weights of the selected scores (topk_idx and
    topk_weights as topk_gate returned them).  counts and tokens as
    balance_loss returned them; k from topk_idx or, without it, given."""
    _dev(scores, "scores", torch.float32)
    T, E = scores.shape
    S = _sequences(seq_offsets, token_mask, T)
    _dev(counts, "counts", torch.int32, (S, E))
    _dev(tokens, "tokens", torch.int32, (S,))
    for name, g in (("grad_balance", grad_balance), ("grad_z", grad_z)):
        if g is not None:
            _dev(g, name, torch.float32, (S,))
    if topk_idx is not None:
        _dev(topk_idx, "topk_idx", torch.int32)
        if k is not None and k != topk_idx.shape[1]:
            raise ValueError(f"k is {k} but topk_idx has {topk_idx.shape[1]} columns")
        k = topk_idx.shape[1]
        _dev(topk_idx, "topk_idx", torch.int32, (T, k))
    elif k is None:
        raise ValueError("k is needed without topk_idx")
    if grad_topk_weights is not None:
        if topk_idx is None or topk_weights is None:
            raise ValueError("grad_topk_weights needs topk_idx and topk_weights")
        _dev(topk_weights, "topk_weights", torch.float32, (T, k))
        _dev(grad_topk_weights, "grad_topk_weights", torch.float32, (T, k))
    g = out if out is not None else _on(stream, torch.empty_like)(scores)
    _dev(g, "out", torch.float32, (T, E))
    rc = lib().moe_balance_loss_backward(
        _ptr(scores), T, E, k, _choice(score_func, _SCORE_FUNC, "score_func"), _ptr(seq_offsets),
        S, _ptr(token_mask), _ptr(counts), _ptr(tokens), _ptr(grad_balance), _ptr(grad_z),
        _ptr(topk_idx), _ptr(topk_weights), _ptr(grad_topk_weights), _ptr(g), _stream(stream))
    _check(rc, "moe_balance_loss_backward")
    return g


def combine_backward(grad_out: torch.Tensor, y: torch.Tensor, topk_weights: torch.Tensor,
                     pos: torch.Tensor, *, sorted_src=None, out=None, stream=None):
    """Gradients of combine: grad_y[pos[t, j]] = w[t, j] * grad_out[t] and
    grad_w[t, j] = <grad_out[t], y[pos[t, j]]>.

    grad_out [T, H] bfloat16 or float32, y [R, H] bfloat16, w [T, k] float32,
    pos [T, k] int32; sorted_src [R] int32 zero-fills grad_y's rows with a
    negative entry (without it, rows no pos names are not written).
    -> (grad_y [R, H] bfloat16, grad_w [T, k] float32)."""
    gd = _dt(grad_out, "grad_out")
    _dev(grad_out, "grad_out", grad_out.dtype)
    T, H = grad_out.shape
    R, k = y.shape[0], topk_weights.shape[1]
    _dev(y, "y", torch.bfloat16, (R, H))
    _dev(topk_weights, "topk_weights", torch.float32, (T, k))
    _dev(pos, "pos", torch.int32, (T, k))
    if sorted_src is not None:
        _dev(sorted_src, "sorted_src", torch.int32, (R,))
    if out is None:
        empty_like = _on(stream, torch.empty_like)
        gy, gw = empty_like(y), empty_like(topk_weights)
    else:
        gy, gw = out
        _dev(gy, "out[0]", torch.bfloat16, (R, H))
        _dev(gw, "out[1]", torch.float32, (T, k))
    rc = lib().moe_combine_backward(_ptr(grad_out), gd, _ptr(y), _ptr(topk_weights), _ptr(pos),
                                    _ptr(sorted_src), T, H, k, R, _ptr(gy), _ptr(gw),
                                    _stream(stream))
    _check(rc, "moe_combine_backward")
    return gy, gw


def expert_matvec_fp4(x: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, offsets=None, *,
                      sorted_src=None, k: int = 1, group: int = 32, swiglu: bool = False,
                      out_dtype=torch.bfloat16, out=None, stream=None):
    """Products of routed rows with their expert's 4-bit weights, for decode
    batches (few rows per expert).

    w [E, M, K/2] uint8 E2M1 codes (element 2i in the low nibble) and w_sf
    [E, M, K/group] float32 or uint8 (UE8M0), as expand_cast_fp4 writes them.
    Rows are in the route map's order: offsets [E+1] int32 (None: one expert,
    all rows).  x [num_x, K] bfloat16: row r of the output reads x[r], or with
    sorted_src [R] int32 x[sorted_src[r] // k] (a negative entry: a row of zeros).
    swiglu: M = 2N, the gate's outputs first; out = silu(gate) * up.
    -> out [R, N] bfloat16 or float32 (rows past offsets[E] not written)."""
    _dev(x, "x", torch.bfloat16)
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be [rows, K] and w [E, M, K/2]")
    K = x.shape[1]
    E, M = w.shape[0], w.shape[1]
    if group not in (16, 32, 64, 128):
        raise ValueError(f"group must be 16, 32, 64 or 128, got {group}")
    _dev(w, "w", torch.uint8, (E, M, K // 2))
    if w_sf.dtype not in (torch.float32, torch.uint8):
        raise TypeError(f"w_sf must be float32 or uint8, got {w_sf.dtype}")
    _dev(w_sf, "w_sf", w_sf.dtype, (E, M, K // group))
    if swiglu and M % 2:
        raise ValueError("swiglu needs an even number of weight rows")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    if offsets is not None:
        _dev(offsets, "offsets", torch.int32, (E + 1,))
    if sorted_src is not None:
        _dev(sorted_src, "sorted_src", torch.int32)
        R = sorted_src.shape[0]
    else:
        R = x.shape[0]
    N = M // 2 if swiglu else M
    if out is None:
        o = _empty((R, N), out_dtype, x, stream)
    else:
        o = _dev(out, "out", out_dtype, (R, N))
    rc = lib().moe_expert_matvec_fp4(_ptr(x), x.shape[0], _ptr(w), _ptr(w_sf),
                                     WSF_UE8M0 if w_sf.dtype == torch.uint8 else WSF_F32, group,
                                     _ptr(offsets), _ptr(sorted_src), E, k, R, K, N, int(swiglu),
                                     _ptr(o), MOE_OUT_F32 if out_dtype == torch.float32 else
                                     MOE_OUT_BF16, _stream(stream))
    _check(rc, "moe_expert_matvec_fp4")
    return o


def peak_copy(src: torch.Tensor, dst: torch.Tensor, *, stream=None):
    """Device copy of src's bytes into dst (the HBM roofline probe)."""
    if src.device.type != "cuda" or dst.device.type != "cuda":
        raise ValueError("peak_copy needs CUDA tensors")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < n:
        raise ValueError("dst too small")
    _check(lib().moe_peak_copy(_ptr(src), _ptr(dst), n, _stream(stream)), "moe_peak_copy")


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error bits."""
    bits = ctypes.c_uint32(0)
    rc = lib().moe_get_device_status(_stream(stream), ctypes.byref(bits))
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        _check(rc, "moe_get_device_status")
    return int(bits.value)


def launch_count() -> int:
    return int(lib().moe_kernel_launch_count())


__all__ = ["lib", "MoeError", "topk_gate", "route_map", "route_map_workspace_bytes",
           "route_map_aligned", "expand_cast_fp8_padded", "expand_cast_fp8_ex",
           "expand_cast_fp8_ex_workspace_bytes", "swiglu_cast_fp8_ex", "sf_empty",
           "route_expand_cast_fp8", "route_expand_cast_workspace", "debug_set", "debug_cvt", "expand_cast_fp4", "swiglu_cast_fp4",
           "expand_cast_fp8", "swiglu_cast_fp8", "combine", "peak_copy", "device_status",
           "launch_count", "SIGNATURES", "block_norm", "block_norm_backward",
           "block_norm_backward_workspace_bytes", "balance_loss", "balance_loss_backward",
           "balance_loss_workspace_bytes", "combine_backward", "expert_matvec_fp4"]
