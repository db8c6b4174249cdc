"""GB300 (sm_103a) Mamba2 decode-step selective state update.

Python binding of ``libssu.so`` (C ABI declared in ``include/ssu.h``).  The functions carry
the C names and only marshal arguments: tensor pointers, sizes and element strides go into
the ABI structs, and every step of the update runs in the library's CUDA kernels.  There is
no CPU or PyTorch fallback: if the library is missing, every entry point raises.

Operand layout (sglang PR #41223, Details / Kernel measurement): ``state_pool`` fp32 or bf16
``[pool, H, P, N]`` (N = 64, 128 or 256); ``state_batch_indices`` int32/int64 ``[bs]``; ``x`` and ``out`` bf16
``[bs, H, P]``; ``B`` and ``C`` bf16 ``[bs, G, N]``; ``dt`` bf16 ``[bs, H]`` (or the
head-expanded ``[bs, H, P]`` view with stride 0 over P); ``dt_bias`` and ``D`` fp32 ``[H]``
(or ``[H, P]`` with stride 0); ``A`` fp32 ``[H]`` (or ``[H, P, N]`` with strides 0).
Strided views are accepted as they are; nothing is copied.
"""

from __future__ import annotations

import ctypes
import struct
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libssu.so"

SSU_OK = 0
SSU_ERR_INVALID_ARG = 1
SSU_ERR_UNSUPPORTED = 2
SSU_ERR_MISALIGNED = 3
SSU_ERR_CUDA = 4
SSU_ERR_INDEX_OOB = 5

SSU_INDEX_I32 = 0
SSU_INDEX_I64 = 1

SSU_STATE_F32 = 0
SSU_STATE_BF16 = 1

SSU_MODE_AUTO = 0
SSU_MODE_VEC = 1

_i64 = ctypes.c_int64


class ssu_shape_t(ctypes.Structure):
    _fields_ = [("batch", _i64), ("nheads", _i64), ("headdim", _i64), ("dstate", _i64),
                ("ngroups", _i64), ("pool_size", _i64), ("index_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32)]


class ssu_strides_t(ctypes.Structure):
    _fields_ = [("state", _i64 * 4), ("x", _i64 * 3), ("out", _i64 * 3), ("dt", _i64 * 3),
                ("B", _i64 * 3), ("C", _i64 * 3), ("dt_bias", _i64 * 2), ("D", _i64 * 2),
                ("A", _i64 * 3), ("idx", _i64)]


class ssu_launch_t(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("rows_per_warp", ctypes.c_int32),
                ("warps_per_cta", ctypes.c_int32), ("stages", ctypes.c_int32)]


class ssu_token_strides_t(ctypes.Structure):
    _fields_ = [("x", _i64), ("out", _i64), ("dt", _i64), ("B", _i64), ("C", _i64),
                ("intermediate", _i64 * 5)]


SSU_MAX_TOKENS = 64


class ssu_block_tensor_t(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("block_bytes", _i64),
                ("block_stride_bytes", _i64), ("num_blocks", _i64)]


class ssu_copy_launch_t(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("chunk_kib", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("threads", ctypes.c_int32)]


SSU_COPY_AUTO = 0
SSU_COPY_VEC = 1
SSU_COPY_MAX_TENSORS = 64


class ssu_rotate_shape_t(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("q_heads", _i64), ("kv_heads", _i64), ("headdim", _i64),
                ("rotary", _i64), ("num_positions", _i64), ("num_pages", _i64),
                ("page_size", _i64), ("index_dtype", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class ssu_rotate_strides_t(ctypes.Structure):
    _fields_ = [("q", _i64 * 2), ("k", _i64 * 2), ("v", _i64 * 2), ("q_out", _i64 * 2),
                ("k_pages", _i64 * 3), ("v_pages", _i64 * 3), ("table", _i64),
                ("positions", _i64), ("slots", _i64)]


class ssu_attend_shape_t(ctypes.Structure):
    _fields_ = [("requests", _i64), ("q_heads", _i64), ("kv_heads", _i64), ("headdim", _i64),
                ("num_pages", _i64), ("page_size", _i64), ("max_pages", _i64),
                ("index_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ssu_attend_strides_t(ctypes.Structure):
    _fields_ = [("q", _i64 * 2), ("out", _i64 * 2), ("k_pages", _i64 * 3),
                ("v_pages", _i64 * 3), ("page_table", _i64 * 2), ("lengths", _i64)]


class SsuError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {message}")


_lib = None
_vp = ctypes.c_void_p
_EXPORTS = {
    "ssu_abi_version": (ctypes.c_int32, []),
    "ssu_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ssu_last_error": (ctypes.c_char_p, []),
    "ssu_create": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.c_int32]),
    "ssu_destroy": (ctypes.c_int, [_vp]),
    "ssu_validate": (ctypes.c_int, [_vp] * 10 + [ctypes.POINTER(ssu_shape_t),
                                                 ctypes.POINTER(ssu_strides_t)]),
    "ssu_update": (ctypes.c_int, [_vp] * 11 + [ctypes.POINTER(ssu_shape_t),
                                               ctypes.POINTER(ssu_strides_t), _vp]),
    "ssu_get_error": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_uint32),
                                     ctypes.POINTER(ctypes.c_int64)]),
    "ssu_set_launch": (ctypes.c_int, [_vp, ctypes.POINTER(ssu_launch_t)]),
    "ssu_set_launch_override": (ctypes.c_int, [_vp, ctypes.c_char_p]),
    "ssu_get_launch": (ctypes.c_int, [_vp, ctypes.POINTER(ssu_shape_t),
                                      ctypes.POINTER(ssu_launch_t)]),
    "ssu_set_pdl": (ctypes.c_int, [_vp, ctypes.c_int32]),
    "ssu_check_indices": (ctypes.c_int, [_vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64,
                                         ctypes.POINTER(ctypes.c_int64)]),
    "ssu_update_tokens": (ctypes.c_int, [_vp] * 12 + [ctypes.POINTER(ssu_shape_t),
                                                      ctypes.POINTER(ssu_strides_t),
                                                      ctypes.c_int64,
                                                      ctypes.POINTER(ssu_token_strides_t), _vp]),
    "ssu_prompts_workspace_bytes": (ctypes.c_int, [_vp, _vp, _i64, ctypes.POINTER(_i64)]),
    "ssu_update_prompts": (ctypes.c_int, [_vp] * 15 + [_i64, _vp, _i64, _vp]),
    "ssu_rotate_qk": (ctypes.c_int, [_vp] * 14 + [ctypes.c_float, _vp]),
    "ssu_attend_workspace_bytes": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(_i64)]),
    "ssu_attend": (ctypes.c_int, [_vp] * 9 + [ctypes.c_float, _i64, _i64, _vp, _i64, _vp]),
    "ssu_copy_blocks": (ctypes.c_int, [_vp, ctypes.POINTER(ssu_block_tensor_t), ctypes.c_int32,
                                       _vp, _vp, ctypes.c_int64, ctypes.c_int32, _vp]),
    "ssu_copy_set_launch": (ctypes.c_int, [_vp, ctypes.POINTER(ssu_copy_launch_t)]),
    "ssu_update_static": (ctypes.c_int, [_vp] * 10 + [ctypes.POINTER(ssu_shape_t),
                                                      ctypes.POINTER(ssu_strides_t), _vp, _vp]),
    "ssu_host_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(ssu_shape_t),
                                                ctypes.POINTER(ctypes.c_int64)]),
    "ssu_update_from_host": (ctypes.c_int, [_vp] * 11 + [ctypes.POINTER(ssu_shape_t),
                                                         ctypes.POINTER(ssu_strides_t), _vp,
                                                         ctypes.c_int64, _vp]),
}

SSU_STATIC_SCRATCH_BYTES = 256
SSU_ABI_VERSION = 2
SSU_STATIC_MAX_BATCH = 2147483647


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in _EXPORTS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if handle.ssu_abi_version() != SSU_ABI_VERSION:
            raise RuntimeError("libssu.so ABI version mismatch")
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().ssu_status_string(status).decode()


def last_error() -> str:
    return lib().ssu_last_error().decode()


def _check(status: int, where: str) -> None:
    if status != SSU_OK:
        raise SsuError(status, where, last_error())


# ---- marshalling -------------------------------------------------------------------------

def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _expect(t: torch.Tensor, name: str, dtype: torch.dtype, ndims: tuple[int, ...]):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() not in ndims:
        raise ValueError(f"{name} must have {' or '.join(map(str, ndims))} dims, got {t.dim()}")


def _broadcast_strides(t: torch.Tensor, name: str, dims: tuple[int, ...], full: int):
    """Strides of a per-head operand in its expanded form of `full` dims (missing dims: 0)."""
    if t.shape[:1] != dims[:1]:
        raise ValueError(f"{name} must start with dimension {dims[0]}, got {tuple(t.shape)}")
    st = list(t.stride()) + [0] * (full - t.dim())
    for i in range(1, t.dim()):
        if t.shape[i] != dims[i]:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected prefix of {dims}")
    return st


def describe(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out):
    """Build ``(ssu_shape_t, ssu_strides_t)`` for a set of tensors (no data is touched)."""
    if not isinstance(state_pool, torch.Tensor) or state_pool.dim() != 4 or \
            state_pool.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("state_pool must be a 4-D float32 or bfloat16 tensor")
    if state_batch_indices.dtype not in (torch.int32, torch.int64) or \
            state_batch_indices.dim() != 1:
        raise TypeError("state_batch_indices must be a 1-D int32 or int64 tensor")
    _expect(x, "x", torch.bfloat16, (3,))
    _expect(out, "out", torch.bfloat16, (3,))
    _expect(dt, "dt", torch.bfloat16, (2, 3))
    _expect(dt_bias, "dt_bias", torch.float32, (1, 2))
    _expect(D, "D", torch.float32, (1, 2))
    _expect(A, "A", torch.float32, (1, 3))
    _expect(B, "B", torch.bfloat16, (3,))
    _expect(C, "C", torch.bfloat16, (3,))
    pool, H, P, N = state_pool.shape
    bs = x.shape[0]
    G = B.shape[1]
    if tuple(x.shape) != (bs, H, P) or tuple(out.shape) != (bs, H, P):
        raise ValueError(f"x and out must be [bs, H, P] = {(bs, H, P)}")
    if tuple(B.shape) != (bs, G, N) or tuple(C.shape) != (bs, G, N):
        raise ValueError(f"B and C must be [bs, G, N] = {(bs, G, N)}")
    if state_batch_indices.shape[0] != bs:
        raise ValueError("state_batch_indices must have one entry per request")
    if tuple(dt.shape[:2]) != (bs, H) or (dt.dim() == 3 and dt.shape[2] != P):
        raise ValueError("dt must be [bs, H] or [bs, H, P]")
    shape = ssu_shape_t(bs, H, P, N, G, pool,
                        SSU_INDEX_I64 if state_batch_indices.dtype == torch.int64
                        else SSU_INDEX_I32,
                        SSU_STATE_BF16 if state_pool.dtype == torch.bfloat16 else SSU_STATE_F32)
    st = ssu_strides_t()
    st.state[:] = list(state_pool.stride())
    st.x[:] = list(x.stride())
    st.out[:] = list(out.stride())
    st.dt[:] = list(dt.stride()) + [0] * (3 - dt.dim())
    st.B[:] = list(B.stride())
    st.C[:] = list(C.stride())
    st.dt_bias[:] = _broadcast_strides(dt_bias, "dt_bias", (H, P), 2)
    st.D[:] = _broadcast_strides(D, "D", (H, P), 2)
    st.A[:] = _broadcast_strides(A, "A", (H, P, N), 3)
    st.idx = state_batch_indices.stride(0)
    return shape, st


def _stream_ptr(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- the C entry points --------------------------------------------------------------------

def ssu_abi_version() -> int:
    return int(lib().ssu_abi_version())


def ssu_create(device: int = 0) -> int:
    """Create a handle on ``device``; returns it as an integer."""
    h = _vp()
    _check(lib().ssu_create(ctypes.byref(h), int(device)), "ssu_create")
    return h.value


def ssu_destroy(handle: int) -> None:
    _check(lib().ssu_destroy(handle), "ssu_destroy")


def ssu_validate(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
                 shape: ssu_shape_t | None = None, strides: ssu_strides_t | None = None) -> int:
    """Host-side validation only; returns the status code (0 = valid).

    With tensors, the shape and strides are derived from them.  With integer pointers (no
    memory is touched), ``shape`` and ``strides`` must be given.
    """
    if shape is None or strides is None:
        shape, strides = describe(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D,
                                  out)
    ptrs = [_ptr(t) for t in (state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)]
    return int(lib().ssu_validate(*ptrs, ctypes.byref(shape), ctypes.byref(strides)))


def ssu_update(handle: int, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
               stream=None) -> None:
    """Enqueue one decode step on ``stream`` (default: torch's current stream)."""
    shape, strides = describe(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)
    ptrs = [_ptr(t) for t in (state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)]
    _check(lib().ssu_update(handle, *ptrs, ctypes.byref(shape), ctypes.byref(strides),
                            _stream_ptr(stream)), "ssu_update")


def ssu_update_static(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
                      counters_out=None, stream=None) -> None:
    """Allocation-free ssu_update on the current device (no handle).

    For callers that cannot allocate device memory: the kernel's counters live in a fixed
    256-byte array inside the library.  ``counters_out`` is an optional caller-owned int32/uint32
    device tensor of >= 3 elements that receives [skipped, smallest skipped index or
    0xFFFFFFFF, 0].  Calls that overlap on the GPU race on the shared counters.
    """
    shape, strides = describe(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)
    if counters_out is not None:
        _check_counters(counters_out, state_pool)
    ptrs = [_ptr(t) for t in (state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)]
    _check(lib().ssu_update_static(*ptrs, ctypes.byref(shape), ctypes.byref(strides),
                                   _ptr(counters_out), _stream_ptr(stream)),
           "ssu_update_static")


def _check_counters(counters_out, state_pool) -> None:
    """``counters_out`` receives a 12-byte device-to-device copy: it must be a contiguous CUDA
    tensor of 4-byte elements with at least 3 of them, on the state pool's device."""
    t = counters_out
    if not isinstance(t, torch.Tensor):
        raise ValueError("counters_out must be a torch.Tensor (or None)")
    if t.device.type != "cuda" or t.device != state_pool.device:
        raise ValueError(f"counters_out must be on {state_pool.device}, got {t.device}")
    if t.element_size() != 4 or t.dtype.is_floating_point:
        raise ValueError(f"counters_out must hold 4-byte integers, got {t.dtype}")
    if t.numel() < 3 or not t.is_contiguous():
        raise ValueError("counters_out must be contiguous with at least 3 elements")


def ssu_host_workspace_bytes(shape: ssu_shape_t) -> int:
    """Device workspace bytes ``ssu_update_from_host`` needs for ``shape``."""
    n = ctypes.c_int64()
    _check(lib().ssu_host_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssu_host_workspace_bytes")
    return int(n.value)


def ssu_update_from_host(handle: int, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C,
                         D, out, workspace, stream=None) -> None:
    """One decode step with the per-step operands (``state_batch_indices``, ``x``, ``dt``,
    ``B``, ``C``) and ``out`` in page-locked host memory (``pin_memory()`` tensors); the state
    pool, ``dt_bias``, ``A`` and ``D`` on the device.  ``workspace`` is a device uint8 tensor of
    at least ``ssu_host_workspace_bytes(shape)`` bytes.  ``out`` is complete once ``stream``
    has passed the call."""
    shape, strides = describe(state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)
    ptrs = [_ptr(t) for t in (state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out)]
    nbytes = workspace.numel() * workspace.element_size() if isinstance(workspace, torch.Tensor) \
        else 0
    _check(lib().ssu_update_from_host(handle, *ptrs, ctypes.byref(shape), ctypes.byref(strides),
                                      _ptr(workspace), nbytes, _stream_ptr(stream)),
           "ssu_update_from_host")


def ssu_update_from_host_raw(handle: int, ptrs, shape: ssu_shape_t, strides: ssu_strides_t,
                             workspace: int, workspace_bytes: int, stream: int | None) -> int:
    """ssu_update_from_host with precomputed pointers/structs; returns the status."""
    return int(lib().ssu_update_from_host(handle, *ptrs, ctypes.byref(shape),
                                          ctypes.byref(strides), workspace, workspace_bytes,
                                          stream))


def ssu_update_raw(handle: int, ptrs, shape: ssu_shape_t, strides: ssu_strides_t,
                   stream: int | None) -> int:
    """ssu_update with precomputed pointers/structs (for tight timing loops); returns status."""
    return int(lib().ssu_update(handle, *ptrs, ctypes.byref(shape), ctypes.byref(strides),
                                stream))


def ssu_get_error(handle: int, stream=None) -> tuple[int, int]:
    """Synchronise, then read and clear the skipped-request counters: (skipped, first_bad)."""
    skipped = ctypes.c_uint32()
    first = ctypes.c_int64()
    st = lib().ssu_get_error(handle, _stream_ptr(stream), ctypes.byref(skipped),
                             ctypes.byref(first))
    if st not in (SSU_OK, SSU_ERR_INDEX_OOB):
        _check(st, "ssu_get_error")
    return int(skipped.value), int(first.value)


def ssu_set_launch(handle: int, mode: int = SSU_MODE_AUTO, rows_per_warp: int = 0,
                   warps_per_cta: int = 0, stages: int = 0) -> None:
    """Force a launch shape (mode AUTO restores the built-in table)."""
    cfg = ssu_launch_t(mode, rows_per_warp, warps_per_cta, stages)
    _check(lib().ssu_set_launch(handle, ctypes.byref(cfg)), "ssu_set_launch")


def ssu_set_launch_override(handle: int, spec: str | None) -> None:
    """Force a launch shape from text: "rows_per_warp,warps_per_cta" (optionally "vec,..."),
    or None / "" / "auto" for the built-in table."""
    _check(lib().ssu_set_launch_override(handle, None if spec is None else spec.encode()),
           "ssu_set_launch_override")


def ssu_check_indices(state_batch_indices, pool_size: int) -> int:
    """Debug check of a host (CPU) index tensor: in range and no repeated slot.  Returns -1
    when the indices are valid, else the position of the first bad entry."""
    t = state_batch_indices
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu" or t.dim() != 1:
        raise TypeError("state_batch_indices must be a 1-D CPU tensor")
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError("state_batch_indices must be int32 or int64")
    t = t.contiguous()
    first = ctypes.c_int64(-1)
    st = lib().ssu_check_indices(t.data_ptr(), t.shape[0],
                                 SSU_INDEX_I64 if t.dtype == torch.int64 else SSU_INDEX_I32,
                                 int(pool_size), ctypes.byref(first))
    if st not in (SSU_OK, SSU_ERR_INVALID_ARG):
        _check(st, "ssu_check_indices")
    return int(first.value) if st != SSU_OK else -1


def ssu_set_pdl(handle: int, enable: bool = True) -> None:
    """Turn programmatic dependent launch on or off for this handle (on by default)."""
    _check(lib().ssu_set_pdl(handle, 1 if enable else 0), "ssu_set_pdl")


def ssu_get_launch(handle: int, shape: ssu_shape_t) -> tuple[int, int, int, int]:
    cfg = ssu_launch_t()
    _check(lib().ssu_get_launch(handle, ctypes.byref(shape), ctypes.byref(cfg)),
           "ssu_get_launch")
    return cfg.mode, cfg.rows_per_warp, cfg.warps_per_cta, cfg.stages


def ssu_update_tokens(handle: int, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D,
                      out, intermediate=None, stream=None) -> None:
    """T consecutive decode steps per request.  ``x`` and ``out`` are ``[bs, T, H, P]``;
    ``dt`` is ``[bs, T, H]`` (or ``[bs, T, H, P]`` with stride 0 over P); ``B`` and ``C`` are
    ``[bs, T, G, N]``; ``intermediate`` (optional, ``[bs, T, H, P, N]`` of the state's dtype)
    receives the state after every token.  Per-head operands as for ``ssu_update``."""
    for name, t, nd in (("x", x, 4), ("out", out, 4), ("B", B, 4), ("C", C, 4)):
        if not isinstance(t, torch.Tensor) or t.dim() != nd:
            raise ValueError(f"{name} must be a {nd}-D tensor with a token dimension")
    if dt.dim() not in (3, 4):
        raise ValueError("dt must be [bs, T, H] or [bs, T, H, P]")
    T = x.shape[1]
    for name, t in (("out", out), ("dt", dt), ("B", B), ("C", C)):
        if t.shape[1] != T:
            raise ValueError(f"{name} must have {T} tokens")
    shape, strides = describe(state_pool, state_batch_indices, x[:, 0], dt[:, 0], dt_bias, A,
                              B[:, 0], C[:, 0], D, out[:, 0])
    ts = ssu_token_strides_t()
    ts.x, ts.out, ts.dt, ts.B, ts.C = (x.stride(1), out.stride(1), dt.stride(1), B.stride(1),
                                       C.stride(1))
    if intermediate is not None:
        _expect(intermediate, "intermediate", state_pool.dtype, (5,))
        if tuple(intermediate.shape) != (x.shape[0], T, x.shape[2], x.shape[3],
                                         state_pool.shape[3]):
            raise ValueError("intermediate must be [bs, T, H, P, N]")
        ts.intermediate[:] = list(intermediate.stride())
    ptrs = [_ptr(t) for t in (state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
                               intermediate)]
    _check(lib().ssu_update_tokens(handle, *ptrs, ctypes.byref(shape), ctypes.byref(strides), T,
                                   ctypes.byref(ts), _stream_ptr(stream)), "ssu_update_tokens")


# ---- prompts and attention ---------------------------------------------------------------
#
# These calls sit in a serving loop beside the decode step and are often shorter on the device
# than their marshalling, so it is written out: one look at every tensor, the ABI's structs packed
# as bytes (a struct of N words costs 0.3 us this way, 1.6 us as a ctypes array), and messages only
# where a check has failed.

_BF16, _F32 = torch.bfloat16, torch.float32
_INDEX_TYPE = {torch.int32: SSU_INDEX_I32, torch.int64: SSU_INDEX_I64}
_STATE_TYPE = {_F32: SSU_STATE_F32, _BF16: SSU_STATE_BF16}
_SHAPE = struct.Struct("6q2i")            # ssu_shape_t
_STRIDES = struct.Struct("27q")           # ssu_strides_t
_ROTATE_SHAPE = struct.Struct("8q2i")     # ssu_rotate_shape_t
_ROTATE_STRIDES = struct.Struct("17q")    # ssu_rotate_strides_t
_ATTEND_SHAPE = struct.Struct("7q2i")     # ssu_attend_shape_t
_ATTEND_STRIDES = struct.Struct("13q")    # ssu_attend_strides_t
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else \
    lambda device: torch.cuda.current_stream(device).cuda_stream


def _refuse_types(**wanted) -> None:
    """Raises for the first tensor that is not of its wanted (dtype, dims)."""
    for name, (t, dtypes, dims) in wanted.items():
        if t.dtype not in dtypes or t.dim() not in dims:
            raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))} with "
                            f"{' or '.join(map(str, dims))} dims, got {t.dtype} with {t.dim()}")
    raise TypeError("operand types do not fit together")


def _device_of(tensors) -> int:
    """The CUDA device on which every tensor lies."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or dev < 0:
            raise ValueError("every operand must be a CUDA tensor of one device, got "
                             + ", ".join(sorted({str(u.device) for u in tensors})))
    return dev


def _workspace(workspace, dev: int) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor of the operands' device")
    return workspace.data_ptr(), workspace.nbytes


def _stream_on(dev: int, stream) -> int:
    if stream is None:
        return _raw_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _head_strides(t, name: str, dims: tuple[int, ...]) -> tuple[int, ...]:
    """Strides of a per-head operand in its expanded form (missing dimensions: 0)."""
    if t.shape != dims[:t.dim()]:
        raise ValueError(f"{name} must have the shape {dims} or {dims[:1]}, got {tuple(t.shape)}")
    st = t.stride()
    return st if len(st) == len(dims) else (*st, *(0,) * (len(dims) - len(st)))


def describe_prompts(state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias, A, B, C, D,
                     out) -> tuple[bytes, bytes]:
    """The ``ssu_shape_t`` and ``ssu_strides_t`` of a prompt call, as bytes (no data is touched)."""
    kind, state = _INDEX_TYPE.get(cu_tokens.dtype), _STATE_TYPE.get(state_pool.dtype)
    sp, sx, so, sd = state_pool.stride(), x.stride(), out.stride(), dt.stride()
    sb, sc, si = B.stride(), C.stride(), state_batch_indices.stride()
    if not (x.dtype is dt.dtype is B.dtype is C.dtype is out.dtype is _BF16
            and dt_bias.dtype is A.dtype is D.dtype is _F32 and kind is not None
            and state_batch_indices.dtype is cu_tokens.dtype and state is not None
            and len(sp) == 4 and len(sx) == len(so) == len(sb) == len(sc) == 3
            and len(sd) in (2, 3) and len(si) == cu_tokens.dim() == 1
            and dt_bias.dim() in (1, 2) and D.dim() in (1, 2) and A.dim() in (1, 3)):
        ints = (torch.int32, torch.int64)
        _refuse_types(state_pool=(state_pool, (_F32, _BF16), (4,)), x=(x, (_BF16,), (3,)),
                      dt=(dt, (_BF16,), (2, 3)), B=(B, (_BF16,), (3,)), C=(C, (_BF16,), (3,)),
                      out=(out, (_BF16,), (3,)), dt_bias=(dt_bias, (_F32,), (1, 2)),
                      A=(A, (_F32,), (1, 3)), D=(D, (_F32,), (1, 2)),
                      cu_tokens=(cu_tokens, ints, (1,)),
                      state_batch_indices=(state_batch_indices, (cu_tokens.dtype,), (1,)))
    pool, H, P, N = state_pool.shape
    T, G, _ = B.shape
    bs, = state_batch_indices.shape
    if x.shape != (T, H, P) or out.shape != x.shape:
        raise ValueError(f"x and out must be [tokens, H, P] = {(T, H, P)}")
    if B.shape != (T, G, N) or C.shape != B.shape:
        raise ValueError(f"B and C must be [tokens, G, N] = {(T, G, N)}")
    if dt.shape != (T, H, P)[:len(sd)]:
        raise ValueError(f"dt must be {(T, H)} or {(T, H, P)}")
    if cu_tokens.shape[0] != bs + 1 or cu_tokens.stride(0) != 1:
        raise ValueError(f"cu_tokens must be contiguous with {bs + 1} entries")
    return (_SHAPE.pack(bs, H, P, N, G, pool, kind, state),
            _STRIDES.pack(*sp, *sx, *so, *(sd if len(sd) == 3 else (*sd, 0)), *sb, *sc,
                          *_head_strides(dt_bias, "dt_bias", (H, P)),
                          *_head_strides(D, "D", (H, P)), *_head_strides(A, "A", (H, P, N)), *si))


def ssu_prompts_workspace_bytes(handle: int, state_pool, x, B, state_batch_indices) -> int:
    """Device workspace bytes ``ssu_update_prompts`` needs for these operands' sizes."""
    pool, H, P, N = state_pool.shape
    shape = _SHAPE.pack(state_batch_indices.shape[0], H, P, N, B.shape[1], pool, SSU_INDEX_I32,
                        _STATE_TYPE.get(state_pool.dtype, SSU_STATE_F32))
    n = _i64()
    _check(lib().ssu_prompts_workspace_bytes(handle, shape, x.shape[0], ctypes.byref(n)),
           "ssu_prompts_workspace_bytes")
    return int(n.value)


def ssu_update_prompts(handle: int, state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias,
                       A, B, C, D, out, workspace=None, fresh=None, stream=None) -> None:
    """Whole prompts, packed: prompt ``b`` is rows ``cu_tokens[b]:cu_tokens[b + 1]`` of ``x``,
    ``out`` ``[tokens, H, P]``, ``dt`` ``[tokens, H]``, ``B`` and ``C`` ``[tokens, G, N]``.  It
    continues slot ``state_batch_indices[b]``, or starts from zero where ``fresh[b]`` (uint8 or
    bool) is set, and leaves its last state there.  ``cu_tokens`` and ``state_batch_indices``
    have one type; ``workspace`` is a device uint8 tensor of ``ssu_prompts_workspace_bytes``."""
    shape, strides = describe_prompts(state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias,
                                      A, B, C, D, out)
    tensors = (state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias, A, B, C, D, out)
    dev = _device_of(tensors)
    if fresh is not None:
        if fresh.dtype not in (torch.uint8, torch.bool) or \
                fresh.shape != state_batch_indices.shape or not fresh.is_contiguous() or \
                fresh.get_device() != dev:
            raise ValueError("fresh must be a contiguous uint8 or bool CUDA tensor with one entry "
                             "per prompt")
        fresh = fresh.data_ptr()
    ws, nbytes = _workspace(workspace, dev)
    p = [t.data_ptr() for t in tensors]
    st = lib().ssu_update_prompts(handle, p[0], p[1], p[2], fresh, *p[3:], shape, strides,
                                  x.shape[0], ws, nbytes, _stream_on(dev, stream))
    if st:
        _check(st, "ssu_update_prompts")


def ssu_rotate_qk(handle: int, q, k, v, q_weight, k_weight, table, positions, q_out, k_pages,
                  v_pages, slots, eps: float = 1e-6, interleaved: bool = False,
                  stream=None) -> None:
    """RMS norm of every head of ``q`` ``[tokens, Hq, D]`` and ``k`` ``[tokens, Hk, D]``
    (weights fp32 ``[D]``), rotation by ``table[positions[t]]`` (fp32 ``[places, rotary]``:
    cosines, then sines), queries to ``q_out``, keys and ``v`` to row ``slots[t]`` of the pages
    ``[pages, page_size, Hk, D]`` (-1: not stored)."""
    sq, sk, sv, so = q.stride(), k.stride(), v.stride(), q_out.stride()
    kp, vp, st = k_pages.stride(), v_pages.stride(), table.stride()
    kind = _INDEX_TYPE.get(slots.dtype)
    if not (q.dtype is k.dtype is v.dtype is q_out.dtype is k_pages.dtype is v_pages.dtype is _BF16
            and q_weight.dtype is k_weight.dtype is table.dtype is _F32 and kind is not None
            and positions.dtype is slots.dtype and len(sq) == len(sk) == len(sv) == len(so) == 3
            and len(kp) == len(vp) == 4 and len(st) == 2):
        ints = (torch.int32, torch.int64)
        _refuse_types(q=(q, (_BF16,), (3,)), k=(k, (_BF16,), (3,)), v=(v, (_BF16,), (3,)),
                      q_out=(q_out, (_BF16,), (3,)), k_pages=(k_pages, (_BF16,), (4,)),
                      v_pages=(v_pages, (_BF16,), (4,)), q_weight=(q_weight, (_F32,), (1,)),
                      k_weight=(k_weight, (_F32,), (1,)), table=(table, (_F32,), (2,)),
                      slots=(slots, ints, (1,)), positions=(positions, (slots.dtype,), (1,)))
    T, Hq, D = q.shape
    Hk = k.shape[1]
    if q_out.shape != q.shape or k.shape != (T, Hk, D) or v.shape != k.shape:
        raise ValueError(f"q and q_out must be {(T, Hq, D)}, k and v {(T, Hk, D)}")
    pages, page = k_pages.shape[:2]
    if k_pages.shape != (pages, page, Hk, D) or v_pages.shape != k_pages.shape:
        raise ValueError(f"k_pages and v_pages must be [pages, page_size, {Hk}, {D}]")
    if q_weight.shape != (D,) or k_weight.shape != (D,) or q_weight.stride() != (1,) or \
            k_weight.stride() != (1,):
        raise ValueError(f"q_weight and k_weight must be contiguous with {D} elements")
    if positions.shape != (T,) or slots.shape != (T,):
        raise ValueError("positions and slots must have one entry per token")
    if not (sq[2] == sk[2] == sv[2] == so[2] == kp[3] == vp[3] == st[1] == 1):
        raise ValueError("the last dimension of every operand must have stride 1")
    tensors = (q, k, v, q_weight, k_weight, table, positions, q_out, k_pages, v_pages, slots)
    dev = _device_of(tensors)
    places, rotary = table.shape
    status = lib().ssu_rotate_qk(
        handle, *[t.data_ptr() for t in tensors],
        _ROTATE_SHAPE.pack(T, Hq, Hk, D, rotary, places, pages, page, kind, bool(interleaved)),
        _ROTATE_STRIDES.pack(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1], kp[0], kp[1],
                             kp[2], vp[0], vp[1], vp[2], st[0], *positions.stride(),
                             *slots.stride()), eps, _stream_on(dev, stream))
    if status:
        _check(status, "ssu_rotate_qk")


def ssu_attend_workspace_bytes(handle: int, q, k_pages) -> int:
    """Device workspace bytes ``ssu_attend`` needs for these operands' sizes (fill it with zeros
    once)."""
    n = _i64()
    shape = _ATTEND_SHAPE.pack(*q.shape[:2], k_pages.shape[2], q.shape[2], *k_pages.shape[:2], 0,
                               SSU_INDEX_I32, 0)
    _check(lib().ssu_attend_workspace_bytes(handle, shape, ctypes.byref(n)),
           "ssu_attend_workspace_bytes")
    return int(n.value)


def ssu_attend(handle: int, q, k_pages, v_pages, page_table, lengths, out, workspace=None,
               scale: float | None = None, window: int = 0, sinks: int = 0, stream=None) -> None:
    """One new token per request: ``q`` and ``out`` ``[requests, Hq, D]``, the cache in pages
    ``[pages, page_size, Hk, D]`` named by ``page_table`` ``[requests, max_pages]``, of which
    the first ``lengths[b]`` positions are visible (with ``window``: its last ``window`` and the
    first ``sinks``).  ``scale`` defaults to ``D ** -0.5``.  ``workspace`` is a device tensor of
    ``ssu_attend_workspace_bytes``, zero before its first use, not shared by overlapping calls."""
    sq, so, kp, vp = q.stride(), out.stride(), k_pages.stride(), v_pages.stride()
    st, sl = page_table.stride(), lengths.stride()
    kind = _INDEX_TYPE.get(lengths.dtype)
    if not (q.dtype is k_pages.dtype is v_pages.dtype is out.dtype is _BF16 and kind is not None
            and page_table.dtype is lengths.dtype and len(sq) == len(so) == 3
            and len(kp) == len(vp) == 4 and len(st) == 2 and len(sl) == 1):
        _refuse_types(q=(q, (_BF16,), (3,)), out=(out, (_BF16,), (3,)),
                      k_pages=(k_pages, (_BF16,), (4,)), v_pages=(v_pages, (_BF16,), (4,)),
                      lengths=(lengths, (torch.int32, torch.int64), (1,)),
                      page_table=(page_table, (lengths.dtype,), (2,)))
    bs, Hq, D = q.shape
    pages, page, Hk, _ = k_pages.shape
    most = page_table.shape[1]
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if k_pages.shape[3] != D or v_pages.shape != k_pages.shape:
        raise ValueError(f"k_pages and v_pages must be [pages, page_size, Hk, {D}]")
    if page_table.shape[0] != bs or lengths.shape[0] != bs:
        raise ValueError("page_table and lengths must have one row per request")
    if not (sq[2] == so[2] == kp[3] == vp[3] == 1):
        raise ValueError("the last dimension of q, out and the pages must have stride 1")
    tensors = (q, k_pages, v_pages, page_table, lengths, out)
    dev = _device_of(tensors)
    ws, nbytes = _workspace(workspace, dev)
    status = lib().ssu_attend(
        handle, *[t.data_ptr() for t in tensors],
        _ATTEND_SHAPE.pack(bs, Hq, Hk, D, pages, page, most, kind, 0),
        _ATTEND_STRIDES.pack(sq[0], sq[1], so[0], so[1], kp[0], kp[1], kp[2], vp[0], vp[1], vp[2],
                             *st, *sl), D ** -0.5 if scale is None else scale, window, sinks, ws,
        nbytes, _stream_on(dev, stream))
    if status:
        _check(status, "ssu_attend")


def describe_blocks(tensors) -> tuple[ctypes.Array, int]:
    """ABI descriptors for state tensors laid out as ``[num_blocks, ...]``: block k is the
    slice ``t[k]``, which must be contiguous (its bytes are copied verbatim)."""
    arr = (ssu_block_tensor_t * len(tensors))()
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or t.dim() < 1:
            raise TypeError("each state tensor must be a torch.Tensor of >= 1 dims")
        if t.dim() > 1 and not t[0].is_contiguous():
            raise ValueError("each block (t[k]) must be contiguous")
        item = t.element_size()
        block = item * (t[0].numel() if t.dim() > 1 else 1)
        arr[i] = ssu_block_tensor_t(t.data_ptr(), block, t.stride(0) * item, t.shape[0])
    return arr, len(tensors)


def ssu_copy_blocks(handle: int, tensors, src_idx, dst_idx, stream=None) -> None:
    """Copy block src_idx[i] -> dst_idx[i] of every tensor in ``tensors`` (each
    ``[num_blocks, ...]``), for every request i.  Enqueued on ``stream``."""
    if src_idx.dtype != dst_idx.dtype or src_idx.dtype not in (torch.int32, torch.int64):
        raise TypeError("src_idx and dst_idx must both be int32 or both int64")
    if src_idx.dim() != 1 or src_idx.shape != dst_idx.shape:
        raise ValueError("src_idx and dst_idx must be 1-D of the same length")
    if not (src_idx.is_contiguous() and dst_idx.is_contiguous()):
        raise ValueError("src_idx and dst_idx must be contiguous")
    arr, count = describe_blocks(tensors)
    dtype = SSU_INDEX_I64 if src_idx.dtype == torch.int64 else SSU_INDEX_I32
    _check(lib().ssu_copy_blocks(handle, arr, count, src_idx.data_ptr(), dst_idx.data_ptr(),
                                 src_idx.shape[0], dtype, _stream_ptr(stream)),
           "ssu_copy_blocks")


def ssu_copy_set_launch(handle: int, mode: int = SSU_COPY_AUTO, chunk_kib: int = 32,
                        stages: int = 8, threads: int = 256) -> None:
    cfg = ssu_copy_launch_t(mode, chunk_kib, stages, threads)
    _check(lib().ssu_copy_set_launch(handle, ctypes.byref(cfg)), "ssu_copy_set_launch")


class SelectiveStateUpdate:
    """Owns one handle; ``__call__`` is ``ssu_update`` on it."""

    def __init__(self, device: int | None = None):
        if device is None:
            device = torch.cuda.current_device()
        self.device = int(device)
        self.handle = ssu_create(self.device)

    def __call__(self, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
                 stream=None):
        ssu_update(self.handle, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D,
                   out, stream)
        return out

    def tokens(self, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C, D, out,
               intermediate=None, stream=None):
        ssu_update_tokens(self.handle, state_pool, state_batch_indices, x, dt, dt_bias, A, B, C,
                          D, out, intermediate, stream)
        return out

    def prompts_workspace_bytes(self, state_pool, x, B, state_batch_indices) -> int:
        return ssu_prompts_workspace_bytes(self.handle, state_pool, x, B, state_batch_indices)

    def prompts(self, state_pool, state_batch_indices, cu_tokens, x, dt, dt_bias, A, B, C, D,
                out, workspace=None, fresh=None, stream=None):
        ssu_update_prompts(self.handle, state_pool, state_batch_indices, cu_tokens, x, dt,
                           dt_bias, A, B, C, D, out, workspace, fresh, stream)
        return out

    def rotate_qk(self, q, k, v, q_weight, k_weight, table, positions, q_out, k_pages, v_pages,
                  slots, eps=1e-6, interleaved=False, stream=None):
        ssu_rotate_qk(self.handle, q, k, v, q_weight, k_weight, table, positions, q_out, k_pages,
                      v_pages, slots, eps, interleaved, stream)
        return q_out

    def attend_workspace_bytes(self, q, k_pages) -> int:
        return ssu_attend_workspace_bytes(self.handle, q, k_pages)

    def attend(self, q, k_pages, v_pages, page_table, lengths, out, workspace=None, scale=None,
               window=0, sinks=0, stream=None):
        ssu_attend(self.handle, q, k_pages, v_pages, page_table, lengths, out, workspace, scale,
                   window, sinks, stream)
        return out

    def copy_blocks(self, tensors, src_idx, dst_idx, stream=None):
        ssu_copy_blocks(self.handle, tensors, src_idx, dst_idx, stream)

    def get_error(self, stream=None):
        return ssu_get_error(self.handle, stream)

    def set_launch(self, *args, **kw):
        ssu_set_launch(self.handle, *args, **kw)

    def close(self):
        if self.handle:
            ssu_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
