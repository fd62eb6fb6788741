"""ctypes binding of libdora_hip.so (the C ABI declared in include/dora.h).

Argument marshalling only: these functions check that the torch tensors they
are given have the shapes, dtypes and device the C ABI expects, pass their data
pointers and torch's current HIP stream, and raise DoraError on a non-zero
status.  Every step of the computation runs in the HIP kernels; there is no
fallback.  Importing this module raises ImportError when the library has not
been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# DORA_HIP_LIB selects another build of the same library (the host-sanitizer
# build of the CPU validation check); by default the in-tree libdora_hip.so.
LIB_PATH = os.environ.get("DORA_HIP_LIB") or os.path.join(_HERE, "libdora_hip.so")

DORA_OK, DORA_INVALID_ARG, DORA_UNSUPPORTED, DORA_HIP_ERROR = 0, 1, 2, 3
DTYPE_CODE = {torch.bfloat16: 0, torch.float16: 1}

EXPORTS = (
    "dora_norm_workspace_bytes",
    "dora_norm_factored",
    "dora_norm_factored_cached",
    "dora_row_sqnorm",
    "dora_compose_fwd",
    "dora_lora_compose_fwd",
    "dora_lora_compose_bwd_workspace_bytes",
    "dora_lora_compose_bwd",
    "dora_compose_bwd_workspace_bytes",
    "dora_compose_bwd",
    "dora_compose_bwd_noalloc",
    "dora_norm_bwd_workspace_bytes",
    "dora_norm_bwd",
    "dora_norm_bwd_slab",
    "dora_q8_pack",
    "dora_q8_pack_weight",
    "dora_q8_unpack",
    "dora_q8_linear_workspace_bytes",
    "dora_q8_linear_fwd",
    "dora_q8_linear_bwd_workspace_bytes",
    "dora_q8_linear_bwd",
    "dora_q8_lora_compose_bwd_workspace_bytes",
    "dora_q8_lora_compose_bwd",
    "dora_q8_grad_a_workspace_bytes",
    "dora_q8_grad_a",
    "dora_q4_pack_weight",
    "dora_q4_unpack_weight",
    "dora_q4_linear_workspace_bytes",
    "dora_q4_linear_fwd",
    "dora_q4_linear_bwd_workspace_bytes",
    "dora_q4_linear_bwd",
    "dora_q4_plan",
    "dora_q4_norm_workspace_bytes",
    "dora_q4_norm_cached",
    "dora_adapter_sort_workspace_bytes",
    "dora_adapter_sort",
    "dora_adapter_gather",
    "dora_adapter_combine",
    "dora_adapter_combine_bwd",
    "dora_last_error",
    "dora_version",
)


class DoraError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"status {status}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc for gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.dora_norm_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.dora_norm_workspace_bytes.restype = sz
    lib.dora_norm_factored.argtypes = [vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, sz, vp]
    lib.dora_norm_factored.restype = i32
    lib.dora_norm_factored_cached.argtypes = [vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, sz, vp]
    lib.dora_norm_factored_cached.restype = i32
    lib.dora_row_sqnorm.argtypes = [vp, i64, i64, i32, vp, vp]
    lib.dora_row_sqnorm.restype = i32
    lib.dora_compose_fwd.argtypes = [vp, vp, vp, vp, f32, i64, i64, i32, i32, vp, vp]
    lib.dora_compose_fwd.restype = i32
    lib.dora_lora_compose_fwd.argtypes = [vp, vp, vp, vp, vp, f32, i64, i64, i64, i32, i32, vp, vp]
    lib.dora_lora_compose_fwd.restype = i32
    lib.dora_lora_compose_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    lib.dora_lora_compose_bwd_workspace_bytes.restype = sz
    lib.dora_lora_compose_bwd.argtypes = [vp, vp, vp, vp, vp, vp, f32, i64, i64, i64, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.dora_lora_compose_bwd.restype = i32
    lib.dora_compose_bwd_workspace_bytes.argtypes = [i64, i64]
    lib.dora_compose_bwd_workspace_bytes.restype = sz
    lib.dora_compose_bwd.argtypes = [vp, vp, vp, vp, vp, f32, i64, i64, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.dora_compose_bwd.restype = i32
    lib.dora_compose_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, f32, i64, i64, i32, i32, vp, vp, vp, vp]
    lib.dora_compose_bwd_noalloc.restype = i32
    lib.dora_norm_bwd_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.dora_norm_bwd_workspace_bytes.restype = sz
    lib.dora_norm_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, vp, sz, vp]
    lib.dora_norm_bwd.restype = i32
    lib.dora_norm_bwd_slab.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, f32, i32, i32, vp, vp, vp, sz, vp]
    lib.dora_norm_bwd_slab.restype = i32
    lib.dora_q8_pack.argtypes = lib.dora_q8_pack_weight.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.dora_q8_pack.restype = lib.dora_q8_pack_weight.restype = i32
    lib.dora_q8_unpack.argtypes = [vp, vp, i64, i64, i32, i32, vp, vp]
    lib.dora_q8_unpack.restype = i32
    for name in ("dora_q8_linear_workspace_bytes", "dora_q8_linear_bwd_workspace_bytes",
                 "dora_q8_lora_compose_bwd_workspace_bytes", "dora_q8_grad_a_workspace_bytes"):
        getattr(lib, name).argtypes = [i64, i64, i64]
        getattr(lib, name).restype = sz
    for name in ("dora_q8_linear_fwd", "dora_q8_linear_bwd"):
        getattr(lib, name).argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        getattr(lib, name).restype = i32
    lib.dora_q8_lora_compose_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, i64, i64, i64, i32, i32, vp, vp, vp, vp,
                                             vp, vp, sz, vp]
    lib.dora_q8_lora_compose_bwd.restype = i32
    lib.dora_q8_grad_a.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
    lib.dora_q8_grad_a.restype = i32
    lib.dora_q4_pack_weight.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    lib.dora_q4_unpack_weight.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    lib.dora_q4_pack_weight.restype = lib.dora_q4_unpack_weight.restype = i32
    for name in ("dora_q4_linear_workspace_bytes", "dora_q4_linear_bwd_workspace_bytes",
                 "dora_adapter_sort_workspace_bytes"):
        getattr(lib, name).argtypes = [i64, i64, i64]
        getattr(lib, name).restype = sz
    for name in ("dora_q4_linear_fwd", "dora_q4_linear_bwd"):
        getattr(lib, name).argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        getattr(lib, name).restype = i32
    lib.dora_q4_plan.argtypes = [i64, i64, i64, i32, vp]
    lib.dora_q4_plan.restype = i32
    lib.dora_q4_norm_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.dora_q4_norm_workspace_bytes.restype = sz
    lib.dora_q4_norm_cached.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, f32, i32, vp, vp, sz, vp]
    lib.dora_q4_norm_cached.restype = i32
    lib.dora_adapter_sort.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.dora_adapter_sort.restype = i32
    lib.dora_adapter_gather.argtypes = [vp, vp, i64, i64, i64, i32, vp, vp]
    lib.dora_adapter_gather.restype = i32
    lib.dora_adapter_combine.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    lib.dora_adapter_combine.restype = i32
    lib.dora_adapter_combine_bwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp]
    lib.dora_adapter_combine_bwd.restype = i32
    lib.dora_last_error.argtypes = []
    lib.dora_last_error.restype = ctypes.c_char_p
    lib.dora_version.argtypes = []
    lib.dora_version.restype = ctypes.c_char_p
    return lib


LIB = _load()


def dora_last_error() -> str:
    return LIB.dora_last_error().decode()


def dora_version() -> str:
    return LIB.dora_version().decode()


def _check(status: int) -> None:
    if status != DORA_OK:
        raise DoraError(status, dora_last_error())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _matrix(t, name, shape, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _code(t) -> int:
    if t.dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype}; bf16 and fp16 are")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    return DTYPE_CODE[t.dtype]


def dora_norm_workspace_bytes(out: int, in_: int, r: int, dtype=torch.bfloat16) -> int:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(LIB.dora_norm_workspace_bytes(out, in_, r, code))


def dora_compose_bwd_workspace_bytes(T: int, out: int) -> int:
    return int(LIB.dora_compose_bwd_workspace_bytes(T, out))


def dora_norm_factored(W0, A, B, s: float, norm_out=None, workspace=None):
    """norm_out[i] = ||W0_i + s B_i A||_2 (fp32) via the factored kernels."""
    code = _code(W0)
    out, in_ = W0.shape
    r = A.shape[0]
    dev = W0.device
    _matrix(W0, "W0", (out, in_), W0.dtype, dev)
    _matrix(A, "A", (r, in_), W0.dtype, dev)
    _matrix(B, "B", (out, r), W0.dtype, dev)
    if norm_out is None:
        norm_out = torch.empty(out, dtype=torch.float32, device=dev)
    _matrix(norm_out, "norm_out", (out,), torch.float32, dev)
    need = dora_norm_workspace_bytes(out, in_, r, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_norm_factored(_ptr(W0), _ptr(A), _ptr(B), out, in_, r, float(s), code, _ptr(norm_out),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev)))
    return norm_out


def dora_norm_factored_cached(W0, A, B, base_sq, s: float, norm_out=None, workspace=None):
    """dora_norm_factored with the base term ||W0_i||^2 taken from base_sq (fp32 [out])."""
    code = _code(W0)
    out, in_ = W0.shape
    r = A.shape[0]
    dev = W0.device
    _matrix(W0, "W0", (out, in_), W0.dtype, dev)
    _matrix(A, "A", (r, in_), W0.dtype, dev)
    _matrix(B, "B", (out, r), W0.dtype, dev)
    _matrix(base_sq, "base_sq", (out,), torch.float32, dev)
    if norm_out is None:
        norm_out = torch.empty(out, dtype=torch.float32, device=dev)
    _matrix(norm_out, "norm_out", (out,), torch.float32, dev)
    need = dora_norm_workspace_bytes(out, in_, r, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_norm_factored_cached(_ptr(W0), _ptr(A), _ptr(B), _ptr(base_sq), out, in_, r, float(s), code,
                                         _ptr(norm_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(dev)))
    return norm_out


def dora_row_sqnorm(W0, sq_out=None):
    """sq_out[i] = ||W0_i||^2 (fp32)."""
    code = _code(W0)
    out, in_ = W0.shape
    dev = W0.device
    _matrix(W0, "W0", (out, in_), W0.dtype, dev)
    if sq_out is None:
        sq_out = torch.empty(out, dtype=torch.float32, device=dev)
    _matrix(sq_out, "sq_out", (out,), torch.float32, dev)
    _check(LIB.dora_row_sqnorm(_ptr(W0), out, in_, code, _ptr(sq_out), _stream(dev)))
    return sq_out


def dora_compose_fwd(base, lora, mag, norm, s: float, add_base: bool = False, y=None):
    """y = (g-1)*base + g*s*lora (+ base), g = mag/norm per column."""
    code = _code(base)
    T, out = base.shape
    dev = base.device
    _matrix(lora, "lora", (T, out), base.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(base)
    _matrix(y, "y", (T, out), base.dtype, dev)
    _check(LIB.dora_compose_fwd(_ptr(base), _ptr(lora), _ptr(mag), _ptr(norm), float(s), T, out, code,
                                int(bool(add_base)), _ptr(y), _stream(dev)))
    return y


def dora_lora_compose_fwd(base, h, B, mag, norm, s: float, add_base: bool = False, y=None):
    """y = (g-1)*base + g*s*(h B^T) (+ base), g = mag/norm per column; lora never stored."""
    code = _code(base)
    T, out = base.shape
    r = h.shape[1]
    dev = base.device
    _matrix(h, "h", (T, r), base.dtype, dev)
    _matrix(B, "B", (out, r), base.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(base)
    _matrix(y, "y", (T, out), base.dtype, dev)
    _check(LIB.dora_lora_compose_fwd(_ptr(base), _ptr(h), _ptr(B), _ptr(mag), _ptr(norm), float(s), T, out, r, code,
                                     int(bool(add_base)), _ptr(y), _stream(dev)))
    return y


def dora_lora_compose_bwd_workspace_bytes(T: int, out: int, r: int) -> int:
    return int(LIB.dora_lora_compose_bwd_workspace_bytes(T, out, r))


def dora_lora_compose_bwd(dy, base, h, B, mag, norm, s: float, add_base: bool = False, d_base=None, d_B=None,
                          d_mag=None, workspace=None, want_d_base: bool = True):
    """(d_base, d_B, d_mag) of the fused compose; d_base is None if not wanted."""
    code = _code(dy)
    T, out = dy.shape
    r = h.shape[1]
    dev = dy.device
    _matrix(base, "base", (T, out), dy.dtype, dev)
    _matrix(h, "h", (T, r), dy.dtype, dev)
    _matrix(B, "B", (out, r), dy.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    if d_base is None and want_d_base:
        d_base = torch.empty_like(dy)
    if d_B is None:
        d_B = torch.empty_like(B)
    if d_mag is None:
        d_mag = torch.empty(out, dtype=torch.float32, device=dev)
    if d_base is not None:
        _matrix(d_base, "d_base", (T, out), dy.dtype, dev)
    _matrix(d_B, "d_B", (out, r), dy.dtype, dev)
    _matrix(d_mag, "d_mag", (out,), torch.float32, dev)
    need = dora_lora_compose_bwd_workspace_bytes(T, out, r)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_lora_compose_bwd(_ptr(dy), _ptr(base), _ptr(h), _ptr(B), _ptr(mag), _ptr(norm), float(s), T, out,
                                     r, code, int(bool(add_base)), _ptr(d_base), _ptr(d_B), _ptr(d_mag),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev)))
    return d_base, d_B, d_mag


def dora_compose_bwd(dy, base, lora, mag, norm, s: float, add_base: bool = False, d_lora=None, d_base=None,
                     d_mag=None, workspace=None, want_d_base: bool = True):
    """(d_lora, d_base, d_mag) of the compose; d_base is None if not wanted."""
    code = _code(dy)
    T, out = dy.shape
    dev = dy.device
    _matrix(base, "base", (T, out), dy.dtype, dev)
    _matrix(lora, "lora", (T, out), dy.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    if d_lora is None:
        d_lora = torch.empty_like(dy)
    if d_base is None and want_d_base:
        d_base = torch.empty_like(dy)
    if d_mag is None:
        d_mag = torch.empty(out, dtype=torch.float32, device=dev)
    _matrix(d_lora, "d_lora", (T, out), dy.dtype, dev)
    if d_base is not None:
        _matrix(d_base, "d_base", (T, out), dy.dtype, dev)
    _matrix(d_mag, "d_mag", (out,), torch.float32, dev)
    need = dora_compose_bwd_workspace_bytes(T, out)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_compose_bwd(_ptr(dy), _ptr(base), _ptr(lora), _ptr(mag), _ptr(norm), float(s), T, out, code,
                                int(bool(add_base)), _ptr(d_lora), _ptr(d_base), _ptr(d_mag), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(dev)))
    return d_lora, d_base, d_mag


def dora_compose_bwd_noalloc(dy, base, lora, mag, norm, s: float, add_base: bool = False, d_lora=None, d_base=None,
                             d_mag=None, want_d_base: bool = True):
    """dora_compose_bwd with the library's own scratch in place of a workspace
    (the entry point that allocates nothing; outputs passed in are written in
    place, missing ones are allocated here, outside the library call)."""
    code = _code(dy)
    T, out = dy.shape
    dev = dy.device
    _matrix(base, "base", (T, out), dy.dtype, dev)
    _matrix(lora, "lora", (T, out), dy.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    if d_lora is None:
        d_lora = torch.empty_like(dy)
    if d_base is None and want_d_base:
        d_base = torch.empty_like(dy)
    if d_mag is None:
        d_mag = torch.empty(out, dtype=torch.float32, device=dev)
    _matrix(d_lora, "d_lora", (T, out), dy.dtype, dev)
    if d_base is not None:
        _matrix(d_base, "d_base", (T, out), dy.dtype, dev)
    _matrix(d_mag, "d_mag", (out,), torch.float32, dev)
    _check(LIB.dora_compose_bwd_noalloc(_ptr(dy), _ptr(base), _ptr(lora), _ptr(mag), _ptr(norm), float(s), T, out,
                                        code, int(bool(add_base)), _ptr(d_lora), _ptr(d_base), _ptr(d_mag),
                                        _stream(dev)))
    return d_lora, d_base, d_mag


def dora_norm_bwd_workspace_bytes(out: int, in_: int, r: int, dtype=torch.bfloat16) -> int:
    return int(LIB.dora_norm_bwd_workspace_bytes(out, in_, r, DTYPE_CODE.get(dtype, -1)))


def dora_norm_bwd(W0, A, B, norm, d_norm, s: float, d_A=None, d_B=None, workspace=None):
    """(d_A, d_B): the gradients of sum(d_norm * n) with respect to A and B,
    n = the weight norm of W0 + s B A (norm: the forward's n)."""
    code = _code(W0)
    out, in_ = W0.shape
    r = A.shape[0]
    dev = W0.device
    _matrix(W0, "W0", (out, in_), W0.dtype, dev)
    _matrix(A, "A", (r, in_), W0.dtype, dev)
    _matrix(B, "B", (out, r), W0.dtype, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    _matrix(d_norm, "d_norm", (out,), torch.float32, dev)
    if d_A is None:
        d_A = torch.empty_like(A)
    if d_B is None:
        d_B = torch.empty_like(B)
    _matrix(d_A, "d_A", (r, in_), W0.dtype, dev)
    _matrix(d_B, "d_B", (out, r), W0.dtype, dev)
    need = dora_norm_bwd_workspace_bytes(out, in_, r, W0.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_norm_bwd(_ptr(W0), _ptr(A), _ptr(B), _ptr(norm), _ptr(d_norm), out, in_, r, float(s), code,
                             _ptr(d_A), _ptr(d_B), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(dev)))
    return d_A, d_B


def dora_norm_bwd_slab(W0, A, B, norm, d_norm, s: float, d_A, add: bool):
    """d_B of a slab of rows; its part of d_A [r x in] goes to the fp32 ``d_A``,
    added to what that holds with ``add``."""
    code = _code(W0)
    out, in_ = W0.shape
    r = A.shape[0]
    dev = W0.device
    _matrix(W0, "W0", (out, in_), W0.dtype, dev)
    _matrix(A, "A", (r, in_), W0.dtype, dev)
    _matrix(B, "B", (out, r), W0.dtype, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    _matrix(d_norm, "d_norm", (out,), torch.float32, dev)
    _matrix(d_A, "d_A", (r, in_), torch.float32, dev)
    d_B = torch.empty_like(B)
    need = dora_norm_bwd_workspace_bytes(out, in_, r, W0.dtype)
    workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(LIB.dora_norm_bwd_slab(_ptr(W0), _ptr(A), _ptr(B), _ptr(norm), _ptr(d_norm), out, in_, r, float(s), code,
                                  int(bool(add)), _ptr(d_A), _ptr(d_B), _ptr(workspace), workspace.numel(),
                                  _stream(dev)))
    return d_B


# ------------------------------------------------------------ the frozen side in 8 bits
#
# A packed matrix is a pair (q, e): torch.float8_e4m3fn values and uint8 exponent
# bytes in the layout of include/dora.h.  These calls run on the tensors' own
# device, whatever the current one is.  They are short calls of a serving loop, so
# what they do besides the launch is kept small (the raw stream handle, no device
# switch where the device is the current one).

Q8_BLOCK = 128


def q8_row_shapes(rows: int, cols: int):
    """Shapes of (q, e) for packed rows [rows x cols]."""
    nb = -(-cols // Q8_BLOCK)
    return (rows, nb * Q8_BLOCK), (rows, -(-nb // 4) * 4)


def q8_weight_shapes(out: int, in_: int):
    """Shapes of (q, e) for a packed weight [out x in]."""
    ob = -(-out // Q8_BLOCK)
    q, e = q8_row_shapes(ob, in_)
    return (ob * Q8_BLOCK, q[1]), e


def _packed(q, e, name, shapes, device):
    if (q.shape != shapes[0] or e.shape != shapes[1] or q.dtype != torch.float8_e4m3fn or e.dtype != torch.uint8
            or q.device != device or e.device != device or not q.is_contiguous() or not e.is_contiguous()):
        _matrix(q, name, shapes[0], torch.float8_e4m3fn, device)  # says which it is
        _matrix(e, name + "'s exponents", shapes[1], torch.uint8, device)
    if q.data_ptr() % 16 or e.data_ptr() % 4:
        raise ValueError(f"{name} must be 16-byte aligned, its exponents 4-byte")


def _dtype_code(dtype) -> int:
    if dtype not in DTYPE_CODE:
        raise ValueError(f"unsupported dtype {dtype}; bf16 and fp16 are")
    return DTYPE_CODE[dtype]


def _on_gpu(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device")
    return t.device


class _Stay:
    """In place of a device switch where there is nothing to switch."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_STAY = _Stay()


def _on_device(device):
    return _STAY if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _new_packed(shapes, device):
    return (torch.empty(shapes[0], dtype=torch.float8_e4m3fn, device=device),
            torch.empty(shapes[1], dtype=torch.uint8, device=device))


def _workspace(need: int, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def dora_q8_pack(x):
    """(q, e): the rows of x [T x K] in blocks of 128 columns."""
    code = _code(x)
    rows, cols = x.shape
    _matrix(x, "x", (rows, cols))
    with _on_device(x.device):
        q, e = _new_packed(q8_row_shapes(rows, cols), x.device)
        _check(LIB.dora_q8_pack(_ptr(x), rows, cols, code, _ptr(q), _ptr(e), _raw_stream(x.device)))
    return q, e


def dora_q8_pack_weight(W):
    """(q, e): the weight W [out x in] in blocks of 128 x 128."""
    code = _code(W)
    out, in_ = W.shape
    _matrix(W, "W", (out, in_))
    with _on_device(W.device):
        q, e = _new_packed(q8_weight_shapes(out, in_), W.device)
        _check(LIB.dora_q8_pack_weight(_ptr(W), out, in_, code, _ptr(q), _ptr(e), _raw_stream(W.device)))
    return q, e


def dora_q8_unpack(q, e, rows: int, cols: int, dtype, weight: bool = False):
    """The values of packed rows, or of the first rows of a packed weight, in dtype."""
    code, dev = _dtype_code(dtype), _on_gpu(q, "q")
    if weight:
        if not 0 <= rows <= q.shape[0]:
            raise ValueError(f"rows {rows} out of range of a packed weight of {q.shape[0]}")
        _packed(q, e, "q", q8_weight_shapes(q.shape[0], cols), dev)
    else:
        _packed(q, e, "q", q8_row_shapes(rows, cols), dev)
    with _on_device(dev):
        x = torch.empty((rows, cols), dtype=dtype, device=dev)
        _check(LIB.dora_q8_unpack(_ptr(q), _ptr(e), rows, cols, int(weight), code, _ptr(x), _raw_stream(dev)))
    return x


def dora_q8_linear_fwd(xq, xe, wq, we, out: int, in_: int, dtype):
    """y [T x out] = x W^T from packed rows [T x in] and a packed weight [out x in]."""
    code, dev, T = _dtype_code(dtype), _on_gpu(xq, "xq"), xq.shape[0]
    _packed(xq, xe, "xq", q8_row_shapes(T, in_), dev)
    _packed(wq, we, "wq", q8_weight_shapes(out, in_), dev)
    with _on_device(dev):
        y = torch.empty((T, out), dtype=dtype, device=dev)
        need = int(LIB.dora_q8_linear_workspace_bytes(T, out, in_))
        ws = _workspace(need, dev)
        _check(LIB.dora_q8_linear_fwd(_ptr(xq), _ptr(xe), _ptr(wq), _ptr(we), T, out, in_, code, _ptr(y), _ptr(ws),
                                      need, _raw_stream(dev)))
    return y


def dora_q8_linear_bwd(gq, ge, wq, we, out: int, in_: int, dtype):
    """dx [T x in] = g W from packed rows [T x out] and a packed weight [out x in]."""
    code, dev, T = _dtype_code(dtype), _on_gpu(gq, "gq"), gq.shape[0]
    _packed(gq, ge, "gq", q8_row_shapes(T, out), dev)
    _packed(wq, we, "wq", q8_weight_shapes(out, in_), dev)
    with _on_device(dev):
        dx = torch.empty((T, in_), dtype=dtype, device=dev)
        need = int(LIB.dora_q8_linear_bwd_workspace_bytes(T, out, in_))
        ws = _workspace(need, dev)
        _check(LIB.dora_q8_linear_bwd(_ptr(gq), _ptr(ge), _ptr(wq), _ptr(we), T, out, in_, code, _ptr(dx), _ptr(ws),
                                      need, _raw_stream(dev)))
    return dx


def _aligned(t):
    """t itself, or a copy where a slice starts off a 16-byte boundary."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def dora_q8_lora_compose_bwd(dy, bq, be, h, B, mag, norm, s: float, add_base: bool = False, want_d_base: bool = True,
                             packed: bool = False):
    """(d_base, d_B, d_mag) of the fused compose with the base from packed rows.
    d_base is None if not wanted, or with packed the pair (q, e)."""
    code = _code(dy)
    T, out = dy.shape
    r, dev = h.shape[1], dy.device
    _matrix(dy, "dy", (T, out))
    _packed(bq, be, "bq", q8_row_shapes(T, out), dev)
    _matrix(h, "h", (T, r), dy.dtype, dev)
    _matrix(B, "B", (out, r), dy.dtype, dev)
    _matrix(mag, "mag", (out,), torch.float32, dev)
    _matrix(norm, "norm", (out,), torch.float32, dev)
    dy, h, B = _aligned(dy), _aligned(h), _aligned(B)
    with _on_device(dev):
        d_base = q = e = None
        if want_d_base and packed:
            q, e = _new_packed(q8_row_shapes(T, out), dev)
        elif want_d_base:
            d_base = torch.empty((T, out), dtype=dy.dtype, device=dev)
        d_B = torch.empty((out, r), dtype=dy.dtype, device=dev)
        d_mag = torch.empty(out, dtype=torch.float32, device=dev)
        need = int(LIB.dora_q8_lora_compose_bwd_workspace_bytes(T, out, r))
        ws = _workspace(need, dev)
        _check(LIB.dora_q8_lora_compose_bwd(_ptr(dy), _ptr(bq), _ptr(be), _ptr(h), _ptr(B), _ptr(mag), _ptr(norm),
                                            float(s), T, out, r, code, int(bool(add_base)), _ptr(d_base), _ptr(q),
                                            _ptr(e), _ptr(d_B), _ptr(d_mag), _ptr(ws), need, _raw_stream(dev)))
    return (q, e) if q is not None else d_base, d_B, d_mag


def dora_q8_grad_a(dh, xq, xe, in_: int):
    """d_A [r x in] = d_h^T x from packed rows x [T x in]."""
    code = _code(dh)
    T, r = dh.shape
    dev = dh.device
    _matrix(dh, "dh", (T, r))
    _packed(xq, xe, "xq", q8_row_shapes(T, in_), dev)
    dh = _aligned(dh)
    with _on_device(dev):
        d_A = torch.empty((r, in_), dtype=dh.dtype, device=dev)
        need = int(LIB.dora_q8_grad_a_workspace_bytes(T, in_, r))
        ws = _workspace(need, dev)
        _check(LIB.dora_q8_grad_a(_ptr(dh), _ptr(xq), _ptr(xe), T, in_, r, code, _ptr(d_A), _ptr(ws), need,
                                  _raw_stream(dev)))
    return d_A


# ------------------------------------------------------------ the frozen weight in 4 bits
#
# A packed weight is a pair (q, e) of uint8 tensors in the layout of include/dora.h.

Q4_ROWS, Q4_COLS = 32, 64  # a tile


def q4_weight_shapes(out: int, in_: int):
    """Shapes of (q, e) for a packed weight [out x in]."""
    tiles = (-(-out // Q4_ROWS), -(-in_ // Q4_COLS))
    return (*tiles, 1024), (*tiles, 64)


def _q4_packed(q, e, shapes, device):
    if (q.shape != shapes[0] or e.shape != shapes[1] or q.dtype != torch.uint8 or e.dtype != torch.uint8
            or q.device != device or e.device != device or not q.is_contiguous() or not e.is_contiguous()):
        _matrix(q, "the packed weight", shapes[0], torch.uint8, device)  # says which it is
        _matrix(e, "the packed weight's exponents", shapes[1], torch.uint8, device)
    if q.data_ptr() % 16 or e.data_ptr() % 16:
        raise ValueError("the packed weight and its exponents must be 16-byte aligned")


def dora_q4_pack_weight(W):
    """(q, e): the weight W [out x in] in 4-bit blocks of 32 columns."""
    code = _code(W)
    out, in_ = W.shape
    _matrix(W, "W", (out, in_))
    with _on_device(W.device):
        qs, es = q4_weight_shapes(out, in_)
        q = torch.empty(qs, dtype=torch.uint8, device=W.device)
        e = torch.empty(es, dtype=torch.uint8, device=W.device)
        _check(LIB.dora_q4_pack_weight(_ptr(W), out, in_, code, _ptr(q), _ptr(e), _raw_stream(W.device)))
    return q, e


def dora_q4_unpack_weight(q, e, rows: int, cols: int, dtype):
    """The values of the first ``rows`` rows of a packed weight of ``cols`` columns, in dtype."""
    code, dev = _dtype_code(dtype), _on_gpu(q, "q")
    if not 0 <= rows <= q.shape[0] * Q4_ROWS:
        raise ValueError(f"rows {rows} out of range of a packed weight of {q.shape[0] * Q4_ROWS}")
    _q4_packed(q, e, q4_weight_shapes(q.shape[0] * Q4_ROWS, cols), dev)
    with _on_device(dev):
        W = torch.empty((rows, cols), dtype=dtype, device=dev)
        _check(LIB.dora_q4_unpack_weight(_ptr(q), _ptr(e), rows, cols, code, _ptr(W), _raw_stream(dev)))
    return W


def dora_q4_linear_fwd(x, q, e, out: int):
    """y [T x out] = x W^T from x [T x in] and a packed weight [out x in]."""
    code = _code(x)
    (T, in_), dev = x.shape, x.device
    _matrix(x, "x", (T, in_))
    _q4_packed(q, e, q4_weight_shapes(out, in_), dev)
    x = _aligned(x)
    with _on_device(dev):
        y = torch.empty((T, out), dtype=x.dtype, device=dev)
        need = int(LIB.dora_q4_linear_workspace_bytes(T, out, in_))
        ws = _workspace(need, dev)
        _check(LIB.dora_q4_linear_fwd(_ptr(x), _ptr(q), _ptr(e), T, out, in_, code, _ptr(y), _ptr(ws), need,
                                      _raw_stream(dev)))
    return y


def dora_q4_linear_bwd(g, q, e, in_: int):
    """dx [T x in] = g W from g [T x out] and a packed weight [out x in]."""
    code = _code(g)
    (T, out), dev = g.shape, g.device
    _matrix(g, "g", (T, out))
    _q4_packed(q, e, q4_weight_shapes(out, in_), dev)
    g = _aligned(g)
    with _on_device(dev):
        dx = torch.empty((T, in_), dtype=g.dtype, device=dev)
        need = int(LIB.dora_q4_linear_bwd_workspace_bytes(T, out, in_))
        ws = _workspace(need, dev)
        _check(LIB.dora_q4_linear_bwd(_ptr(g), _ptr(q), _ptr(e), T, out, in_, code, _ptr(dx), _ptr(ws), need,
                                      _raw_stream(dev)))
    return dx


def dora_q4_plan(T: int, out: int, in_: int, product: int) -> tuple[int, ...]:
    """(tile rows, tile columns, tiles of whole rounds, other tiles, ranges of these, workgroups) of the kernel
    that the forward (product 0), the backward (1) or the norm's product (2) of these sizes takes."""
    plan = (ctypes.c_int64 * 6)()
    _check(LIB.dora_q4_plan(T, out, in_, product, ctypes.addressof(plan)))
    return tuple(plan)


def dora_q4_norm_cached(q, e, A, B, base_sq, s: float):
    """||W + s*B*A|| per row (fp32 [out]) of a packed weight, with ||W_i||^2 from base_sq (fp32 [out])."""
    code = _code(A)
    (r, in_), out, dev = _shape2(A, "A"), _shape2(B, "B")[0], A.device
    _matrix(A, "A", (r, in_))
    _matrix(B, "B", (out, r), A.dtype, dev)
    _matrix(base_sq, "base_sq", (out,), torch.float32, dev)
    _q4_packed(q, e, q4_weight_shapes(out, in_), dev)
    A, B = _aligned(A), _aligned(B)
    with _on_device(dev):
        n = torch.empty(out, dtype=torch.float32, device=dev)
        need = int(LIB.dora_q4_norm_workspace_bytes(out, in_, r, code))
        ws = _workspace(need, dev)
        _check(LIB.dora_q4_norm_cached(_ptr(q), _ptr(e), _ptr(A), _ptr(B), _ptr(base_sq), out, in_, r, float(s), code,
                                       _ptr(n), _ptr(ws), need, _raw_stream(dev)))
    return n


# ------------------------------------------------------------ tokens sorted by adapter


def _shape2(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected two dimensions")
    return t.shape


def dora_adapter_sort(ids, adapters: int):
    """(order [T k], place [T x k], bounds [adapters + 1]), int32, of ids [T x k] (int64 or int32)."""
    if ids.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"ids are {ids.dtype}; int64 and int32 are taken")
    dev = _on_gpu(ids, "ids")
    T, k = _shape2(ids, "ids")
    _matrix(ids, "ids", (T, k))
    with _on_device(dev):
        order = torch.empty(T * k, dtype=torch.int32, device=dev)
        place = torch.empty((T, k), dtype=torch.int32, device=dev)
        bounds = torch.empty(max(adapters, 0) + 1, dtype=torch.int32, device=dev)
        need = int(LIB.dora_adapter_sort_workspace_bytes(T, k, adapters))
        ws = _workspace(need, dev)
        _check(LIB.dora_adapter_sort(_ptr(ids), ids.element_size(), T, k, adapters, _ptr(order), _ptr(place),
                                     _ptr(bounds), _ptr(ws), need, _raw_stream(dev)))
    return order, place, bounds


def dora_adapter_gather(x, place):
    """rows [T k x D]: x[t] at the row of each of its slots, zeros at those without an adapter."""
    code = _code(x)
    (T, D), dev = _shape2(x, "x"), x.device
    k = _shape2(place, "place")[1]
    _matrix(x, "x", (T, D))
    _matrix(place, "place", (T, k), torch.int32, dev)
    with _on_device(dev):
        rows = torch.empty((T * k, D), dtype=x.dtype, device=dev)
        _check(LIB.dora_adapter_gather(_ptr(x), _ptr(place), T, k, D, code, _ptr(rows), _raw_stream(dev)))
    return rows


def dora_adapter_combine(rows, weights, place, base=None):
    """y [T x D]: base (or zeros) plus each token's rows times their weights (fp32 [T x k], or None for ones)."""
    code = _code(rows)
    (T, k), D, dev = _shape2(place, "place"), _shape2(rows, "rows")[1], rows.device
    _matrix(rows, "rows", (T * k, D))
    _matrix(place, "place", (T, k), torch.int32, dev)
    if weights is not None:
        _matrix(weights, "weights", (T, k), torch.float32, dev)
    if base is not None:
        _matrix(base, "base", (T, D), rows.dtype, dev)
    with _on_device(dev):
        y = torch.empty((T, D), dtype=rows.dtype, device=dev)
        _check(LIB.dora_adapter_combine(_ptr(rows), _ptr(weights), _ptr(place), _ptr(base), T, k, D, code, _ptr(y),
                                        _raw_stream(dev)))
    return y


def dora_adapter_combine_bwd(dy, rows, weights, place, want_rows: bool = True, want_weights: bool = True):
    """(d_rows [T k x D], d_weights [T x k] fp32) of the combination, None where not wanted (rows: None without
    the latter)."""
    code = _code(dy)
    (T, D), k, dev = _shape2(dy, "dy"), _shape2(place, "place")[1], dy.device
    _matrix(dy, "dy", (T, D))
    if rows is not None:
        _matrix(rows, "rows", (T * k, D), dy.dtype, dev)
    elif want_weights:
        raise ValueError("the gradient of the weights needs the rows")
    _matrix(place, "place", (T, k), torch.int32, dev)
    if weights is not None:
        _matrix(weights, "weights", (T, k), torch.float32, dev)
    with _on_device(dev):
        d_rows = torch.empty((T * k, D), dtype=dy.dtype, device=dev) if want_rows else None
        d_w = torch.empty((T, k), dtype=torch.float32, device=dev) if want_weights else None
        _check(LIB.dora_adapter_combine_bwd(_ptr(dy), _ptr(rows), _ptr(weights), _ptr(place), T, k, D, code,
                                            _ptr(d_rows), _ptr(d_w), _raw_stream(dev)))
    return d_rows, d_w
