"""PyTorch integration of the DoRA hot path: custom operators and a DoRA linear layer.

The press summary of arXiv:2603.22276 describes the fused kernels as a PyTorch
custom operator, which compiled graphs keep without breaks (paragraph on
framework compatibility). It also describes a three-tier dispatch (paragraph
on the dispatch tiers): training runs the fused forward and the fused
backward, inference runs the forward kernel alone, and whatever the kernels
cannot take goes to eager PyTorch.

This module registers:

* ``dora_amd::weight_norm`` -- the factored norm ||W0 + s*B*A|| per output row
  (fp32).  Callers that treat the norm as a constant (the usual DoRA reading)
  pass detached A and B.  Otherwise its autograd formula is
  ``dora_amd::weight_norm_backward``, the factored backward into A and B (W0
  is frozen and gets no gradient); ``weight_norm_cached`` has the same formula.
* ``dora_amd::lora_compose`` -- the compose with the adapter's second
  projection fused in: from h = x A^T and B it forms lora = h B^T inside the
  kernel and never stores it.  Its autograd formula is
  ``dora_amd::lora_compose_backward`` (d_base, d_B and d_mag without lora or
  d_lora), plus d_h = dy (g s .* B), a GEMM done by torch.
* ``dora_amd::row_sqnorm`` and ``dora_amd::weight_norm_cached`` -- the cached
  base term the page proposes as future work (W0 is frozen): ||W0_i||^2 once,
  then the norm that takes it instead of re-deriving it from W0.
* ``dora_amd::compose`` -- the stable compose (g - 1)*base + g*s*lora
  (+ base), g = m / n. Its autograd formula is the fused backward
  ``dora_amd::compose_backward``, which gives the gradients of base, lora and
  the magnitude m.
* the 8-bit operators: ``q8_pack`` / ``q8_pack_weight`` / ``q8_unpack`` /
  ``q8_unpack_weight`` (e4m3 blocks of 128 with a power-of-two scale each),
  ``q8_linear`` and ``q8_linear_backward`` (the frozen layer's product and its
  gradient of x, on packed operands), ``q8_lora_compose_backward`` (and
  ``_packed``: the compose's backward from the base kept in 8 bits) and
  ``q8_grad_a`` (the gradient of A from x kept in 8 bits).  ``q8_layer`` runs
  them together under autograd.
* the 4-bit weight: ``q4_pack_weight`` / ``q4_unpack_weight`` (e2m1 blocks of 32
  with a power-of-two scale each), ``q4_linear`` (x W0^T from 16-bit x) and
  ``q4_linear_backward`` (g W0), each the other's autograd formula, and
  ``q4_weight_norm``, the norm of a W0 held so, from the packed values.
* tokens sorted by adapter: ``adapter_sort`` (a batch's slots by adapter),
  ``adapter_gather`` (tokens' rows in that order) and ``adapter_combine`` (rows
  added up per token, with weights; ``adapter_combine_backward`` is its formula).
* ``DoRALinear`` -- a linear layer with frozen W0 and trainable A, B and m:
  y = x W0^T + compose(x W0^T, x A^T B^T, m, n, s), with n = ||W0 + s*B*A||
  detached by default.  With ``detach_norm=False`` the gradient also flows
  through n: the compose's formula gives dL/dn = -(m / n) * d_mag (L depends on
  n only through g = m / n; this [out]-sized product is the one step of the
  chain done by torch), and the norm's formula turns it into d_A and d_B.
  ``q8_weight`` and ``q4_weight`` hold W0 in 8 or 4 bits.
* ``DoRAAdapters`` -- several adapters over one W0, each token with its own.

Tiers (paragraph on the dispatch tiers): autograd records the compose only
when a gradient is needed (training: the fused forward, then the fused
backward); under ``torch.no_grad()`` or ``torch.inference_mode()`` the forward
kernel runs alone.  ``DoRALinear`` runs the compose with the second projection
fused in on both tiers, so lora = x A^T B^T is never stored.  The third tier
is eager PyTorch for inputs the kernels do not take: tensors on the CPU, matrix
dtypes other than bf16/fp16 (fp32), and a call the library refuses with
DORA_UNSUPPORTED.  Those run the plain, unfused torch form of each operator
(dense B A for the norm, the compose written out elementwise), computed in
fp32.  Supported inputs on a HIP device always take the kernels; a missing
library raises on import, it never falls back.

On that path every operator is argument marshalling around the C ABI
(``binding``); the arithmetic runs in the HIP kernels.
"""
from __future__ import annotations

import functools
import math
from typing import Optional

import numpy as np
import torch
import torch.autograd.forward_ad as fwad
import torch.nn.functional as F

from . import binding

Tensor = torch.Tensor


# ---------------------------------------------------------------- eager tier
#
# The plain PyTorch form of each operator, for inputs the kernels do not take
# (the page's fallback tier).  fp32 arithmetic, outputs in the matrices' dtype.


def _kernels_take(*mats: Tensor) -> bool:
    """True when the kernels take these matrix arguments: all on a HIP device,
    in bf16 or fp16."""
    return all(t.device.type == "cuda" and t.dtype in binding.DTYPE_CODE for t in mats)


def _unsupported(e: Exception) -> bool:
    return isinstance(e, binding.DoraError) and e.status == binding.DORA_UNSUPPORTED


def _eager_weight_norm(W0, A, B, s):
    V = W0.float() + s * (B.float() @ A.float())
    return torch.linalg.vector_norm(V, dim=1)


def _eager_row_sqnorm(W0):
    W = W0.float()
    return (W * W).sum(dim=1)


def _eager_weight_norm_cached(W0, A, B, base_sq, s):
    V = B.float() @ A.float()
    n2 = base_sq.float() + 2.0 * s * (W0.float() * V).sum(dim=1) + (s * s) * (V * V).sum(dim=1)
    return torch.sqrt(torch.clamp(n2, min=0.0))


def _eager_weight_norm_backward(W0, A, B, norm, d_norm, s):
    n, d = norm.float(), d_norm.float()
    c = torch.where(n != 0, d / torch.where(n != 0, n, torch.ones_like(n)), torch.zeros_like(n))
    dV = c[:, None] * (W0.float() + s * (B.float() @ A.float()))
    return (s * (B.float().t() @ dV)).to(A.dtype), (s * (dV @ A.float().t())).to(B.dtype)


def _scales(mag, norm):
    m, n = mag.float(), norm.float()
    return m / n, (m - n) / n  # g and g - 1 (the subtraction is exact near g = 1)


def _eager_compose(base, lora, mag, norm, s, add_base):
    g, gm1 = _scales(mag, norm)
    b = base.float()
    y = gm1 * b + g * s * lora.float()
    return (y + b if add_base else y).to(base.dtype)


def _eager_compose_backward(dy, base, lora, mag, norm, s, add_base, want_base):
    g, gm1 = _scales(mag, norm)
    d = dy.float()
    d_lora = (g * s * d).to(dy.dtype)
    d_base = ((g if add_base else gm1) * d).to(dy.dtype) if want_base else dy.new_empty((0,))
    d_mag = (d * (base.float() + s * lora.float())).sum(dim=0) / norm.float()
    return d_lora, d_base, d_mag


def _eager_lora_compose(base, h, B, mag, norm, s, add_base):
    return _eager_compose(base, h.float() @ B.float().t(), mag, norm, s, add_base)


def _eager_lora_compose_backward(dy, base, h, B, mag, norm, s, add_base, want_base):
    g, gm1 = _scales(mag, norm)
    d, hf, Bf = dy.float(), h.float(), B.float()
    E = d.t() @ hf  # dy^T h
    d_base = ((g if add_base else gm1) * d).to(dy.dtype) if want_base else dy.new_empty((0,))
    d_B = ((g * s)[:, None] * E).to(B.dtype)
    d_mag = ((d * base.float()).sum(dim=0) + s * (Bf * E).sum(dim=1)) / norm.float()
    return d_base, d_B, d_mag


# --------------------------------------------------------------------------- norm


@torch.library.custom_op("dora_amd::weight_norm", mutates_args=(), device_types="cuda")
def weight_norm(W0: Tensor, A: Tensor, B: Tensor, s: float) -> Tensor:
    """||W0_i + s * B_i A||_2 per output row i, fp32, via the factored kernels."""
    if not _kernels_take(W0, A, B):
        return _eager_weight_norm(W0, A, B, s)
    return binding.dora_norm_factored(W0.contiguous(), A.contiguous(), B.contiguous(), s)


@weight_norm.register_fake
def _weight_norm_fake(W0, A, B, s):
    return W0.new_empty((W0.shape[0],), dtype=torch.float32)


@torch.library.custom_op("dora_amd::row_sqnorm", mutates_args=(), device_types="cuda")
def row_sqnorm(W0: Tensor) -> Tensor:
    """||W0_i||^2 per output row, fp32."""
    if not _kernels_take(W0):
        return _eager_row_sqnorm(W0)
    return binding.dora_row_sqnorm(W0.contiguous())


@row_sqnorm.register_fake
def _row_sqnorm_fake(W0):
    return W0.new_empty((W0.shape[0],), dtype=torch.float32)


@torch.library.custom_op("dora_amd::weight_norm_cached", mutates_args=(), device_types="cuda")
def weight_norm_cached(W0: Tensor, A: Tensor, B: Tensor, base_sq: Tensor, s: float) -> Tensor:
    """The weight norm with the base term ||W0_i||^2 taken from base_sq."""
    if not _kernels_take(W0, A, B):
        return _eager_weight_norm_cached(W0, A, B, base_sq, s)
    return binding.dora_norm_factored_cached(W0.contiguous(), A.contiguous(), B.contiguous(),
                                             base_sq.contiguous().float(), s)


@weight_norm_cached.register_fake
def _weight_norm_cached_fake(W0, A, B, base_sq, s):
    return W0.new_empty((W0.shape[0],), dtype=torch.float32)


@torch.library.custom_op("dora_amd::weight_norm_backward", mutates_args=(), device_types="cuda")
def weight_norm_backward(W0: Tensor, A: Tensor, B: Tensor, norm: Tensor, d_norm: Tensor,
                         s: float) -> tuple[Tensor, Tensor]:
    """(d_A, d_B) of sum(d_norm * n) for n = ||W0 + s*B*A|| (norm: the forward's n)."""
    if not _kernels_take(W0, A, B):
        return _eager_weight_norm_backward(W0, A, B, norm, d_norm, s)
    return binding.dora_norm_bwd(W0.contiguous(), A.contiguous(), B.contiguous(), norm.contiguous().float(),
                                 d_norm.contiguous().float(), s)


@weight_norm_backward.register_fake
def _weight_norm_backward_fake(W0, A, B, norm, d_norm, s):
    return torch.empty_like(A), torch.empty_like(B)


def _norm_setup(ctx, inputs, output):
    W0, A, B = inputs[0], inputs[1], inputs[2]
    ctx.save_for_backward(W0, A, B, output)
    ctx.s = inputs[-1]
    ctx.n_inputs = len(inputs)


def _norm_grad(ctx, d_norm):
    W0, A, B, n = ctx.saved_tensors
    need_a, need_b = ctx.needs_input_grad[1], ctx.needs_input_grad[2]
    if ctx.needs_input_grad[0]:
        raise RuntimeError("dora_amd: W0 is frozen; the weight-norm backward gives gradients of A and B only")
    d_A = d_B = None
    if need_a or need_b:
        d_A, d_B = weight_norm_backward(W0, A, B, n, d_norm, ctx.s)
    return (None, d_A if need_a else None, d_B if need_b else None) + (None,) * (ctx.n_inputs - 3)


weight_norm.register_autograd(_norm_grad, setup_context=_norm_setup)
weight_norm_cached.register_autograd(_norm_grad, setup_context=_norm_setup)


# ------------------------------------------------------------------------ compose


@torch.library.custom_op("dora_amd::compose", mutates_args=(), device_types="cuda")
def compose(base: Tensor, lora: Tensor, mag: Tensor, norm: Tensor, s: float, add_base: bool) -> Tensor:
    """(g - 1) * base + g * s * lora, plus base when add_base, with g = mag / norm per column."""
    if not _kernels_take(base, lora):
        return _eager_compose(base, lora, mag, norm, s, add_base)
    return binding.dora_compose_fwd(base.contiguous(), lora.to(base.dtype).contiguous(), mag.contiguous().float(),
                                    norm.contiguous().float(), s, add_base=add_base)


@compose.register_fake
def _compose_fake(base, lora, mag, norm, s, add_base):
    return torch.empty_like(base)


@torch.library.custom_op("dora_amd::compose_backward", mutates_args=(), device_types="cuda")
def compose_backward(dy: Tensor, base: Tensor, lora: Tensor, mag: Tensor, norm: Tensor, s: float, add_base: bool,
                     want_base: bool) -> tuple[Tensor, Tensor, Tensor]:
    """(d_lora, d_base, d_mag) of the compose.  With want_base false the kernel
    does not write d_base and an empty tensor stands in for it."""
    if not _kernels_take(dy, base, lora):
        return _eager_compose_backward(dy, base, lora, mag, norm, s, add_base, want_base)
    d_lora, d_base, d_mag = binding.dora_compose_bwd(dy.contiguous(), base.contiguous(), lora.contiguous(),
                                                     mag.contiguous().float(), norm.contiguous().float(), s,
                                                     add_base=add_base, want_d_base=want_base)
    if d_base is None:
        d_base = dy.new_empty((0,))
    return d_lora, d_base, d_mag


@compose_backward.register_fake
def _compose_backward_fake(dy, base, lora, mag, norm, s, add_base, want_base):
    d_base = torch.empty_like(dy) if want_base else dy.new_empty((0,))
    return torch.empty_like(dy), d_base, mag.new_empty(mag.shape)


@torch.library.custom_op("dora_amd::lora_compose", mutates_args=(), device_types="cuda")
def lora_compose(base: Tensor, h: Tensor, B: Tensor, mag: Tensor, norm: Tensor, s: float, add_base: bool) -> Tensor:
    """(g - 1) * base + g * s * (h B^T), plus base when add_base; lora never stored."""
    if not _kernels_take(base, h, B):
        return _eager_lora_compose(base, h, B, mag, norm, s, add_base)
    return binding.dora_lora_compose_fwd(base.contiguous(), h.contiguous(), B.contiguous(), mag.contiguous().float(),
                                         norm.contiguous().float(), s, add_base=add_base)


@lora_compose.register_fake
def _lora_compose_fake(base, h, B, mag, norm, s, add_base):
    return torch.empty_like(base)


def _compose_setup(ctx, inputs, output):
    base, lora, mag, norm, s, add_base = inputs
    ctx.save_for_backward(base, lora, mag, norm)
    ctx.s = s
    ctx.add_base = add_base


def _compose_grad(ctx, dy):
    base, lora, mag, norm = ctx.saved_tensors
    want_base = bool(ctx.needs_input_grad[0])
    d_lora, d_base, d_mag = compose_backward(dy, base, lora, mag, norm, ctx.s, ctx.add_base, want_base)
    # a norm that is not detached: L depends on n only through g = m / n, so
    # dL/dn = -(m / n) * d_mag, with d_mag = sum_t dy (base + s lora) / n
    d_norm = -(mag / norm) * d_mag if ctx.needs_input_grad[3] else None
    return (d_base if want_base else None,
            d_lora if ctx.needs_input_grad[1] else None,
            d_mag if ctx.needs_input_grad[2] else None,
            d_norm, None, None)


compose.register_autograd(_compose_grad, setup_context=_compose_setup)


@torch.library.custom_op("dora_amd::lora_compose_backward", mutates_args=(), device_types="cuda")
def lora_compose_backward(dy: Tensor, base: Tensor, h: Tensor, B: Tensor, mag: Tensor, norm: Tensor, s: float,
                          add_base: bool, want_base: bool) -> tuple[Tensor, Tensor, Tensor]:
    """(d_base, d_B, d_mag) of ``lora_compose``, lora and d_lora never formed.
    With want_base false the kernel does not write d_base and an empty tensor
    stands in for it."""
    if not _kernels_take(dy, base, h, B):
        return _eager_lora_compose_backward(dy, base, h, B, mag, norm, s, add_base, want_base)
    try:
        d_base, d_B, d_mag = binding.dora_lora_compose_bwd(dy.contiguous(), base.contiguous(), h.contiguous(),
                                                           B.contiguous(), mag.contiguous().float(),
                                                           norm.contiguous().float(), s, add_base=add_base,
                                                           want_d_base=want_base)
    except binding.DoraError as e:
        if not _unsupported(e):  # a shape the library refuses (its slow path would be too slow): eager tier
            raise
        return _eager_lora_compose_backward(dy, base, h, B, mag, norm, s, add_base, want_base)
    if d_base is None:
        d_base = dy.new_empty((0,))
    return d_base, d_B, d_mag


@lora_compose_backward.register_fake
def _lora_compose_backward_fake(dy, base, h, B, mag, norm, s, add_base, want_base):
    d_base = torch.empty_like(dy) if want_base else dy.new_empty((0,))
    return d_base, torch.empty_like(B), mag.new_empty(mag.shape)


def _lora_compose_setup(ctx, inputs, output):
    base, h, B, mag, norm, s, add_base = inputs
    ctx.save_for_backward(base, h, B, mag, norm)
    ctx.s = s
    ctx.add_base = add_base


def _lora_compose_grad(ctx, dy):
    base, h, B, mag, norm = ctx.saved_tensors
    need = ctx.needs_input_grad
    d_base, d_B, d_mag = lora_compose_backward(dy, base, h, B, mag, norm, ctx.s, ctx.add_base, bool(need[0]))
    # the gradient of h through lora = h B^T: d_lora B = dy (g s .* B), the
    # caller's GEMM (a [T x out] by [out x r] product), with g s folded into B
    d_h = None
    if need[1]:
        gsB = ((mag / norm) * ctx.s)[:, None] * B.float()
        d_h = (dy @ gsB.to(dy.dtype))
    d_norm = -(mag / norm) * d_mag if need[4] else None
    return (d_base if need[0] else None, d_h, d_B if need[2] else None, d_mag if need[3] else None, d_norm,
            None, None)


lora_compose.register_autograd(_lora_compose_grad, setup_context=_lora_compose_setup)


# The eager tier is also each operator's kernel for CPU tensors.
weight_norm.register_kernel("cpu")(_eager_weight_norm)
row_sqnorm.register_kernel("cpu")(_eager_row_sqnorm)
weight_norm_cached.register_kernel("cpu")(_eager_weight_norm_cached)
weight_norm_backward.register_kernel("cpu")(_eager_weight_norm_backward)
compose.register_kernel("cpu")(_eager_compose)
compose_backward.register_kernel("cpu")(_eager_compose_backward)
lora_compose.register_kernel("cpu")(_eager_lora_compose)
lora_compose_backward.register_kernel("cpu")(_eager_lora_compose_backward)


# ------------------------------------------------------------ the frozen side in 8 bits
#
# Packed matrices are pairs (q, e): float8_e4m3fn values in blocks of 128 (of a
# row, or 128 x 128 of a weight) and uint8 exponent bytes 127 + e, laid out as
# include/dora.h says.  W0 is frozen and x and base are needed by the backward
# only inside sums over the tokens, so 8 bits hold them.

_F8 = torch.float8_e4m3fn


_AUTOCAST_KEYS = torch._C.DispatchKeySet(torch._C.DispatchKey.AutocastCUDA) | torch._C.DispatchKeySet(
    torch._C.DispatchKey.AutocastCPU)


def _without_autocast(fn):
    """fn with autocast off inside: its products keep the types they are given."""

    @functools.wraps(fn)
    def inner(*args):
        with torch._C._ExcludeDispatchKeyGuard(_AUTOCAST_KEYS):
            return fn(*args)

    return inner


def _q8_eager(fn):
    """The eager form of an operator: without autocast, and with outputs in the
    kernels' order of memory whatever its arguments' strides."""

    @functools.wraps(fn)
    def inner(*args):
        with torch._C._ExcludeDispatchKeyGuard(_AUTOCAST_KEYS):
            out = fn(*args)
        return tuple(t.contiguous() for t in out) if isinstance(out, tuple) else out.contiguous()

    return inner


def _autocast(*mats):
    """The matrices in autocast's type where it is on for their device, as linear
    takes them (64-bit and packed ones stay as they are)."""
    kind = mats[0].device.type
    if kind not in ("cuda", "cpu") or not torch.is_autocast_enabled(kind):
        return mats
    to, cast = torch.get_autocast_dtype(kind), (torch.float32, torch.float16, torch.bfloat16)
    return tuple(t.to(to) if t.dtype in cast else t for t in mats)


def _round_up(n: int, k: int) -> int:
    return -(-n // k) * k


def _exp2i(k: Tensor) -> Tensor:
    """2^k in fp32 for whole k in [-126, 127], by its exponent field (exact on every device)."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _eager_blocks(v: Tensor, dims) -> tuple[Tensor, Tensor]:
    """(values, exponent bytes) of fp32 blocks that lie along ``dims``."""
    amax = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(dim=dims, keepdim=True)
    bits = amax.view(torch.int32)  # 448 = 1.75 * 2^8
    e = ((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=-126)
    q = torch.where(torch.isfinite(v), v * _exp2i(-e), torch.full_like(v, math.nan))
    return q.to(_F8), (e + 127).to(torch.uint8)


def _padded_exponents(e: Tensor) -> Tensor:
    return F.pad(e, (0, _round_up(e.shape[1], 4) - e.shape[1]), value=127)


@_q8_eager
def _eager_q8_pack(x):
    T, K = x.shape
    if x.numel() == 0:
        (qs, es) = binding.q8_row_shapes(T, K)
        return x.new_empty(qs, dtype=_F8), x.new_empty(es, dtype=torch.uint8)
    v = F.pad(x.float(), (0, _round_up(K, 128) - K)).reshape(T, -1, 128)
    q, e = _eager_blocks(v, (2,))
    return q.reshape(T, -1), _padded_exponents(e[:, :, 0])


@_q8_eager
def _eager_q8_pack_weight(W):
    o, i = W.shape
    if W.numel() == 0:
        (qs, es) = binding.q8_weight_shapes(o, i)
        return W.new_empty(qs, dtype=_F8), W.new_empty(es, dtype=torch.uint8)
    v = F.pad(W.float(), (0, _round_up(i, 128) - i, 0, _round_up(o, 128) - o))
    q, e = _eager_blocks(v.reshape(v.shape[0] // 128, 128, -1, 128), (1, 3))
    return q.reshape(v.shape), _padded_exponents(e[:, 0, :, 0])


def _values(q, e, cols, name, shapes, weight=False):
    """The fp32 values of packed rows (or of a packed weight), which have to be
    laid out as the kernels ask for."""
    for t, what, shape, dtype in ((q, name, shapes[0], _F8), (e, name + "'s exponents", shapes[1], torch.uint8)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{what} is {tuple(t.shape)} in {t.dtype}, expected {shape} in {dtype}")
    nb = q.shape[1] // 128
    s = _exp2i(e[:, :nb].to(torch.int32) - 127)
    s = s.repeat_interleave(128, dim=1)
    if weight:
        s = s.repeat_interleave(128, dim=0)
    return (q.float() * s)[:, :cols]


def _held(v, dtype):
    big = torch.finfo(dtype).max
    return v.clamp(-big, big).to(dtype)


@_q8_eager
def _eager_q8_unpack(q, e, cols, dtype):
    return _held(_values(q, e, cols, "q", binding.q8_row_shapes(q.shape[0], cols)), dtype)


@_q8_eager
def _eager_q8_unpack_weight(q, e, rows, cols, dtype):
    if not 0 <= rows <= q.shape[0]:
        raise ValueError(f"rows {rows} out of range of a packed weight of {q.shape[0]}")
    return _held(_values(q, e, cols, "q", binding.q8_weight_shapes(q.shape[0], cols), True)[:rows], dtype)


@_q8_eager
def _eager_q8_linear(xq, xe, wq, we, out_features, dtype):
    T, n = xq.shape
    x = _values(xq, xe, n, "xq", binding.q8_row_shapes(T, n))
    W = _values(wq, we, n, "wq", binding.q8_weight_shapes(out_features, n), True)
    return (x @ W[:out_features].t()).to(dtype)


@_q8_eager
def _eager_q8_linear_backward(gq, ge, wq, we, in_features, dtype):
    T, n = gq.shape
    g = _values(gq, ge, n, "gq", binding.q8_row_shapes(T, n))
    return (g @ _values(wq, we, in_features, "wq", binding.q8_weight_shapes(n, in_features), True)).to(dtype)


@_q8_eager
def _eager_q8_lora_compose_backward(dy, bq, be, h, B, mag, norm, s, add_base, want_base):
    base = _values(bq, be, dy.shape[1], "bq", binding.q8_row_shapes(*dy.shape))
    return _eager_lora_compose_backward(dy, base, h, B, mag, norm, s, add_base, want_base)


@_q8_eager
def _eager_q8_lora_compose_backward_packed(dy, bq, be, h, B, mag, norm, s, add_base):
    _, d_B, d_mag = _eager_q8_lora_compose_backward(dy, bq, be, h, B, mag, norm, s, add_base, False)
    g, gm1 = _scales(mag, norm)
    q, e = _eager_q8_pack((g if add_base else gm1) * dy.float())
    return q, e, d_B, d_mag


@_q8_eager
def _eager_q8_grad_a(dh, xq, xe, in_features):
    x = _values(xq, xe, in_features, "xq", binding.q8_row_shapes(dh.shape[0], in_features))
    return (dh.float().t() @ _held(x, dh.dtype).float()).to(dh.dtype)


# These operators are registered without the wrapper of a custom operator: they
# run in serving loops, where its layers cost as much as a launch.  Those without
# an autograd formula of their own (the 8-bit ones, for which ``q8_layer`` has it)
# refuse arguments that require a gradient: none would come back through them.
# None takes arguments that carry a tangent.  Gradients and refusals are the
# operators' Autograd kernel, which tracing and functorch run as well as an eager
# call.
_Q8_LIB = torch.library.Library("dora_amd", "FRAGMENT")
_BELOW_AUTOGRAD = torch._C._after_autograd_keyset


def _refuse_tangents(name, args):
    for a in args:
        if isinstance(a, Tensor) and fwad.unpack_dual(a).tangent is not None:
            raise RuntimeError(f"{name} has no gradient of its own in forward mode: pass tensors without tangents")


def _q8_kernel(name, gradient=None):
    """Register a function as the GPU kernel of the operator ``name``, the eager
    form of the same name as its CPU kernel (and for a call the library refuses
    with DORA_UNSUPPORTED); the operator takes its place.  ``gradient``, where the
    operator has one, is an autograd function: it is given the call below autograd
    and the operator's arguments."""

    def register(fn):
        eager = globals()["_eager_" + name]

        def on_gpu(*args):
            try:
                return fn(*args)
            except binding.DoraError as e:
                if not _unsupported(e):
                    raise
                return eager(*args)

        kernels = {torch._C.DispatchKey.CUDA: on_gpu, torch._C.DispatchKey.CPU: eager}
        direct = {}  # by a key set's bits: the device's kernel where nothing else is left of it, else None

        def autograd(keyset, *args):
            if fwad._current_level >= 0:
                _refuse_tangents(name, args)
            if torch.is_grad_enabled():
                for a in args:
                    if isinstance(a, Tensor) and a.requires_grad:
                        if gradient is None:
                            hint = ", or use q8_layer" if name.startswith("q8_") else ""
                            raise RuntimeError(f"{name} has no gradient of its own: pass detached tensors{hint}")
                        return gradient.apply(functools.partial(below, keyset), *args)
            return below(keyset, *args)

        def below(keyset, *args):
            bits = keyset.raw_repr()
            if bits not in direct:
                direct[bits] = kernels.get((keyset & _BELOW_AUTOGRAD).highestPriorityTypeId())
            kernel = direct[bits]
            if kernel is not None:  # a second way through the dispatcher would cost 3 us
                return kernel(*args)
            with torch._C._AutoDispatchBelowAutograd():
                return op.redispatch(keyset & _BELOW_AUTOGRAD, *args)

        schema = torch.library.infer_schema(fn, mutates_args=())
        _Q8_LIB.define(name + schema)
        _Q8_LIB.impl(name, on_gpu, "CUDA")
        _Q8_LIB.impl(name, eager, "CPU")
        _Q8_LIB.impl(name, autograd, "Autograd", with_keyset=True)
        op = getattr(torch.ops.dora_amd, name).default
        op.__doc__ = fn.__doc__
        return op

    return register


@_q8_kernel("q8_pack")
def q8_pack(x: Tensor) -> tuple[Tensor, Tensor]:
    """(q, e): the rows of x [T x K] in 8-bit blocks of 128 columns."""
    if not _kernels_take(x):
        return _eager_q8_pack(x)
    return binding.dora_q8_pack(x.contiguous())


@torch.library.register_fake("dora_amd::q8_pack")
def _q8_pack_fake(x):
    qs, es = binding.q8_row_shapes(x.shape[0], x.shape[1])
    return x.new_empty(qs, dtype=_F8), x.new_empty(es, dtype=torch.uint8)


@_q8_kernel("q8_pack_weight")
def q8_pack_weight(W: Tensor) -> tuple[Tensor, Tensor]:
    """(q, e): a weight [out x in] in 8-bit blocks of 128 x 128 (once: it is frozen)."""
    if not _kernels_take(W):
        return _eager_q8_pack_weight(W)
    return binding.dora_q8_pack_weight(W.contiguous())


@torch.library.register_fake("dora_amd::q8_pack_weight")
def _q8_pack_weight_fake(W):
    qs, es = binding.q8_weight_shapes(W.shape[0], W.shape[1])
    return W.new_empty(qs, dtype=_F8), W.new_empty(es, dtype=torch.uint8)


@_q8_kernel("q8_unpack")
def q8_unpack(q: Tensor, e: Tensor, cols: int, dtype: torch.dtype) -> Tensor:
    """The values that packed rows are held as, [T x cols] in dtype."""
    if dtype not in binding.DTYPE_CODE:
        return _eager_q8_unpack(q, e, cols, dtype)
    return binding.dora_q8_unpack(q.contiguous(), e.contiguous(), q.shape[0], cols, dtype)


@torch.library.register_fake("dora_amd::q8_unpack")
def _q8_unpack_fake(q, e, cols, dtype):
    return q.new_empty((q.shape[0], cols), dtype=dtype)


@_q8_kernel("q8_unpack_weight")
def q8_unpack_weight(q: Tensor, e: Tensor, rows: int, cols: int, dtype: torch.dtype) -> Tensor:
    """The values of the first ``rows`` rows of a packed weight, [rows x cols] in dtype."""
    if dtype not in binding.DTYPE_CODE:
        return _eager_q8_unpack_weight(q, e, rows, cols, dtype)
    return binding.dora_q8_unpack(q.contiguous(), e.contiguous(), rows, cols, dtype, weight=True)


@torch.library.register_fake("dora_amd::q8_unpack_weight")
def _q8_unpack_weight_fake(q, e, rows, cols, dtype):
    return q.new_empty((rows, cols), dtype=dtype)


@_q8_kernel("q8_linear")
def q8_linear(xq: Tensor, xe: Tensor, wq: Tensor, we: Tensor, out_features: int, dtype: torch.dtype) -> Tensor:
    """y [T x out] = x W^T from packed rows and a packed weight."""
    if dtype not in binding.DTYPE_CODE:
        return _eager_q8_linear(xq, xe, wq, we, out_features, dtype)
    return binding.dora_q8_linear_fwd(xq.contiguous(), xe.contiguous(), wq.contiguous(), we.contiguous(),
                                      out_features, xq.shape[1], dtype)


@torch.library.register_fake("dora_amd::q8_linear")
def _q8_linear_fake(xq, xe, wq, we, out_features, dtype):
    return xq.new_empty((xq.shape[0], out_features), dtype=dtype)


@_q8_kernel("q8_linear_backward")
def q8_linear_backward(gq: Tensor, ge: Tensor, wq: Tensor, we: Tensor, in_features: int,
                       dtype: torch.dtype) -> Tensor:
    """dx [T x in] = g W from packed rows g [T x out] and the same packed weight."""
    if dtype not in binding.DTYPE_CODE:
        return _eager_q8_linear_backward(gq, ge, wq, we, in_features, dtype)
    return binding.dora_q8_linear_bwd(gq.contiguous(), ge.contiguous(), wq.contiguous(), we.contiguous(),
                                      gq.shape[1], in_features, dtype)


@torch.library.register_fake("dora_amd::q8_linear_backward")
def _q8_linear_backward_fake(gq, ge, wq, we, in_features, dtype):
    return gq.new_empty((gq.shape[0], in_features), dtype=dtype)


def _q8_compose_args(dy, bq, be, h, B, mag, norm, s):
    return (dy.contiguous(), bq.contiguous(), be.contiguous(), h.contiguous(), B.contiguous(),
            mag.contiguous().float(), norm.contiguous().float(), s)


@_q8_kernel("q8_lora_compose_backward")
def q8_lora_compose_backward(dy: Tensor, bq: Tensor, be: Tensor, h: Tensor, B: Tensor, mag: Tensor, norm: Tensor,
                             s: float, add_base: bool, want_base: bool) -> tuple[Tensor, Tensor, Tensor]:
    """``lora_compose_backward`` with the base from packed rows."""
    if not _kernels_take(dy, h, B):
        return _eager_q8_lora_compose_backward(dy, bq, be, h, B, mag, norm, s, add_base, want_base)
    d_base, d_B, d_mag = binding.dora_q8_lora_compose_bwd(*_q8_compose_args(dy, bq, be, h, B, mag, norm, s), add_base,
                                                          want_d_base=want_base)
    return dy.new_empty((0,)) if d_base is None else d_base, d_B, d_mag


@torch.library.register_fake("dora_amd::q8_lora_compose_backward")
def _q8_lora_compose_backward_fake(dy, bq, be, h, B, mag, norm, s, add_base, want_base):
    d_base = dy.new_empty(dy.shape if want_base else (0,))
    return d_base, B.new_empty(B.shape), mag.new_empty(mag.shape, dtype=torch.float32)


@_q8_kernel("q8_lora_compose_backward_packed")
def q8_lora_compose_backward_packed(dy: Tensor, bq: Tensor, be: Tensor, h: Tensor, B: Tensor, mag: Tensor,
                                    norm: Tensor, s: float, add_base: bool) -> tuple[Tensor, Tensor, Tensor, Tensor]:
    """The same with d_base packed straight from fp32: (q, e, d_B, d_mag)."""
    if not _kernels_take(dy, h, B):
        return _eager_q8_lora_compose_backward_packed(dy, bq, be, h, B, mag, norm, s, add_base)
    (q, e), d_B, d_mag = binding.dora_q8_lora_compose_bwd(*_q8_compose_args(dy, bq, be, h, B, mag, norm, s), add_base,
                                                          packed=True)
    return q, e, d_B, d_mag


@torch.library.register_fake("dora_amd::q8_lora_compose_backward_packed")
def _q8_lora_compose_backward_packed_fake(dy, bq, be, h, B, mag, norm, s, add_base):
    q, e = _q8_pack_fake(dy)
    return q, e, B.new_empty(B.shape), mag.new_empty(mag.shape, dtype=torch.float32)


@_q8_kernel("q8_grad_a")
def q8_grad_a(dh: Tensor, xq: Tensor, xe: Tensor, in_features: int) -> Tensor:
    """d_A [r x in] = d_h^T x from packed rows x."""
    if not _kernels_take(dh):
        return _eager_q8_grad_a(dh, xq, xe, in_features)
    return binding.dora_q8_grad_a(dh.contiguous(), xq.contiguous(), xe.contiguous(), in_features)


@torch.library.register_fake("dora_amd::q8_grad_a")
def _q8_grad_a_fake(dh, xq, xe, in_features):
    return dh.new_empty((dh.shape[1], in_features))


# The norm of a packed weight: 16-bit values of a slab of rows at a time (32 MiB
# at 8192 columns), so the weight is never whole in 16 bits.
_Q8_SLAB = 2048


def _slabs(wq, we, out, in_, dtype):
    for i in range(0, out, _Q8_SLAB):
        n = min(_Q8_SLAB, out - i)
        rows = slice(i, _round_up(i + n, 128))
        blocks = slice(i // 128, -(-(i + n) // 128))
        yield slice(i, i + n), q8_unpack_weight(wq[rows], we[blocks], n, in_, dtype)


def _norm_of_slabs(slabs, A, B, base_sq, s):
    """``weight_norm_cached`` of a weight that comes in slabs of rows."""
    n = torch.empty(B.shape[0], dtype=torch.float32, device=B.device)
    for rows, W in slabs:
        n[rows] = weight_norm_cached(W, A, B[rows], base_sq[rows], s)
    return n


def _norm_backward_of_slabs(slabs, A, B, norm, d_norm, s):
    """``weight_norm_backward`` of a weight that comes in slabs of rows: (d_A, d_B),
    the slabs' parts of d_A added in fp32 and rounded once."""
    A, B, norm, d_norm = A.contiguous(), B.contiguous(), norm.contiguous().float(), d_norm.contiguous().float()
    d_A, d_B = torch.zeros(A.shape, dtype=torch.float32, device=A.device), torch.empty_like(B)
    for rows, W in slabs:
        if _kernels_take(W, A, B):
            d_B[rows] = binding.dora_norm_bwd_slab(W, A, B[rows], norm[rows], d_norm[rows], s, d_A, rows.start > 0)
        else:
            a, b = _eager_weight_norm_backward(W, A.float(), B[rows].float(), norm[rows], d_norm[rows], s)
            d_A += a
            d_B[rows] = b.to(B.dtype)
    return d_A.to(A.dtype), d_B


@torch.library.custom_op("dora_amd::q8_weight_norm", mutates_args=())
@_without_autocast
def q8_weight_norm(wq: Tensor, we: Tensor, A: Tensor, B: Tensor, base_sq: Tensor, s: float) -> Tensor:
    """``weight_norm_cached`` of a packed weight."""
    return _norm_of_slabs(_slabs(wq, we, B.shape[0], A.shape[1], A.dtype), A, B, base_sq, s)


@q8_weight_norm.register_fake
def _q8_weight_norm_fake(wq, we, A, B, base_sq, s):
    return B.new_empty((B.shape[0],), dtype=torch.float32)


@torch.library.custom_op("dora_amd::q8_weight_norm_backward", mutates_args=())
@_without_autocast
def q8_weight_norm_backward(wq: Tensor, we: Tensor, A: Tensor, B: Tensor, norm: Tensor, d_norm: Tensor,
                            s: float) -> tuple[Tensor, Tensor]:
    """``weight_norm_backward`` of a packed weight."""
    return _norm_backward_of_slabs(_slabs(wq, we, B.shape[0], A.shape[1], A.dtype), A, B, norm, d_norm, s)


@q8_weight_norm_backward.register_fake
def _q8_weight_norm_backward_fake(wq, we, A, B, norm, d_norm, s):
    return A.new_empty(A.shape), B.new_empty(B.shape)


def _q8_norm_setup(ctx, inputs, output):
    wq, we, A, B, _, s = inputs
    ctx.save_for_backward(wq, we, A, B, output)
    ctx.s = s


def _q8_norm_grad(ctx, d_norm):
    wq, we, A, B, n = ctx.saved_tensors
    d_A, d_B = q8_weight_norm_backward(wq, we, A, B, n, d_norm, ctx.s)
    need = ctx.needs_input_grad
    return None, None, d_A if need[2] else None, d_B if need[3] else None, None, None


q8_weight_norm.register_autograd(_q8_norm_grad, setup_context=_q8_norm_setup)


@torch.library.custom_op("dora_amd::q8_layer", mutates_args=())
def q8_layer(x: Tensor, A: Tensor, B: Tensor, mag: Tensor, norm: Tensor, weight: Tensor, we: Optional[Tensor],
             s: float) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    """The layer on x [T x in] with 8-bit checkpoints: (y, then what the backward
    reads, itself without a gradient: x and base packed, and h).  ``weight`` is W0 [out x in] in 16 bits, or,
    with its exponents ``we``, packed in 8 bits: then both products with W0 run on packed
    operands, x's being the checkpoint itself; or packed in 4 bits (uint8).  Its matrices have one type (under
    autocast they are cast to its); its backward has no backward."""
    xq, xe = q8_pack(x)
    if we is None:
        base = F.linear(x, weight)
    elif weight.dtype == torch.uint8:
        base = q4_linear(x, weight, we, B.shape[0])
    else:
        base = q8_linear(xq, xe, weight, we, B.shape[0], x.dtype)
    h = F.linear(x, A)
    y = lora_compose(base, h, B, mag, norm, s, True)
    bq, be = q8_pack(base)
    return y, xq, xe, bq, be, h


@q8_layer.register_fake
def _q8_layer_fake(x, A, B, mag, norm, weight, we, s):
    y = x.new_empty((x.shape[0], B.shape[0]))
    return (y, *_q8_pack_fake(x), *_q8_pack_fake(y), x.new_empty((x.shape[0], A.shape[0])))


def _q8_layer_setup(ctx, inputs, output):
    x, A, B, mag, norm, weight, we, s = inputs
    ctx.mark_non_differentiable(*output[1:])
    ctx.set_materialize_grads(False)  # no zeros for the checkpoints
    ctx.save_for_backward(A, B, mag, norm, weight, we, *output[1:])
    ctx.s = s


def _q8_layer_grad(ctx, dy, *_):
    A, B, mag, norm, weight, we, xq, xe, bq, be, h = ctx.saved_tensors
    need, s, in_ = ctx.needs_input_grad, ctx.s, A.shape[1]
    if dy is None:  # a later function gave no gradient: zeros, as autograd hands them to the 16-bit layer
        dy = h.new_zeros((h.shape[0], B.shape[0]))
    dx = None
    if need[0] and we is not None and weight.dtype != torch.uint8:
        dq, de, d_B, d_mag = q8_lora_compose_backward_packed(dy, bq, be, h, B, mag, norm, s, True)
        dx = q8_linear_backward(dq, de, weight, we, in_, dy.dtype)
    else:
        d_base, d_B, d_mag = q8_lora_compose_backward(dy, bq, be, h, B, mag, norm, s, True, bool(need[0]))
        if need[0]:
            dx = d_base @ weight if we is None else q4_linear_backward(d_base, weight, we, in_)
    d_A = None
    if need[0] or need[1]:
        gsB = ((mag / norm) * s)[:, None] * B.float()
        d_h = dy @ gsB.to(dy.dtype)
        if need[0]:
            dx = torch.addmm(dx, d_h, A)
        if need[1]:
            d_A = q8_grad_a(d_h, xq, xe, in_)
    d_norm = -(mag / norm) * d_mag if need[4] else None
    return dx, d_A, d_B if need[2] else None, d_mag if need[3] else None, d_norm, None, None, None


q8_layer.register_autograd(_q8_layer_grad, setup_context=_q8_layer_setup)


def _q8_layer_autocast(x, A, B, mag, norm, weight, we, s):
    x, A, B, weight = _autocast(x, A, B, weight)
    return _without_autocast(q8_layer)(x, A, B, mag, norm, weight, we, s)


for _key in ("AutocastCUDA", "AutocastCPU"):
    _Q8_LIB.impl("q8_layer", _q8_layer_autocast, _key)


# ------------------------------------------------------------ the frozen weight in 4 bits
#
# A packed weight is a pair (q, e) of uint8 tensors, tiles of 32 rows x 64 columns
# laid out as include/dora.h says.  The rows it is multiplied with stay in 16 bits.


def _q4_where(device) -> tuple[Tensor, Tensor]:
    """Byte positions within a tile of each row's two blocks (16 bytes each) and of their exponents."""
    r, b = torch.arange(32, device=device)[:, None], torch.arange(2, device=device)[None, :]
    g, i = r // 8, r % 8
    at = 128 * i + 32 * g + 16 * (b ^ (i // 2 % 2))
    exponents = 32 * b + 8 * g + 2 * (i % 4) + i // 4
    return (at[:, :, None] + torch.arange(16, device=device)).flatten(), exponents.flatten()


def _q4_values(q, e, rows, cols) -> Tensor:
    """The fp32 values of the first rows of a packed weight, which has to be laid out as the kernels ask for."""
    shapes = binding.q4_weight_shapes(q.shape[0] * binding.Q4_ROWS, cols)
    for t, what, shape in ((q, "the packed weight", shapes[0]), (e, "the packed weight's exponents", shapes[1])):
        if tuple(t.shape) != shape or t.dtype != torch.uint8:
            raise ValueError(f"{what} is {tuple(t.shape)} in {t.dtype}, expected {shape} in {torch.uint8}")
    if not 0 <= rows <= q.shape[0] * binding.Q4_ROWS:
        raise ValueError(f"rows {rows} out of range of a packed weight of {q.shape[0] * binding.Q4_ROWS}")
    at, ea = _q4_where(q.device)
    a, b = q.shape[:2]
    byte = q[:, :, at].reshape(a, b, 32, 2, 16)
    eb = e[:, :, ea].reshape(a, b, 32, 2).to(torch.int32)
    c = torch.stack((byte & 15, byte >> 4), dim=5).reshape(a, b, 32, 2, 32).to(torch.int32)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    scale = torch.where(eb == 255, torch.full((), math.nan, device=q.device), _exp2i((eb - 127).clamp(-126, 127)))
    v = torch.cat((grid, -grid))[c] * scale[..., None]
    return v.transpose(1, 2).reshape(a * 32, b * 64)[:rows, :cols]


def _q4_rows(q, out):
    """Refuse a packed weight of another number of row tiles."""
    if q.dim() != 3 or q.shape[0] != -(-out // binding.Q4_ROWS):
        raise ValueError(f"the packed weight is {tuple(q.shape)}, not one of {out} rows")


@_q8_eager
def _eager_q4_pack_weight(W):
    o, i = W.shape
    qs, es = binding.q4_weight_shapes(o, i)
    q, e = W.new_empty(qs, dtype=torch.uint8), W.new_empty(es, dtype=torch.uint8)
    if W.numel() == 0:
        return q, e
    v = F.pad(W.float(), (0, qs[1] * 64 - i, 0, qs[0] * 32 - o)).reshape(qs[0], 32, qs[1], 2, 32)
    amax = v.abs().amax(dim=4)
    bad = ~torch.isfinite(v).all(dim=4)
    bits = torch.where(bad, torch.zeros_like(amax), amax).view(torch.int32)  # 7 = 1.75 * 2^2
    k = ((bits >> 23) - 127 - 2 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(-23, 13)
    s = v * _exp2i(-k)[..., None]
    a = s.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for border, even_above in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (a >= border) if even_above else (a > border)
    code = torch.where(bad[..., None], torch.zeros_like(code), code | (torch.signbit(s).to(torch.uint8) << 3))
    at, ea = _q4_where(W.device)
    q[:, :, at] = (code[..., 0::2] | (code[..., 1::2] << 4)).transpose(1, 2).reshape(qs[0], qs[1], 1024)
    e[:, :, ea] = torch.where(bad, torch.full_like(k, 255), k + 127).to(torch.uint8).transpose(1, 2).reshape(es)
    return q, e


@_q8_eager
def _eager_q4_unpack_weight(q, e, rows, cols, dtype):
    return _q4_values(q, e, rows, cols).to(dtype)


@_q8_eager
def _eager_q4_linear(x, q, e, out_features):
    _q4_rows(q, out_features)
    return (x.float() @ _q4_values(q, e, out_features, x.shape[1]).t()).to(x.dtype)


@_q8_eager
def _eager_q4_linear_backward(g, q, e, in_features):
    _q4_rows(q, g.shape[1])
    return (g.float() @ _q4_values(q, e, g.shape[1], in_features)).to(g.dtype)


class _Q4Linear(torch.autograd.Function):
    """y = x W^T: W is frozen, and the gradient of x is the other product."""

    @staticmethod
    def forward(ctx, below, x, q, e, out_features):
        ctx.save_for_backward(q, e)
        ctx.in_features = x.shape[1]
        return below(x, q, e, out_features)

    @staticmethod
    def backward(ctx, dy):
        return None, q4_linear_backward(dy, *ctx.saved_tensors, ctx.in_features), None, None, None


class _Q4LinearBackward(torch.autograd.Function):
    """dx = g W, whose gradient of g is the first product again."""

    @staticmethod
    def forward(ctx, below, g, q, e, in_features):
        ctx.save_for_backward(q, e)
        ctx.out_features = g.shape[1]
        return below(g, q, e, in_features)

    @staticmethod
    def backward(ctx, d):
        return None, q4_linear(d, *ctx.saved_tensors, ctx.out_features), None, None, None


@_q8_kernel("q4_pack_weight")
def q4_pack_weight(W: Tensor) -> tuple[Tensor, Tensor]:
    """(q, e): a weight [out x in] in 4-bit blocks of 32 columns of a row (once: it is frozen)."""
    if not _kernels_take(W):
        return _eager_q4_pack_weight(W)
    return binding.dora_q4_pack_weight(W.contiguous())


@torch.library.register_fake("dora_amd::q4_pack_weight")
def _q4_pack_weight_fake(W):
    qs, es = binding.q4_weight_shapes(W.shape[0], W.shape[1])
    return W.new_empty(qs, dtype=torch.uint8), W.new_empty(es, dtype=torch.uint8)


@_q8_kernel("q4_unpack_weight")
def q4_unpack_weight(q: Tensor, e: Tensor, rows: int, cols: int, dtype: torch.dtype) -> Tensor:
    """The values of the first ``rows`` rows of a packed weight, [rows x cols] in dtype (exact in 16 bits)."""
    if dtype not in binding.DTYPE_CODE:
        return _eager_q4_unpack_weight(q, e, rows, cols, dtype)
    return binding.dora_q4_unpack_weight(q.contiguous(), e.contiguous(), rows, cols, dtype)


@torch.library.register_fake("dora_amd::q4_unpack_weight")
def _q4_unpack_weight_fake(q, e, rows, cols, dtype):
    return q.new_empty((rows, cols), dtype=dtype)


@_q8_kernel("q4_linear", gradient=_Q4Linear)
def q4_linear(x: Tensor, q: Tensor, e: Tensor, out_features: int) -> Tensor:
    """y [T x out] = x W^T from rows x [T x in] and a packed weight; differentiable in x."""
    if not _kernels_take(x):
        return _eager_q4_linear(x, q, e, out_features)
    return binding.dora_q4_linear_fwd(x.contiguous(), q.contiguous(), e.contiguous(), out_features)


@torch.library.register_fake("dora_amd::q4_linear")
def _q4_linear_fake(x, q, e, out_features):
    return x.new_empty((x.shape[0], out_features))


@_q8_kernel("q4_linear_backward", gradient=_Q4LinearBackward)
def q4_linear_backward(g: Tensor, q: Tensor, e: Tensor, in_features: int) -> Tensor:
    """dx [T x in] = g W from g [T x out] and the same packed weight; differentiable in g."""
    if not _kernels_take(g):
        return _eager_q4_linear_backward(g, q, e, in_features)
    return binding.dora_q4_linear_bwd(g.contiguous(), q.contiguous(), e.contiguous(), in_features)


@torch.library.register_fake("dora_amd::q4_linear_backward")
def _q4_linear_backward_fake(g, q, e, in_features):
    return g.new_empty((g.shape[0], in_features))


def _q4_linear_autocast(x, q, e, out_features):
    return _without_autocast(q4_linear)(*_autocast(x), q, e, out_features)


for _key in ("AutocastCUDA", "AutocastCPU"):
    _Q8_LIB.impl("q4_linear", _q4_linear_autocast, _key)


def _q4_slabs(q, e, out, in_, dtype):
    """As ``_slabs``, of a weight in 4 bits."""
    for i in range(0, out, _Q8_SLAB):
        n = min(_Q8_SLAB, out - i)
        tiles = slice(i // binding.Q4_ROWS, -(-(i + n) // binding.Q4_ROWS))
        yield slice(i, i + n), q4_unpack_weight(q[tiles], e[tiles], n, in_, dtype)


@torch.library.custom_op("dora_amd::q4_weight_norm", mutates_args=())
@_without_autocast
def q4_weight_norm(q: Tensor, e: Tensor, A: Tensor, B: Tensor, base_sq: Tensor, s: float) -> Tensor:
    """``weight_norm_cached`` of a weight packed in 4 bits (by slabs of unpacked rows
    where the kernel does not take the sizes, or A and B in fp32, under autocast too)."""
    if _kernels_take(A, B):
        try:
            return binding.dora_q4_norm_cached(q.contiguous(), e.contiguous(), A.contiguous(), B.contiguous(),
                                               base_sq.contiguous().float(), s)
        except binding.DoraError as err:
            if not _unsupported(err):
                raise
    return _norm_of_slabs(_q4_slabs(q, e, B.shape[0], A.shape[1], A.dtype), A, B, base_sq, s)


@q4_weight_norm.register_fake
def _q4_weight_norm_fake(q, e, A, B, base_sq, s):
    return B.new_empty((B.shape[0],), dtype=torch.float32)


@torch.library.custom_op("dora_amd::q4_weight_norm_backward", mutates_args=())
@_without_autocast
def q4_weight_norm_backward(q: Tensor, e: Tensor, A: Tensor, B: Tensor, norm: Tensor, d_norm: Tensor,
                            s: float) -> tuple[Tensor, Tensor]:
    """``weight_norm_backward`` of a weight packed in 4 bits."""
    return _norm_backward_of_slabs(_q4_slabs(q, e, B.shape[0], A.shape[1], A.dtype), A, B, norm, d_norm, s)


@q4_weight_norm_backward.register_fake
def _q4_weight_norm_backward_fake(q, e, A, B, norm, d_norm, s):
    return A.new_empty(A.shape), B.new_empty(B.shape)


def _q4_norm_grad(ctx, d_norm):
    q, e, A, B, n = ctx.saved_tensors
    d_A, d_B = q4_weight_norm_backward(q, e, A, B, n, d_norm, ctx.s)
    need = ctx.needs_input_grad
    return None, None, d_A if need[2] else None, d_B if need[3] else None, None, None


q4_weight_norm.register_autograd(_q4_norm_grad, setup_context=_q8_norm_setup)


# ------------------------------------------------------------ tokens sorted by adapter
#
# Several adapters over one frozen weight: token t of a batch has k slots, each with
# the number of an adapter or none.  adapter_sort gives every slot a row, adapter by
# adapter (place, int32 [T x k]; the complement of the row for a slot without one);
# adapter_gather and adapter_combine go to the rows and back.


def _whole_ids(ids, adapters):
    if adapters < 0 or ids.dim() != 2 or ids.is_floating_point() or ids.is_complex():
        raise ValueError(f"{adapters} adapters, ids {tuple(ids.shape)} in {ids.dtype}: expected whole numbers [T x k]")
    return ids if ids.dtype in (torch.int64, torch.int32) else ids.to(torch.int64)


@_q8_eager
def _eager_adapter_sort(ids, adapters):
    ids = _whole_ids(ids, adapters)
    flat = ids.flatten().to(torch.int64)
    has = (flat >= 0) & (flat < adapters)
    key = torch.where(has, flat, torch.full_like(flat, adapters))
    slots = torch.sort(key, stable=True).indices
    row = torch.arange(flat.numel(), device=flat.device)
    there = has[slots]
    order = torch.where(there, slots, -1 - slots)
    place = torch.empty_like(row)
    place[slots] = torch.where(there, row, -1 - row)
    count = torch.zeros(adapters + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))
    bounds = torch.cumsum(count, 0) - count
    return order.to(torch.int32), place.to(torch.int32).reshape(ids.shape), bounds.to(torch.int32)


def _rows_of(place, R):
    """(row of each slot, R where it is out of range; whether it is a row of an adapter) as flat int64 and bool."""
    p = place.flatten().to(torch.int64)
    row = torch.where(p < 0, -1 - p, p)
    return torch.where(row < R, row, torch.full_like(row, R)), (p >= 0) & (row < R)


def _check_place(place, T, what):
    if place.dim() != 2 or place.dtype != torch.int32 or place.shape[0] != T:
        raise ValueError(f"place is {tuple(place.shape)} in {place.dtype}, expected int32 [{T} x k], as for {what}")


@_q8_eager
def _eager_adapter_gather(x, place):
    _check_place(place, x.shape[0], "x")
    R, k = place.numel(), place.shape[1]
    row, has = _rows_of(place, R)
    rows = x.new_zeros((R + 1, x.shape[1]))
    v = x.repeat_interleave(k, dim=0)
    rows[row] = torch.where(has[:, None], v, torch.zeros_like(v))
    return rows[:R]


def _slot_rows(rows, place):
    """[T, k, D] in fp32: the rows of the slots, zeros for those without an adapter."""
    row, has = _rows_of(place, rows.shape[0])
    padded = F.pad(rows, (0, 0, 0, 1)).float()[row]
    return torch.where(has[:, None], padded, torch.zeros_like(padded)).reshape(*place.shape, rows.shape[1])


def _check_rows(rows, weights, place, base=None):
    if rows is not None and (rows.dim() != 2 or rows.shape[0] != place.numel()):
        raise ValueError(f"rows are {tuple(rows.shape)}, expected one for each of {place.numel()} slots")
    if weights is not None and weights.shape != place.shape:
        raise ValueError(f"weights are {tuple(weights.shape)}, expected {tuple(place.shape)}")
    if base is not None and (tuple(base.shape) != (place.shape[0], rows.shape[1]) or base.dtype != rows.dtype):
        raise ValueError(f"base is {tuple(base.shape)} in {base.dtype}, expected {(place.shape[0], rows.shape[1])} "
                         f"in {rows.dtype}")


@_q8_eager
def _eager_adapter_combine(rows, weights, place, base):
    _check_place(place, place.shape[0], "rows")
    _check_rows(rows, weights, place, base)
    v = _slot_rows(rows, place)
    if weights is not None:
        _, has = _rows_of(place, rows.shape[0])
        w = torch.where(has.reshape(place.shape), weights.float(), torch.zeros_like(weights, dtype=torch.float32))
        v = v * w[:, :, None]
    y = v.sum(dim=1)
    return (y if base is None else y + base.float()).to(rows.dtype)


@_q8_eager
def _eager_adapter_combine_backward(dy, rows, weights, place, want_rows, want_weights):
    _check_place(place, dy.shape[0], "dy")
    if rows is None and want_weights:
        raise ValueError("the gradient of the weights needs the rows")
    _check_rows(rows, weights, place)
    R, (T, k) = place.numel(), place.shape
    d = dy.float()
    d_rows, d_w = dy.new_empty((0,)), dy.new_empty((0,), dtype=torch.float32)
    if want_rows:
        row, has = _rows_of(place, R)
        v = d[:, None, :].expand(T, k, d.shape[1])
        if weights is not None:
            v = v * weights.float()[:, :, None]
        v = v.reshape(R, d.shape[1])
        d_rows = dy.new_zeros((R + 1, d.shape[1]))
        d_rows[row] = torch.where(has[:, None], v, torch.zeros_like(v)).to(dy.dtype)
        d_rows = d_rows[:R]
    if want_weights:
        _, has = _rows_of(place, R)
        d_w = (d[:, None, :] * _slot_rows(rows, place)).sum(dim=2)
        d_w = torch.where(has.reshape(place.shape), d_w, torch.zeros_like(d_w))
    return d_rows, d_w


class _AdapterGather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, below, x, place):
        ctx.save_for_backward(place)
        return below(x, place)

    @staticmethod
    def backward(ctx, d_rows):
        return None, adapter_combine(d_rows, None, ctx.saved_tensors[0], None), None


class _AdapterCombineGrads(torch.autograd.Function):
    """``adapter_combine_backward`` as it stands in a graph of gradients (create_graph): its own
    gradient is refused where it is asked for, as the compose's backward's is."""

    @staticmethod
    def forward(ctx, *args):
        return adapter_combine_backward(*args)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("adapter_combine_backward has no gradient of its own")


class _AdapterCombine(torch.autograd.Function):
    """The rows, T k x D, are kept only where the gradient of the weights reads them."""

    @staticmethod
    def forward(ctx, below, rows, weights, place, base):
        ctx.save_for_backward(rows if ctx.needs_input_grad[2] else None, weights, place)
        return below(rows, weights, place, base)

    @staticmethod
    def backward(ctx, dy):
        rows, weights, place = ctx.saved_tensors
        need = ctx.needs_input_grad
        d_rows = d_w = None
        if need[1] or need[2]:
            d_rows, d_w = _AdapterCombineGrads.apply(dy, rows, weights, place, need[1], need[2])
        return (None, d_rows if need[1] else None, d_w.to(weights.dtype) if need[2] else None, None,
                dy if need[4] else None)


@_q8_kernel("adapter_sort")
def adapter_sort(ids: Tensor, adapters: int) -> tuple[Tensor, Tensor, Tensor]:
    """(order [T k], place [T x k], bounds [adapters + 1]), int32: the slots of ids
    [T x k] sorted by adapter, stably, those of any number outside [0, adapters)
    behind them all.  order holds the slot t * k + j of each row, place the row of
    each slot, both as complements for slots without an adapter; adapter a has rows
    bounds[a] to bounds[a + 1]."""
    return binding.dora_adapter_sort(_whole_ids(ids, adapters).contiguous(), adapters)


@torch.library.register_fake("dora_amd::adapter_sort")
def _adapter_sort_fake(ids, adapters):
    T, k = ids.shape
    return (ids.new_empty((T * k,), dtype=torch.int32), ids.new_empty((T, k), dtype=torch.int32),
            ids.new_empty((adapters + 1,), dtype=torch.int32))


@_q8_kernel("adapter_gather", gradient=_AdapterGather)
def adapter_gather(x: Tensor, place: Tensor) -> Tensor:
    """rows [T k x D] of x [T x D]: x[t] at the row of each of token t's slots, zeros at
    those of slots without an adapter; differentiable in x."""
    if not _kernels_take(x):
        return _eager_adapter_gather(x, place)
    return binding.dora_adapter_gather(x.contiguous(), place.contiguous())


@torch.library.register_fake("dora_amd::adapter_gather")
def _adapter_gather_fake(x, place):
    return x.new_empty((place.shape[0] * place.shape[1], x.shape[1]))


@_q8_kernel("adapter_combine", gradient=_AdapterCombine)
def adapter_combine(rows: Tensor, weights: Optional[Tensor], place: Tensor, base: Optional[Tensor]) -> Tensor:
    """y [T x D]: base (or zeros) plus each token's rows times weights [T x k] (or ones),
    summed in fp32; slots without an adapter add nothing.  Differentiable in rows,
    weights and base."""
    if not _kernels_take(rows):
        return _eager_adapter_combine(rows, weights, place, base)
    return binding.dora_adapter_combine(rows.contiguous(), None if weights is None else weights.contiguous().float(),
                                        place.contiguous(), None if base is None else base.contiguous())


@torch.library.register_fake("dora_amd::adapter_combine")
def _adapter_combine_fake(rows, weights, place, base):
    return rows.new_empty((place.shape[0], rows.shape[1]))


@_q8_kernel("adapter_combine_backward")
def adapter_combine_backward(dy: Tensor, rows: Optional[Tensor], weights: Optional[Tensor], place: Tensor,
                             want_rows: bool, want_weights: bool) -> tuple[Tensor, Tensor]:
    """(d_rows, d_weights in fp32) of ``adapter_combine``; an empty tensor stands in
    for one that is not wanted.  rows are read for d_weights alone and may be None without."""
    if not _kernels_take(dy) or not (rows is None or _kernels_take(rows)):
        return _eager_adapter_combine_backward(dy, rows, weights, place, want_rows, want_weights)
    d_rows, d_w = binding.dora_adapter_combine_bwd(
        dy.contiguous(), None if rows is None else rows.contiguous(),
        None if weights is None else weights.contiguous().float(), place.contiguous(), want_rows, want_weights)
    return (dy.new_empty((0,)) if d_rows is None else d_rows,
            dy.new_empty((0,), dtype=torch.float32) if d_w is None else d_w)


@torch.library.register_fake("dora_amd::adapter_combine_backward")
def _adapter_combine_backward_fake(dy, rows, weights, place, want_rows, want_weights):
    return (dy.new_empty((place.shape[0] * place.shape[1], dy.shape[1]) if want_rows else (0,)),
            dy.new_empty(place.shape if want_weights else (0,), dtype=torch.float32))


# -------------------------------------------------------------------------- layer


class DoRALinear(torch.nn.Module):
    """DoRA-adapted linear layer: frozen W0 [out x in], trainable A [r x in],
    B [out x r] and magnitude m [out] (fp32); scale s = alpha / sqrt(r) (rsLoRA).

    Initialisation follows LoRA/DoRA practice: B = 0 and m = ||W0|| per row,
    so the layer starts out equal to x W0^T.  A is drawn from N(0, 1/in).  On a
    HIP device m is taken from the factored norm itself, so g = m / n is exactly
    1 at B = 0 and the first output equals x W0^T bit for bit.

    W0 is frozen, so its row square norms are computed once (on the first norm
    on a HIP device) and kept in the buffer ``weight_sqnorm``; the norm then
    takes its base term from there.  After changing ``weight``, call
    ``refresh_weight_cache()``.

    ``detach_norm`` (default True) treats n as a constant in the backward; with
    False the gradients of A and B also carry the path through n, by the
    factored norm backward.

    ``q8_checkpoint`` keeps x and base, all that the backward needs of size
    T x in and T x out, in 8-bit blocks instead of 16 bits: half the activation
    memory.  d_mag and d_A then come from those values, d_B and dx do not change.
    ``q8_weight`` (which implies it) also holds W0 itself in 8-bit blocks (the
    buffers ``weight_q``, ``weight_e``; ``weight`` is None) and runs both products
    with W0 on packed operands.  n is the norm of the values W0 is held as, so the
    layer still starts out with g = 1.  Under autocast both compute in its type.
    ``q4_weight`` holds W0 in 4-bit blocks instead (the same buffers) and multiplies
    it with x and d_base in 16 bits; with ``q8_checkpoint`` x and base are kept in 8.
    """

    def __init__(self, in_features: int, out_features: int, r: int, alpha: float = 32.0,
                 weight: Tensor | None = None, dtype: torch.dtype = torch.bfloat16, device=None,
                 detach_norm: bool = True, q8_weight: bool = False, q8_checkpoint: bool = False,
                 q4_weight: bool = False):
        super().__init__()
        if q8_weight and q4_weight:
            raise ValueError("the weight is held in 8 bits or in 4, not both")
        self.detach_norm = detach_norm
        if dtype not in (torch.bfloat16, torch.float16, torch.float32):
            raise ValueError(f"unsupported dtype {dtype}; bf16 and fp16 (HIP kernels) and fp32 (eager tier) are")
        self.in_features, self.out_features, self.r = in_features, out_features, r
        self.s = float(np.float32(alpha / math.sqrt(r)))
        if weight is None:
            weight = torch.randn(out_features, in_features, device=device) / math.sqrt(in_features)
        self.q8_weight, self.q8_checkpoint, self.q4_weight = q8_weight, q8_weight or q8_checkpoint, q4_weight
        weight = weight.to(device=device, dtype=dtype).contiguous()
        if q8_weight or q4_weight:
            # bytes, so that a change of the module's dtype leaves them alone
            weight = weight.detach()  # it may be another layer's parameter
            q, e = (q4_pack_weight if q4_weight else q8_pack_weight)(weight)
            self.register_buffer("weight", None)
            self.register_buffer("weight_q", q.view(torch.uint8))
            self.register_buffer("weight_e", e)
            weight = (q4_unpack_weight if q4_weight else q8_unpack_weight)(q, e, out_features, in_features, dtype)
        else:
            self.register_buffer("weight", weight)
        self.lora_A = torch.nn.Parameter(
            (torch.randn(r, in_features, device=device) / math.sqrt(in_features)).to(dtype))
        self.lora_B = torch.nn.Parameter(torch.zeros(out_features, r, device=device, dtype=dtype))
        self.magnitude = torch.nn.Parameter(weight.float().norm(dim=1))
        self.register_buffer("weight_sqnorm", None)
        if weight.is_cuda:
            self.reset_magnitude()

    def _packed_weight(self) -> tuple[Tensor, Tensor]:
        return self.weight_q if self.q4_weight else self.weight_q.view(_F8), self.weight_e

    @torch.no_grad()
    def refresh_weight_cache(self) -> None:
        """Recompute ||W0_i||^2 (after ``weight`` changed)."""
        if self.q8_weight or self.q4_weight:
            wq, we = self._packed_weight()
            n = torch.empty(self.out_features, dtype=torch.float32, device=wq.device)
            slabs = _q4_slabs if self.q4_weight else _slabs
            for rows, W in slabs(wq, we, self.out_features, self.in_features, self.lora_A.dtype):
                n[rows] = row_sqnorm(W)
            self.weight_sqnorm = n
        else:
            self.weight_sqnorm = row_sqnorm(self.weight)

    @torch.no_grad()
    def reset_magnitude(self) -> None:
        """m = ||W0 + s*B*A|| per row (the DoRA initialisation of the magnitude)."""
        self.magnitude.copy_(self.weight_norm())

    def weight_norm(self) -> Tensor:
        """n = ||W0 + s*B*A|| per output row (base term from the cache); detached
        unless the layer was built with ``detach_norm=False``."""
        if self.weight_sqnorm is None or self.weight_sqnorm.device != self.lora_A.device:
            self.refresh_weight_cache()
        A, B = (self.lora_A.detach(), self.lora_B.detach()) if self.detach_norm else (self.lora_A, self.lora_B)
        if self.q8_weight:
            return q8_weight_norm(*self._packed_weight(), A, B, self.weight_sqnorm, self.s)
        if self.q4_weight:
            return q4_weight_norm(*self._packed_weight(), A, B, self.weight_sqnorm, self.s)
        return weight_norm_cached(self.weight, A, B, self.weight_sqnorm, self.s)

    def forward(self, x: Tensor) -> Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features)
        weight, we = self._packed_weight() if self.q8_weight or self.q4_weight else (self.weight, None)
        n = self.weight_norm()
        trained = (x2, self.lora_A, self.lora_B, self.magnitude, n)
        if self.q8_checkpoint and torch.is_grad_enabled() and any(t.requires_grad for t in trained):
            y = q8_layer(x2, self.lora_A, self.lora_B, self.magnitude, n, weight, we, self.s)[0]
            return y.reshape(*lead, self.out_features)
        B = self.lora_B
        if self.q8_checkpoint or self.q4_weight:  # the types of the training tier
            x2, B = _autocast(x2, B)
        if self.q4_weight:
            base = q4_linear(x2, weight, we, self.out_features)
        elif self.q8_weight:  # x is packed for the product alone
            base = q8_linear(*q8_pack(x2), weight, we, self.out_features, x2.dtype)
        else:
            base = F.linear(x2, weight)
        h = F.linear(x2, self.lora_A)
        # lora = h B^T is formed inside the compose kernel on both tiers; on the
        # training tier autograd records it and its backward (lora_compose_backward)
        # never forms lora or d_lora either, so nothing T x out is saved for lora
        y = lora_compose(base, h, B, self.magnitude, n, self.s, True)
        return y.reshape(*lead, self.out_features)


class DoRAAdapters(torch.nn.Module):
    """Several DoRA adapters over one frozen weight W0 [out x in]: adapter a has its own
    A [r x in], B [out x r] and magnitude [out] (slices of ``lora_A``, ``lora_B`` and
    ``magnitude``), and each token of a batch says which it uses, as in a batch of
    requests to different adapters, or a mixture of them:

      y_t = x_t W0^T + sum_j w_tj * delta_{id_tj}(x_t),
      delta_a(x) = (g_a - 1) * (x W0^T) + g_a * s * (x A_a^T B_a^T),  g_a = m_a / n_a.

    ``forward(x, ids, weights)``: x [.. x in], ids whole numbers [..] or [.. x k] (any
    outside [0, adapters) is no adapter), weights like ids, or None for ones.  The
    product with W0 runs once for all tokens; tokens are then sorted by adapter, each
    adapter's rows go through ``lora_compose`` together, and come back per token with
    their weights.  The rows' bounds are read by the host once a call.  W0 in 16 bits,
    or with ``q4_weight`` in 4-bit blocks; initialisation, ``detach_norm`` and the cache
    of ||W0_i||^2 as in ``DoRALinear``.
    """

    def __init__(self, in_features: int, out_features: int, r: int, adapters: int, alpha: float = 32.0,
                 weight: Tensor | None = None, dtype: torch.dtype = torch.bfloat16, device=None,
                 detach_norm: bool = True, q4_weight: bool = False):
        super().__init__()
        if adapters < 1:
            raise ValueError(f"{adapters} adapters")
        one = DoRALinear(in_features, out_features, r, alpha, weight, dtype, device, detach_norm, q4_weight=q4_weight)
        self.in_features, self.out_features, self.r, self.adapters = in_features, out_features, r, adapters
        self.s, self.detach_norm, self.q4_weight = one.s, detach_norm, q4_weight
        for name in ("weight", "weight_q", "weight_e", "weight_sqnorm"):
            if hasattr(one, name):
                self.register_buffer(name, getattr(one, name))
        A = torch.randn(adapters, r, in_features, device=device) / math.sqrt(in_features)
        self.lora_A = torch.nn.Parameter(A.to(dtype))
        self.lora_B = torch.nn.Parameter(torch.zeros(adapters, out_features, r, device=device, dtype=dtype))
        self.magnitude = torch.nn.Parameter(one.magnitude.detach().repeat(adapters, 1))

    q8_weight = False
    _packed_weight = DoRALinear._packed_weight
    refresh_weight_cache = DoRALinear.refresh_weight_cache

    @torch.no_grad()
    def reset_magnitude(self) -> None:
        """m_a = ||W0 + s*B_a*A_a|| per row, of every adapter."""
        for a in range(self.adapters):
            self.magnitude[a].copy_(self.weight_norm(a))

    def weight_norm(self, adapter: int) -> Tensor:
        """n_a = ||W0 + s*B_a*A_a|| per output row."""
        return self._norm_of(self.lora_A[adapter], self.lora_B[adapter])

    def _norm_of(self, A: Tensor, B: Tensor) -> Tensor:
        if self.weight_sqnorm is None or self.weight_sqnorm.device != A.device:
            self.refresh_weight_cache()
        if self.detach_norm:
            A, B = A.detach(), B.detach()
        if self.q4_weight:
            return q4_weight_norm(*self._packed_weight(), A, B, self.weight_sqnorm, self.s)
        return weight_norm_cached(self.weight, A, B, self.weight_sqnorm, self.s)

    def forward(self, x: Tensor, ids: Tensor, weights: Tensor | None = None) -> Tensor:
        lead = x.shape[:-1]
        if ids.shape[: len(lead)] != lead or ids.dim() > len(lead) + 1:
            raise ValueError(f"ids are {tuple(ids.shape)}, expected {tuple(lead)} or {tuple(lead)} x k")
        if weights is not None and weights.shape != ids.shape:
            raise ValueError(f"weights are {tuple(weights.shape)}, expected {tuple(ids.shape)}")
        k = ids.shape[-1] if ids.dim() > len(lead) else 1
        x2 = x.reshape(-1, self.in_features)
        T = x2.shape[0]
        (x2,) = _autocast(x2)
        if self.q4_weight:
            base = q4_linear(x2, *self._packed_weight(), self.out_features)
        else:
            base = F.linear(x2, self.weight)
        order, place, bounds = adapter_sort(ids.reshape(T, k), self.adapters)
        ends = bounds.tolist()
        sizes = [b - a for a, b in zip(ends, ends[1:] + [T * k])]  # the rows of slots without an adapter last
        # taken apart once: the gradient of each slice by itself would be the whole's, in zeros
        xs, bs = adapter_gather(x2, place).split(sizes), adapter_gather(base, place).split(sizes)
        parts = []
        for xa, ba, A, B, m in zip(xs, bs, self.lora_A.unbind(), self.lora_B.unbind(), self.magnitude.unbind()):
            if xa.shape[0] > 0:
                h, n = F.linear(xa, A), self._norm_of(A, B)
                (B,) = _autocast(B)
                parts.append(lora_compose(ba, h, B, m, n, self.s, False))
        if sizes[-1] > 0:  # not used
            parts.append(base.new_zeros((sizes[-1], self.out_features)))
        rows = torch.cat(parts) if parts else base.new_zeros((0, self.out_features))
        y = adapter_combine(rows, None if weights is None else weights.reshape(T, k), place, base)
        return y.reshape(*lead, self.out_features)
