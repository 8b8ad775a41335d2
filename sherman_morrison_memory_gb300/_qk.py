"""Norm and position rotation of queries and keys (C ABI in include/vla_layer.h),
with the conventions of _layer.py."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import _DTYPES, _call_buffer, _Seq, load_library
from ._layer import _check_f32, _check_out, _check_seq, _done, _handle, _norm_weight, _on, _ptr, _seq, _seq_in


@functools.lru_cache(maxsize=256)
def _scratch(B: int, H: int, T: int, d: int, device_index: int) -> int:
    """vla_qk_norm_scratch_bytes on a device (made current by the caller)."""
    return int(load_library().vla_qk_norm_scratch_bytes(B, H, T, d))


def vla_rotation_frequencies(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """base ** (-2 i / rot) for i < rot / 2, float64 [rot / 2] on ``device``: radians a
    position for vla_qk_norm. ``rot`` is a multiple of 16."""
    if rot <= 0 or rot % 16:
        raise ValueError(f"rot must be a positive multiple of 16, got {rot}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)


def _rows(x: torch.Tensor):
    """x where the kernels can read it (copied if it has to be) and its vla_seq. The common case, every stride positive
    and a multiple of 16 bytes, is decided here: small calls are bound by this file's work."""
    s0, s1, s2, s3 = x.stride()
    p = x.data_ptr()
    if s3 == 1 and not p & 15 and s0 > 0 and s1 > 0 and s2 > 0 and not (s0 | s1 | s2) & (7 if x.dtype == torch.bfloat16 else 3):
        return x, ctypes.byref(_Seq(p, s0, s1, s2))
    x = _seq_in(x)
    return x, _seq(x)


def _rotation(freqs, positions, B, T, d, dev):
    """(freqs, rot, positions, their stride from sequence to sequence), checked."""
    if freqs is None:
        return None, 0, None, 0
    if freqs.dim() != 1 or freqs.dtype != torch.float64 or freqs.device != dev:
        raise ValueError(f"freqs must be float64 [rot / 2] on {dev}")
    rot = 2 * freqs.shape[0]
    if rot == 0 or rot % 16 or rot > d:
        raise ValueError(f"freqs must have a multiple of 8 and at most {d // 2} values, got {rot // 2}")
    freqs = freqs.contiguous()
    if positions is None:
        return freqs, rot, None, 0
    if tuple(positions.shape) not in ((B, T), (T,)) or positions.dtype != torch.int32 or positions.device != dev:
        raise ValueError(f"positions must be int32 ({B}, {T}) or ({T},) on {dev}")
    positions = positions.contiguous()
    return freqs, rot, positions, T if positions.dim() == 2 else 0


def _weights(weight_q, weight_k, H, d, dev):
    if (weight_q is None) != (weight_k is None) or (weight_q is not None and weight_q.shape != weight_k.shape):
        raise ValueError("weight_q and weight_k must have the same shape, or both be None")
    return _norm_weight(weight_q, H, d, dev, "weight_q"), _norm_weight(weight_k, H, d, dev, "weight_k")


def vla_qk_norm(q: torch.Tensor, k: torch.Tensor, weight_q: Optional[torch.Tensor] = None,
                weight_k: Optional[torch.Tensor] = None, eps: float = 1e-6, *, unit: bool = False,
                freqs: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, out=None, stream=None):
    """Norm of each row of q and k [B, H, T, d], and rotation by its position:
    x rstd weight, rstd = 1 / sqrt(mean(x^2) + eps), or 1 / sqrt(sum(x^2) + eps)
    for ``unit`` (rows of length 1, for a delta rule's keys); then coordinates i and
    i + rot / 2 are turned by the angle position * freqs[i].

    ``weight_q``, ``weight_k`` float32 [H, d], or [d] for all heads (None: 1).
    ``freqs`` float64 [rot / 2] (vla_rotation_frequencies; None: no rotation), rot a
    multiple of 16 up to d; ``positions`` int32 [B, T] or [T] (None: token t is at
    t; not looked at without ``freqs``). Returns ``((yq, yk), (rstd_q, rstd_k))``: like q and k, and float32
    [B, H, T] for vla_qk_norm_backward. ``out`` = (yq, yk) preallocated, rows in any
    order; yq may be q, and yk may be k.
    """
    _check_seq(q, "q")
    _check_seq(k, "k", q)
    eps = float(eps)
    if not 0 <= eps < 3.4e38:
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    with _on(dev, stream):
        wq, wk = _weights(weight_q, weight_k, H, d, dev)
        freqs, rot, positions, stride = _rotation(freqs, positions, B, T, d, dev)
        if out is None:
            yq = torch.empty((B, H, T, d), dtype=q.dtype, device=dev)
            yk = torch.empty((B, H, T, d), dtype=q.dtype, device=dev)
        else:
            yq, yk = out
            for i, x in enumerate((yq, yk)):
                _check_out(x, (B, H, T, d), q.dtype, dev, f"out[{i}]", strided=True)
        rstd = (torch.empty((B, H, T), dtype=torch.float32, device=dev), torch.empty((B, H, T), dtype=torch.float32, device=dev))
        (q, sq), (k, sk) = _rows(q), _rows(k)
        st = lib.vla_qk_norm(sq, sk, _DTYPES[q.dtype], B, H, T, d, _ptr(wq), _ptr(wk), int(wq is not None and wq.dim() == 1),
                             int(bool(unit)), eps, _ptr(freqs), rot, _ptr(positions), stride, _seq(yq), _seq(yk),
                             rstd[0].data_ptr(), rstd[1].data_ptr(), _handle(dev, stream))
    _done(st, "vla_qk_norm", dev, stream, False)
    return (yq, yk), rstd


def vla_qk_norm_backward(grad_q: torch.Tensor, grad_k: torch.Tensor, q: torch.Tensor, k: torch.Tensor, stats,
                         weight_q: Optional[torch.Tensor] = None, weight_k: Optional[torch.Tensor] = None, *,
                         unit: bool = False, freqs: Optional[torch.Tensor] = None,
                         positions: Optional[torch.Tensor] = None, out=None, stream=None):
    """Gradient of a scalar loss through vla_qk_norm: ``((dq, dk), (dweight_q,
    dweight_k))``.

    ``grad_q``, ``grad_k`` = dL/dyq, dL/dyk and q, k [B, H, T, d]; ``stats`` =
    (rstd_q, rstd_k) as the forward call returned them; the other arguments as in
    that call. dq and dk are like q; the weights' gradients are float32, shaped as
    the weights (None without weights). ``out`` = (dq, dk) preallocated; each may be
    its gradient's rows or its input's.
    """
    _check_seq(q, "q")
    for name, x in (("k", k), ("grad_q", grad_q), ("grad_k", grad_k)):
        _check_seq(x, name, q)
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    rstd_q, rstd_k = stats
    with _on(dev, stream):
        wq, wk = _weights(weight_q, weight_k, H, d, dev)
        rstd_q = _check_f32(rstd_q, (B, H, T), dev, "rstd_q")
        rstd_k = _check_f32(rstd_k, (B, H, T), dev, "rstd_k")
        freqs, rot, positions, stride = _rotation(freqs, positions, B, T, d, dev)
        if out is None:
            dq = torch.empty((B, H, T, d), dtype=q.dtype, device=dev)
            dk = torch.empty((B, H, T, d), dtype=q.dtype, device=dev)
        else:
            dq, dk = out
            for i, x in enumerate((dq, dk)):
                _check_out(x, (B, H, T, d), q.dtype, dev, f"out[{i}]", strided=True)
        dwq = dwk = scratch = None
        nbytes = 0
        if wq is not None:
            dwq, dwk = torch.empty_like(wq), torch.empty_like(wk)
            nbytes = _scratch(B, H, T, d, dev.index)
            scratch = _call_buffer(dev, nbytes, False) if nbytes else None
        (q, sq), (k, sk), (grad_q, sgq), (grad_k, sgk) = _rows(q), _rows(k), _rows(grad_q), _rows(grad_k)
        st = lib.vla_qk_norm_backward(sgq, sgk, sq, sk, _DTYPES[q.dtype], B, H, T, d, _ptr(wq),
                                      _ptr(wk), int(wq is not None and wq.dim() == 1), int(bool(unit)), _ptr(freqs), rot,
                                      _ptr(positions), stride, _ptr(rstd_q), _ptr(rstd_k), _seq(dq), _seq(dk), _ptr(dwq),
                                      _ptr(dwk), _ptr(scratch), nbytes, _handle(dev, stream))
    _done(st, "vla_qk_norm_backward", dev, stream, False)
    return (dq, dk), (dwq, dwk)
