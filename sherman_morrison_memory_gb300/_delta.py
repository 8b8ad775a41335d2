"""The gated delta rule (C ABI in include/vla_layer.h), with the conventions of
_layer.py. Its gates, ``log_decay`` and ``beta``, are [B, H, T] float32 tensors
with any strides: a projection's [B, T, H] output is passed as
``x.transpose(1, 2)``, a constant one as ``x.expand(B, H, T)``.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import _DTYPES, _call_buffer, _Seq, _workspace, load_library
from ._layer import (_check_f32, _check_index, _check_out, _check_seq, _done, _handle, _on, _ptr, _scale, _seq, _seq_in,
                     _wait_options, _DIMS)


@functools.lru_cache(maxsize=256)
def _scratch(dtype: int, B: int, H: int, T: int, d: int) -> int:
    return int(load_library().vla_delta_scratch_bytes(dtype, B, H, T, d))


def _gate_in(x: torch.Tensor, shape, device, name: str) -> torch.Tensor:
    """A gate, read at its own strides."""
    if tuple(x.shape) != tuple(shape) or x.dtype != torch.float32 or x.device != device:
        raise ValueError(f"{name} must be float32 {tuple(shape)} on {device}, got {x.dtype} {tuple(x.shape)} {x.device}")
    return x


def _gate(x: Optional[torch.Tensor]):
    return None if x is None else ctypes.byref(_Seq(x.data_ptr(), *x.stride()))


def _gate_out(x: torch.Tensor, shape, device, name: str):
    if tuple(x.shape) != tuple(shape) or x.dtype != torch.float32 or x.device != device:
        raise ValueError(f"{name} must be float32 {tuple(shape)} on {device}")
    if any(n > 1 and s <= 0 for n, s in zip(x.shape, x.stride())):
        raise ValueError(f"{name} must have positive strides")


def vla_delta_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                      beta: torch.Tensor, scale: float = 1.0, state: Optional[torch.Tensor] = None, *,
                      lengths: Optional[torch.Tensor] = None, out=None, stream=None, check: bool = False,
                      wait_limit_us: int = 0, test_stall_producer: bool = False):
    """The gated delta rule over a sequence, a_t = exp(log_decay_t):
    S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T, o_t = scale S_t q_t.

    Returns ``(o, S)``: o like q, S [B, H, d, d] float32, the state behind each
    sequence's last token. ``log_decay`` (None: 0) and ``beta`` [B, H, T]
    float32. Keys are taken as they are; vla_qk_norm(unit=True) makes unit rows.
    ``state`` [B, H, d, d] float32 continues a previous call. ``lengths`` [B]
    int32 (on the device): sequence b has only its first lengths[b] tokens; o is
    zero behind them. S is fp32 in bf16 calls too, and o is rounded at the end.
    A token's NaN or Inf (in k, v or a gate) reaches the tokens behind it in its
    head, and may reach those before it in its block of 32. A head that grows
    (log_decay above 0) beyond float32 within 32 tokens gives Inf or NaN.
    ``out`` = (o, S) preallocated; S may be ``state``. ``check=True``
    synchronises and raises on an in-kernel failure or a non-finite result.
    ``wait_limit_us`` (0: 2,000,000) bounds each in-kernel wait;
    ``test_stall_producer=True`` (testing only) makes them run out
    (VLA_ERR_TIMEOUT): bf16 calls of more than 64 tokens have such waits.
    """
    for name, x in (("q", q), ("k", k), ("v", v)):
        _check_seq(x, name, None if x is q else q)
    scale = _scale(scale)
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    with _on(dev, stream):
        g = None if log_decay is None else _gate_in(log_decay, (B, H, T), dev, "log_decay")
        beta = _gate_in(beta, (B, H, T), dev, "beta")
        S0 = _check_f32(state, (B, H, d, d), dev, "state")
        lengths = _check_index(lengths, B, dev, "lengths")
        if out is None:
            o = torch.empty((B, H, T, d), dtype=q.dtype, device=dev)
            S = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
        else:
            o, S = out
            _check_out(o, (B, H, T, d), q.dtype, dev, "out[0]", strided=True)
            _check_out(S, (B, H, d, d), torch.float32, dev, "out[1]")
        q, k, v = (_seq_in(x) for x in (q, k, v))
        args = (_seq(q), _seq(k), _seq(v), _DTYPES[q.dtype], B, H, T, d, _gate(g), _gate(beta), scale, _ptr(lengths),
                _ptr(S0), _seq(o), _ptr(S), _ptr(_workspace(dev)), _handle(dev, stream))
        if wait_limit_us or test_stall_producer:
            st = lib.vla_delta_forward_ex(*args, _wait_options(wait_limit_us, test_stall_producer))
        else:
            st = lib.vla_delta_forward(*args)
    _done(st, "vla_delta_forward", dev, stream, check)
    return o, S


def vla_delta_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                       beta: torch.Tensor, scale: float = 1.0, state: Optional[torch.Tensor] = None,
                       grad_o: Optional[torch.Tensor] = None, grad_state: Optional[torch.Tensor] = None, *,
                       lengths: Optional[torch.Tensor] = None, out=None, stream=None, check: bool = False,
                       wait_limit_us: int = 0, test_stall_producer: bool = False):
    """Gradient of a scalar loss through vla_delta_forward (reverse mode).

    ``grad_o`` = dL/do like q and ``grad_state`` = dL/dS [B, H, d, d] float32
    (each optional, None = zero); the other arguments as in the forward call, of
    which nothing is kept. Returns ``((dq, dk, dv), (dlog_decay, dbeta), dS0)``:
    like q, [B, H, T] float32 (dlog_decay None for a None log_decay), and
    float32 [B, H, d, d]. A gate that is expanded gets its gradient for each
    token, not their sum. A NaN or Inf reaches what depends on it, and may reach
    the other tokens of its block of 64 in the same head. ``out`` = (dq, dk, dv, dlog_decay, dbeta, dS0)
    preallocated (dS0 neither ``state`` nor ``grad_state``). ``wait_limit_us``
    and ``test_stall_producer`` as in the forward call.
    """
    for name, x in (("q", q), ("k", k), ("v", v), ("grad_o", grad_o)):
        if x is not None:
            _check_seq(x, name, None if x is q else q)
    scale = _scale(scale)
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    with _on(dev, stream):
        g = None if log_decay is None else _gate_in(log_decay, (B, H, T), dev, "log_decay")
        beta = _gate_in(beta, (B, H, T), dev, "beta")
        S0 = _check_f32(state, (B, H, d, d), dev, "state")
        dS_T = _check_f32(grad_state, (B, H, d, d), dev, "grad_state")
        lengths = _check_index(lengths, B, dev, "lengths")
        if grad_o is None:
            grad_o = torch.zeros((B, H, T, d), dtype=q.dtype, device=dev)
        if out is None:
            grads = [torch.empty((B, H, T, d), dtype=q.dtype, device=dev) for _ in range(3)]
            dg = None if g is None else torch.empty((B, H, T), dtype=torch.float32, device=dev)
            db = torch.empty((B, H, T), dtype=torch.float32, device=dev)
            dS0 = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
        else:
            if len(out) != 6:
                raise ValueError("out must hold (dq, dk, dv, dlog_decay, dbeta, dS0)")
            *grads, dg, db, dS0 = out
            for i, x in enumerate(grads):
                _check_out(x, (B, H, T, d), q.dtype, dev, f"out[{i}]", strided=True)
            if (dg is None) != (g is None):
                raise ValueError("out[3] must be given with log_decay, and None without")
            if dg is not None:
                _gate_out(dg, (B, H, T), dev, "out[3]")
            _gate_out(db, (B, H, T), dev, "out[4]")
            _check_out(dS0, (B, H, d, d), torch.float32, dev, "out[5]")
        q, k, v, grad_o = (_seq_in(x) for x in (q, k, v, grad_o))
        nbytes = _scratch(_DTYPES[q.dtype], B, H, T, d)
        scratch = _call_buffer(dev, nbytes, False) if nbytes else None
        args = (_seq(q), _seq(k), _seq(v), _seq(grad_o), _DTYPES[q.dtype], B, H, T, d, _gate(g), _gate(beta), scale,
                _ptr(lengths), _ptr(S0), _ptr(dS_T), *(_seq(x) for x in grads), _gate(dg), _gate(db), _ptr(dS0),
                _ptr(scratch), nbytes, _ptr(_workspace(dev)), _handle(dev, stream))
        if wait_limit_us or test_stall_producer:
            st = lib.vla_delta_backward_ex(*args, _wait_options(wait_limit_us, test_stall_producer))
        else:
            st = lib.vla_delta_backward(*args)
    _done(st, "vla_delta_backward", dev, stream, check)
    return tuple(grads), (dg, db), dS0


def vla_delta_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                   beta: torch.Tensor, state: torch.Tensor, scale: float = 1.0, *,
                   slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None,
                   check: bool = False) -> torch.Tensor:
    """One token of vla_delta_forward's rule for a batch of sequences.

    q, k, v [B, H, d], ``log_decay`` (None: 0) and ``beta`` [B, H] float32
    (copied unless contiguous); ``state`` [N, H, d, d] float32, contiguous, is
    updated in place; ``slots`` as for vla_decay_step: [B] int32 (on the device),
    each sequence's entry of it (None: entry b), negative for an idle row, whose
    o is zero; one that is out of range or was used by an earlier row is left
    alone too and recorded (VLA_ERR_BAD_SLOT, raised by ``check=True``).
    Returns o like q.
    """
    if q.dim() != 3 or q.dtype not in _DTYPES or q.device.type != "cuda" or q.shape[-1] not in _DIMS:
        raise ValueError(f"q must be a [B, H, d] float32 or bfloat16 CUDA tensor, d in {_DIMS}")
    for name, x in (("k", k), ("v", v)):
        if x.shape != q.shape or x.dtype != q.dtype or x.device != q.device:
            raise ValueError(f"{name} must match q in shape, dtype and device")
    scale = _scale(scale)
    lib = load_library()
    B, H, d = q.shape
    dev = q.device
    if state.dim() != 4:
        raise ValueError("state must be [N, H, d, d]")
    N = state.shape[0]
    _check_out(state, (N, H, d, d), torch.float32, dev, "state")
    if slots is None and B > N:
        raise ValueError(f"{B} sequences for {N} states")
    with _on(dev, stream):
        log_decay = _check_f32(log_decay, (B, H), dev, "log_decay")
        beta = _check_f32(beta, (B, H), dev, "beta")
        slots = _check_index(slots, B, dev, "slots")
        if out is None:
            out = torch.empty((B, H, d), dtype=q.dtype, device=dev)
        else:
            _check_out(out, (B, H, d), q.dtype, dev, "out")
        q, k, v = (x if x.is_contiguous() and x.data_ptr() % 16 == 0
                   else x.clone(memory_format=torch.contiguous_format) for x in (q, k, v))
        st = lib.vla_delta_step(_ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], B, H, d, _ptr(log_decay), _ptr(beta), scale,
                                _ptr(state), N, _ptr(slots), _ptr(out), _ptr(_workspace(dev)), _handle(dev, stream))
    _done(st, "vla_delta_step", dev, stream, check)
    return out
