"""Operators around the recurrence (C ABI in include/vla_layer.h).

As in _binding.py: arguments are checked, outputs and scratch are allocated
with torch on the call's stream, and the C entry points are called there. All
arithmetic happens in the library. CUDA tensors only.

Sequences are [B, H, T, d] float32 or bfloat16 with any strides: a
projection's [B, T, H, d] output is passed as ``x.transpose(1, 2)`` and read
in place. One whose last dimension is not dense, or whose rows do not start on
16-byte boundaries, is copied first. Results that are sequences have the
inputs' type; states, statistics and weights are float32. Preallocated outputs
share no memory with inputs or each other (VLAError), except where a call says
that it works in place; rows that lie between those of another array are fine.
Any call may be captured in a CUDA graph after one eager call of the package on
the device (which lays out the shared status record).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import Optional

import torch

from ._binding import (_DTYPES, VLA_OK, VLAError, _call_buffer, _Options, _Seq, _workspace, load_library,
                       vla_get_last_device_status)

_DIMS = (32, 64, 96, 128)
_GROUP = 32


_HERE = contextlib.nullcontext()


def _on(dev: torch.device, stream):
    """The device and stream of a call made current (nothing to do where they are)."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"a stream of {stream.device} for tensors on {dev}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _handle(dev: torch.device, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _ptr(x: Optional[torch.Tensor]):
    return None if x is None else x.data_ptr()


@functools.lru_cache(maxsize=256)
def _decay_scratch(B: int, H: int, T: int, d: int, backward: int, device_index: int) -> int:
    """vla_decay_scratch_bytes on a device (made current by the caller)."""
    return int(load_library().vla_decay_scratch_bytes(B, H, T, d, backward))


def _in_place(x: torch.Tensor) -> bool:
    """Whether the kernels can read (and write) x's rows where they are."""
    es = x.element_size()
    return (x.stride(-1) == 1 and x.data_ptr() % 16 == 0
            and all(n <= 1 or (s > 0 and s * es % 16 == 0) for n, s in zip(x.shape[:-1], x.stride()[:-1])))


def _seq_in(x: torch.Tensor) -> torch.Tensor:
    if x.numel() == 0 or _in_place(x):
        return x
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _seq(x: Optional[torch.Tensor]):
    if x is None:
        return None
    return ctypes.byref(_Seq(x.data_ptr(), *x.stride()[:3]))


def _check_seq(x: torch.Tensor, name: str, like: Optional[torch.Tensor] = None):
    if x.dim() != 4 or x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a [B, H, T, d] float32 or bfloat16 tensor")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None and (x.shape != like.shape or x.dtype != like.dtype or x.device != like.device):
        raise ValueError(f"{name} must match in shape, dtype and device: {tuple(x.shape)} {x.dtype} {x.device}, "
                         f"not {tuple(like.shape)} {like.dtype} {like.device}")
    if x.shape[-1] not in _DIMS:
        raise ValueError(f"head dimension {x.shape[-1]} is not one of {_DIMS}")


def _check_out(x: torch.Tensor, shape, dtype, device, name: str, strided: bool = False):
    if tuple(x.shape) != tuple(shape) or x.dtype != dtype or x.device != device:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device}")
    if x.numel() and not (_in_place(x) if strided else x.is_contiguous() and x.data_ptr() % 16 == 0):
        raise ValueError(f"{name} must " + ("have dense rows on 16-byte boundaries" if strided
                                            else "be contiguous and start on a 16-byte boundary"))


def _check_f32(x: Optional[torch.Tensor], shape, device, name: str) -> Optional[torch.Tensor]:
    """A float32 input, contiguous and 16-byte aligned (copied if it is not)."""
    if x is None:
        return None
    if tuple(x.shape) != tuple(shape) or x.dtype != torch.float32 or x.device != device:
        raise ValueError(f"{name} must be float32 {tuple(shape)} on {device}, got {x.dtype} {tuple(x.shape)} {x.device}")
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _check_index(x: Optional[torch.Tensor], n: int, device, name: str) -> Optional[torch.Tensor]:
    if x is None:
        return None
    if tuple(x.shape) != (n,) or x.dtype != torch.int32 or x.device != device:
        raise ValueError(f"{name} must be int32 ({n},) on {device}, got {x.dtype} {tuple(x.shape)} {x.device}")
    return x.contiguous()


def _scale(scale) -> float:
    scale = float(scale)
    if scale != scale or scale in (float("inf"), float("-inf")):
        raise ValueError(f"scale must be finite, got {scale}")
    return scale


def _wait_options(wait_limit_us: int, stall: bool):
    return ctypes.byref(_Options(wait_limit_us=int(wait_limit_us), test_stall_producer=1 if stall else 0))


def _done(st: int, name: str, device, stream, check: bool):
    if st != VLA_OK:
        raise VLAError(st, name)
    if check:
        st, detail = vla_get_last_device_status(device, stream)
        if st != VLA_OK:
            raise VLAError(st, f"{name} (device)", detail)


def vla_decay_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, scale: float = 1.0,
                      state: Optional[torch.Tensor] = None, *, lengths: Optional[torch.Tensor] = None, out=None,
                      stream=None, check: bool = False, wait_limit_us: int = 0, test_stall_producer: bool = False):
    """Linear attention with a decay per head over a sequence:
    S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.

    Returns ``(o, S)``: o like q, S [B, H, d, d] float32, the state behind each
    sequence's last token. ``log_decay`` [H] float32; ``state`` [B, H, d, d]
    float32 continues a previous call. ``lengths`` [B] int32 (on the device):
    sequence b has only its first lengths[b] tokens; o is zero behind them.
    bf16 calls of more than 8 tokens round pair products and the state that a
    chunk's tokens see to bf16 on the way to o (S itself stays fp32).
    ``out`` = (o, S) preallocated; S may be ``state``. ``check=True``
    synchronises and raises on an in-kernel failure or a non-finite result.
    ``wait_limit_us`` (0: 2,000,000) bounds each in-kernel wait;
    ``test_stall_producer=True`` (testing only) makes them run out
    (VLA_ERR_TIMEOUT): bf16 calls of more than 8 tokens have such waits.
    """
    for name, x in (("q", q), ("k", k), ("v", v)):
        _check_seq(x, name, None if x is q else q)
    scale = _scale(scale)
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    with _on(dev, stream):
        log_decay = _check_f32(log_decay, (H,), dev, "log_decay")
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
        nbytes = _decay_scratch(B, H, T, d, 0, dev.index)
        scratch = _call_buffer(dev, nbytes, False) if nbytes else None
        args = (_seq(q), _seq(k), _seq(v), _DTYPES[q.dtype], B, H, T, d, _ptr(log_decay), scale, _ptr(lengths),
                _ptr(S0), _seq(o), _ptr(S), _ptr(scratch), nbytes, _ptr(_workspace(dev)), _handle(dev, stream))
        if wait_limit_us or test_stall_producer:
            st = lib.vla_decay_forward_ex(*args, _wait_options(wait_limit_us, test_stall_producer))
        else:
            st = lib.vla_decay_forward(*args)
    _done(st, "vla_decay_forward", dev, stream, check)
    return o, S


def vla_decay_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, scale: float = 1.0,
                       state: Optional[torch.Tensor] = None, grad_o: Optional[torch.Tensor] = None,
                       grad_state: Optional[torch.Tensor] = None, *, lengths: Optional[torch.Tensor] = None, out=None,
                       stream=None, check: bool = False, wait_limit_us: int = 0, test_stall_producer: bool = False):
    """Gradient of a scalar loss through vla_decay_forward (reverse mode).

    ``grad_o`` = dL/do like q and ``grad_state`` = dL/dS [B, H, d, d] float32
    (each optional, None = zero); the other arguments as in the forward call,
    of which nothing is kept. Returns ``((dq, dk, dv), dS0)``: like q, and
    float32 [B, H, d, d]. No gradient is formed for log_decay and scale.
    ``out`` = (dq, dk, dv, dS0) preallocated (dS0 neither ``state`` nor
    ``grad_state``). ``wait_limit_us`` and ``test_stall_producer`` as in the
    forward call.
    """
    for name, x in (("q", q), ("k", k), ("v", v), ("grad_o", grad_o)):
        if x is not None:
            _check_seq(x, name, None if x is q else q)
    scale = _scale(scale)
    lib = load_library()
    B, H, T, d = q.shape
    dev = q.device
    with _on(dev, stream):
        log_decay = _check_f32(log_decay, (H,), dev, "log_decay")
        S0 = _check_f32(state, (B, H, d, d), dev, "state")
        dS_T = _check_f32(grad_state, (B, H, d, d), dev, "grad_state")
        lengths = _check_index(lengths, B, dev, "lengths")
        if grad_o is None:
            grad_o = torch.zeros((B, H, T, d), dtype=q.dtype, device=dev)
        if out is None:
            grads = [torch.empty((B, H, T, d), dtype=q.dtype, device=dev) for _ in range(3)]
            dS0 = torch.empty((B, H, d, d), dtype=torch.float32, device=dev)
        else:
            if len(out) != 4:
                raise ValueError("out must hold (dq, dk, dv, dS0)")
            *grads, dS0 = out
            for i, x in enumerate(grads):
                _check_out(x, (B, H, T, d), q.dtype, dev, f"out[{i}]", strided=True)
            _check_out(dS0, (B, H, d, d), torch.float32, dev, "out[3]")
        q, k, v, grad_o = (_seq_in(x) for x in (q, k, v, grad_o))
        nbytes = _decay_scratch(B, H, T, d, 1, dev.index)
        scratch = _call_buffer(dev, nbytes, False) if nbytes else None
        args = (_seq(q), _seq(k), _seq(v), _seq(grad_o), _DTYPES[q.dtype], B, H, T, d, _ptr(log_decay), scale,
                _ptr(lengths), _ptr(S0), _ptr(dS_T), *(_seq(x) for x in grads), _ptr(dS0), _ptr(scratch), nbytes,
                _ptr(_workspace(dev)), _handle(dev, stream))
        if wait_limit_us or test_stall_producer:
            st = lib.vla_decay_backward_ex(*args, _wait_options(wait_limit_us, test_stall_producer))
        else:
            st = lib.vla_decay_backward(*args)
    _done(st, "vla_decay_backward", dev, stream, check)
    return tuple(grads), dS0


def vla_decay_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, state: torch.Tensor,
                   scale: float = 1.0, *, slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None, check: bool = False) -> torch.Tensor:
    """One token of vla_decay_forward's recurrence for a batch of sequences.

    q, k, v [B, H, d] (copied unless contiguous); ``state`` [N, H, d, d]
    float32, contiguous, is updated in place; ``slots`` [B] int32 (on the
    device) names each sequence's entry of it (None: entry b). A negative slot
    is an idle row, whose o is zero; one that is out of range or was used by an
    earlier row is left alone too and recorded (VLA_ERR_BAD_SLOT, raised by
    ``check=True``). Returns o like q.
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
        log_decay = _check_f32(log_decay, (H,), dev, "log_decay")
        slots = _check_index(slots, B, dev, "slots")
        if out is None:
            out = torch.empty((B, H, d), dtype=q.dtype, device=dev)
        else:
            _check_out(out, (B, H, d), q.dtype, dev, "out")
        q, k, v = (x if x.is_contiguous() and x.data_ptr() % 16 == 0
                   else x.clone(memory_format=torch.contiguous_format) for x in (q, k, v))
        st = lib.vla_decay_step(_ptr(q), _ptr(k), _ptr(v), _DTYPES[q.dtype], B, H, d, _ptr(log_decay), scale,
                                _ptr(state), N, _ptr(slots), _ptr(out), _ptr(_workspace(dev)),
                                _handle(dev, stream))
    _done(st, "vla_decay_step", dev, stream, check)
    return out


def _norm_weight(w, H, d, dev, name):
    if w is None:
        return None
    if tuple(w.shape) not in ((H, d), (d,)):
        raise ValueError(f"{name} must be ({H}, {d}) or ({d},), got {tuple(w.shape)}")
    return _check_f32(w, w.shape, dev, name)


def vla_head_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, *, out: Optional[torch.Tensor] = None, stream=None):
    """Layer norm of each row of a readout x [B, H, T, d] (vla_decay_forward's
    or vla_forward's o): (x - mean) rstd weight + bias.

    ``weight``, ``bias`` float32 [H, d], or [d] for all heads (None: 1 and 0).
    Returns ``(y, (mean, rstd))``: y like x, mean and rstd [B, H, T] float32
    for vla_head_norm_backward. ``out`` may be y's rows in any order, such as
    ``torch.empty(B, T, H, d).transpose(1, 2)``, or x itself.
    """
    _check_seq(x, "x")
    eps = float(eps)
    if not 0 <= eps < 3.4e38:
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    lib = load_library()
    B, H, T, d = x.shape
    dev = x.device
    if weight is not None and bias is not None and weight.shape != bias.shape:
        raise ValueError("weight and bias must have the same shape")
    with _on(dev, stream):
        weight = _norm_weight(weight, H, d, dev, "weight")
        bias = _norm_weight(bias, H, d, dev, "bias")
        shared = next((w.dim() == 1 for w in (weight, bias) if w is not None), False)
        if out is None:
            out = torch.empty((B, H, T, d), dtype=x.dtype, device=dev)
        else:
            _check_out(out, (B, H, T, d), x.dtype, dev, "out", strided=True)
        mean = torch.empty((B, H, T), dtype=torch.float32, device=dev)
        rstd = torch.empty((B, H, T), dtype=torch.float32, device=dev)
        x = _seq_in(x)
        st = lib.vla_head_norm(_seq(x), _DTYPES[x.dtype], B, H, T, d, _ptr(weight), _ptr(bias), int(shared), eps,
                               _seq(out), _ptr(mean), _ptr(rstd), _handle(dev, stream))
    _done(st, "vla_head_norm", dev, stream, False)
    return out, (mean, rstd)


def vla_head_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, stats, weight: Optional[torch.Tensor] = None, *,
                           out: Optional[torch.Tensor] = None, stream=None):
    """Gradient of a scalar loss through vla_head_norm: ``(dx, dweight, dbias)``.

    ``grad_y`` = dL/dy and x [B, H, T, d], ``stats`` = (mean, rstd) as the
    forward call returned them. dx is like x; dweight and dbias are float32,
    shaped as ``weight`` ([H, d] for None). ``out``: preallocated dx.
    """
    _check_seq(x, "x")
    _check_seq(grad_y, "grad_y", x)
    lib = load_library()
    B, H, T, d = x.shape
    dev = x.device
    mean, rstd = stats
    with _on(dev, stream):
        weight = _norm_weight(weight, H, d, dev, "weight")
        mean = _check_f32(mean, (B, H, T), dev, "mean")
        rstd = _check_f32(rstd, (B, H, T), dev, "rstd")
        shared = weight is not None and weight.dim() == 1
        if out is None:
            out = torch.empty((B, H, T, d), dtype=x.dtype, device=dev)
        else:
            _check_out(out, (B, H, T, d), x.dtype, dev, "out", strided=True)
        dw, db = (torch.empty((d,) if shared else (H, d), dtype=torch.float32, device=dev) for _ in range(2))
        x, grad_y = _seq_in(x), _seq_in(grad_y)
        nbytes = int(lib.vla_head_norm_scratch_bytes(B, H, T, d))
        scratch = _call_buffer(dev, nbytes, False) if nbytes else None
        st = lib.vla_head_norm_backward(_seq(grad_y), _seq(x), _DTYPES[x.dtype], B, H, T, d, _ptr(weight), int(shared),
                                        _ptr(mean), _ptr(rstd), _seq(out), _ptr(dw), _ptr(db), _ptr(scratch), nbytes,
                                        _handle(dev, stream))
    _done(st, "vla_head_norm_backward", dev, stream, False)
    return out, dw, db


def vla_state_cache(num_slots: int, shape, bits: int = 8, device=None):
    """An empty cache of ``num_slots`` states of ``shape`` (say (H, d, d)) in
    ``bits`` (8 or 4) bits a value: ``(codes, scales)``, zero-filled, so that
    every slot reads as the zero state."""
    *lead, d = shape
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    if d not in _DIMS:
        raise ValueError(f"last dimension {d} is not one of {_DIMS}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    codes = (torch.zeros((num_slots, *lead, d), dtype=torch.int8, device=device) if bits == 8
             else torch.zeros((num_slots, *lead, d // 2), dtype=torch.uint8, device=device))
    return codes, torch.zeros((num_slots, *lead, d // _GROUP), dtype=torch.float32, device=device)


def _cache(codes, scales):
    """(bits, N, shape of a state) of a cache, checked."""
    if codes.dtype not in (torch.int8, torch.uint8) or codes.dim() < 2 or codes.device.type != "cuda":
        raise ValueError("codes must be an int8 (8 bits) or uint8 (4 bits) CUDA tensor [N, ..., d or d / 2]")
    bits = 8 if codes.dtype == torch.int8 else 4
    N, *lead, last = codes.shape
    d = last if bits == 8 else 2 * last
    if d not in _DIMS:
        raise ValueError(f"last dimension {d} is not one of {_DIMS}")
    for x, name in ((codes, "codes"), (scales, "scales")):
        if not x.is_contiguous() or x.data_ptr() % 16 != 0:
            raise ValueError(f"{name} must be contiguous and start on a 16-byte boundary")
    if scales.dtype != torch.float32 or tuple(scales.shape) != (N, *lead, d // _GROUP) or scales.device != codes.device:
        raise ValueError(f"scales must be float32 {(N, *lead, d // _GROUP)} on {codes.device}")
    return bits, N, (*lead, d)


def _check_count(B: int):
    if B > 65535:
        raise ValueError(f"{B} states in one call, more than 65,535")


def _rows(shape) -> int:
    n = 1
    for x in shape[:-1]:
        n *= int(x)
    return n


def vla_state_store(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, slots: Optional[torch.Tensor] = None,
                    *, stream=None, check: bool = False) -> None:
    """Write states x [B, ...] (float32: S, A or z^key of the recurrences) into
    ``slots`` ([B] int32 on the device; None: slot b) of a cache, each group of
    32 values of a row rounded to whole multiples of amax / 127 (8 bits) or
    amax / 7 (4 bits).

    A negative slot is skipped; one out of range or used before in the call is
    skipped and recorded (VLA_ERR_BAD_SLOT), as is a group with a NaN or Inf,
    which reads back as NaN (VLA_ERR_NONFINITE). ``check=True`` raises. At
    most 65,535 states a call.
    """
    bits, N, shape = _cache(codes, scales)
    lib = load_library()
    dev = codes.device
    if x.dim() < 2:
        raise ValueError("x must be [B, ...]")
    B = x.shape[0]
    if slots is None and B > N:
        raise ValueError(f"{B} states for {N} slots")
    _check_count(B)
    with _on(dev, stream):
        x = _check_f32(x, (B, *shape), dev, "x")
        slots = _check_index(slots, B, dev, "slots")
        st = lib.vla_state_store(_ptr(x), B, _rows(shape), shape[-1], bits, _ptr(codes), _ptr(scales), N, _ptr(slots),
                                 _ptr(_workspace(dev)), _handle(dev, stream))
    _done(st, "vla_state_store", dev, stream, check)


def vla_state_load(codes: torch.Tensor, scales: torch.Tensor, slots: Optional[torch.Tensor] = None, *,
                   out: Optional[torch.Tensor] = None, stream=None, check: bool = False) -> torch.Tensor:
    """Read the states in ``slots`` ([B] int32 on the device, repeats allowed;
    None: all of them) of a cache: float32 [B, ...], ready to be carried on.

    A negative slot reads as zero, and so does one out of range, which is
    recorded (VLA_ERR_BAD_SLOT). ``out``: preallocated result. At most 65,535
    states a call.
    """
    bits, N, shape = _cache(codes, scales)
    lib = load_library()
    dev = codes.device
    if slots is not None and slots.dim() != 1:
        raise ValueError("slots must be [B]")
    B = N if slots is None else slots.shape[0]
    _check_count(B)
    with _on(dev, stream):
        slots = _check_index(slots, B, dev, "slots")
        if out is None:
            out = torch.empty((B, *shape), dtype=torch.float32, device=dev)
        else:
            _check_out(out, (B, *shape), torch.float32, dev, "out")
        st = lib.vla_state_load(_ptr(codes), _ptr(scales), N, _ptr(slots), B, _rows(shape), shape[-1], bits, _ptr(out),
                                _ptr(_workspace(dev)), _handle(dev, stream))
    _done(st, "vla_state_load", dev, stream, check)
    return out
