"""Refusals of the operators in include/vla_layer.h, before any CUDA work, and
of their binding, without a GPU."""
import ctypes

import pytest
import torch

import sherman_morrison_memory_gb300 as vla
from sherman_morrison_memory_gb300 import _binding

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000  # 16-byte aligned, never read: every call here is refused first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import os

    from sherman_morrison_memory_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    return _binding.load_library()


def seq(ptr=FAKE, sb=4096, sh=2048, st=64):
    return ctypes.byref(_binding._Seq(ptr, sb, sh, st))


def forward(lib, q="s", k="s", v="s", o="s", dtype=1, B=2, H=2, T=32, d=64, g=FAKE, scale=1.0, n=None, S0=None, S=FAKE,
            scratch=None, nb=0, status=None):
    s = lambda x: seq() if x == "s" else x  # noqa: E731
    return lib.vla_decay_forward(s(q), s(k), s(v), dtype, B, H, T, d, P(g), scale, P(n), P(S0), s(o), P(S), P(scratch),
                                 nb, P(status), None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(dtype=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(g=None),
    dict(g=FAKE + 2), dict(S=None), dict(S=FAKE + 4), dict(S0=FAKE + 8), dict(n=FAKE + 1), dict(status=FAKE + 4),
    dict(q=None), dict(o=None), dict(q=seq(None)), dict(k=seq(FAKE + 8)), dict(v=seq(st=60)), dict(q=seq(st=0)),
    dict(o=seq(sh=-64)), dict(k=seq(sb=4)), dict(q=seq(sb=1 << 41)), dict(B=1 << 20, H=1 << 20)])
def test_decay_forward_refuses(lib, bad):
    assert forward(lib, **bad) == INVALID


def test_decay_refuses_other_dims_and_takes_empty(lib):
    for d in (0, 16, 48, 100, 256):
        assert forward(lib, d=d) == UNSUPPORTED
        assert lib.vla_decay_scratch_bytes(1, 1, 4096, d, 0) == 0
    assert forward(lib, B=0) == OK and forward(lib, H=0, S=None) == OK


def test_decay_scratch(lib):
    """Few heads of long sequences are cut into segments, whose states are the scratch."""
    need = lib.vla_decay_scratch_bytes(1, 2, 65536, 64, 0)
    assert need > 0 and need % (2 * 64 * 64 * 4) == 0
    # heads that fill whole waves of blocks are not cut, a few more than that are
    assert lib.vla_decay_scratch_bytes(2, 152, 65536, 64, 0) == 0
    few = lib.vla_decay_scratch_bytes(1, 160, 65536, 64, 0)
    assert few > 0 and few % (8 * 64 * 64 * 4) == 0
    assert lib.vla_decay_scratch_bytes(1, 2, 64, 64, 0) == 0 and lib.vla_decay_scratch_bytes(1, 2, -1, 64, 0) == 0
    big = dict(B=1, H=2, T=65536)
    assert forward(lib, **big) == INVALID
    assert forward(lib, scratch=FAKE, nb=need - 1, **big) == INVALID
    assert forward(lib, scratch=FAKE + 16, nb=need, **big) == INVALID


def test_decay_backward_refuses(lib):
    def call(do="s", dq="s", S0=None, dS=None, dS0=None, d=64, dtype=1):
        s = lambda x: seq() if x == "s" else x  # noqa: E731
        return lib.vla_decay_backward(seq(), seq(), seq(), s(do), dtype, 2, 2, 32, d, P(FAKE), 1.0, None, P(S0), P(dS),
                                      s(dq), seq(), seq(), P(dS0), None, 0, None, None)
    assert call(do=None) == INVALID and call(dq=seq(FAKE + 2)) == INVALID and call(dtype=-1) == INVALID
    assert call(dS0=FAKE, S0=FAKE) == INVALID and call(dS0=FAKE, dS=FAKE) == INVALID
    assert call(dS=FAKE + 4) == INVALID and call(d=80) == UNSUPPORTED


def test_step_refuses(lib):
    def call(q=FAKE, states=FAKE, B=2, H=2, d=64, N=4, slots=None, o=FAKE, scale=1.0, dtype=0, g=FAKE):
        return lib.vla_decay_step(P(q), P(FAKE), P(FAKE), dtype, B, H, d, P(g), scale, P(states), N, P(slots), P(o), None,
                                  None)
    assert call(q=None) == INVALID and call(q=FAKE + 4) == INVALID and call(states=None) == INVALID
    assert call(N=1) == INVALID and call(N=-1) == INVALID and call(slots=FAKE + 2) == INVALID
    assert call(scale=float("inf")) == INVALID and call(dtype=9) == INVALID and call(g=None) == INVALID
    assert call(d=65) == UNSUPPORTED and call(B=0) == OK and call(B=-3) == INVALID


def test_norm_refuses(lib):
    def fwd(x="s", y="s", w=None, eps=1e-5, d=64, T=32, dtype=0, mean=None):
        s = lambda a: seq() if a == "s" else a  # noqa: E731
        return lib.vla_head_norm(s(x), dtype, 2, 2, T, d, P(w), None, 0, eps, s(y), P(mean), None, None)
    assert fwd(x=None) == INVALID and fwd(y=seq(FAKE + 4)) == INVALID and fwd(w=FAKE + 4) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(eps=float("inf")) == INVALID
    assert fwd(mean=FAKE + 1) == INVALID and fwd(d=33) == UNSUPPORTED and fwd(T=0) == OK and fwd(T=-1) == INVALID

    def bwd(dw=None, db=None, scratch=None, nb=0, mean=FAKE, rstd=FAKE, d=64):
        return lib.vla_head_norm_backward(seq(), seq(), 0, 2, 2, 32, d, None, 0, P(mean), P(rstd), seq(), P(dw), P(db),
                                          P(scratch), nb, None)
    need = lib.vla_head_norm_scratch_bytes(2, 2, 32, 64)
    assert need > 0 and lib.vla_head_norm_scratch_bytes(2, 2, 32, 63) == 0
    assert bwd(dw=FAKE) == INVALID and bwd(db=FAKE) == INVALID and bwd(mean=None) == INVALID and bwd(rstd=None) == INVALID
    assert bwd(dw=FAKE, db=FAKE) == INVALID and bwd(dw=FAKE, db=FAKE, scratch=FAKE, nb=need - 1) == INVALID
    assert bwd(d=31) == UNSUPPORTED


def test_state_cache_refuses(lib):
    def store(x=FAKE, B=2, rows=64, d=64, bits=8, codes=FAKE, scales=FAKE, N=4, slots=None):
        return lib.vla_state_store(P(x), B, rows, d, bits, P(codes), P(scales), N, P(slots), None, None)

    def load(x=FAKE, B=2, rows=64, d=64, bits=8, codes=FAKE, scales=FAKE, N=4, slots=None):
        return lib.vla_state_load(P(codes), P(scales), N, P(slots), B, rows, d, bits, P(x), None, None)
    for f in (store, load):
        assert f(x=None) == INVALID and f(x=FAKE + 4) == INVALID and f(codes=None) == INVALID
        assert f(codes=FAKE + 8) == INVALID and f(scales=None) == INVALID and f(scales=FAKE + 2) == INVALID
        assert f(bits=2) == INVALID and f(B=-1) == INVALID and f(N=1) == INVALID and f(slots=FAKE + 1) == INVALID
        assert f(rows=-1) == INVALID and f(rows=1 << 40) == INVALID and f(B=65536, N=70000) == INVALID
        assert f(d=16) == UNSUPPORTED and f(B=0) == OK and f(rows=0) == OK


def test_status_string(lib):
    assert "slot" in vla.vla_status_string(_binding.VLA_ERR_BAD_SLOT)


def test_binding_refuses():
    """What the binding refuses by itself: host tensors, other types and shapes."""
    x = torch.zeros(1, 2, 3, 64)
    g = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_decay_forward(x, x, x, g)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_decay_backward(x, x, x, g, 1.0, None, x)
    with pytest.raises(ValueError):
        vla.vla_decay_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_head_norm(x)
    with pytest.raises(ValueError, match="bfloat16"):
        vla.vla_decay_forward(x.half(), x.half(), x.half(), g)
    with pytest.raises(ValueError):
        vla.vla_state_store(torch.zeros(1, 2, 64), torch.zeros(1, 2, 64, dtype=torch.int8), torch.zeros(1, 2, 2))
    for bad in (dict(bits=3), dict(shape=(2, 48))):
        with pytest.raises(ValueError):
            vla.vla_state_cache(**{"num_slots": 2, "shape": (2, 64), "bits": 8, "device": "cpu", **bad})
    codes, scales = vla.vla_state_cache(3, (2, 64), 4, device="cpu")
    assert codes.shape == (3, 2, 32) and scales.shape == (3, 2, 2)
