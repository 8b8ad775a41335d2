"""Refusals of the gated delta rule and of the norm and rotation of queries and
keys, before any CUDA work, and of their binding, without a GPU."""
import ctypes

import pytest
import torch

import sherman_morrison_memory_gb300 as vla
from sherman_morrison_memory_gb300 import _binding

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
B, H, T, D = 2, 2, 32, 64


def fake(i):
    """Addresses that are never read (every call here is refused first), far apart from each other."""
    return 0x100000000 * (i + 1)


@pytest.fixture(scope="module")
def lib():
    import os

    from sherman_morrison_memory_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    return _binding.load_library()


def seq(ptr, sb=H * T * D, sh=T * D, st=D):
    return ctypes.byref(_binding._Seq(ptr, sb, sh, st))


def gate(ptr, sb=H * T, sh=T, st=1):
    return ctypes.byref(_binding._Seq(ptr, sb, sh, st))


def pick(x, i, make):
    return make(fake(i)) if x == "s" else x


def forward(lib, q="s", k="s", v="s", o="s", g="s", beta="s", dtype=1, B=B, H=H, T=T, d=D, scale=1.0, n=None, S0=None,
            S=fake(9), status=None):
    return lib.vla_delta_forward(pick(q, 0, seq), pick(k, 1, seq), pick(v, 2, seq), dtype, B, H, T, d, pick(g, 3, gate),
                                 pick(beta, 4, gate), scale, P(n), P(S0), pick(o, 5, seq), P(S), P(status), None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(dtype=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(S=None), dict(S=fake(9) + 4),
    dict(S0=fake(8) + 8), dict(n=fake(8) + 1), dict(status=fake(8) + 4), dict(q=None), dict(o=None), dict(beta=None),
    dict(q=seq(None)), dict(k=seq(fake(1) + 8)), dict(v=seq(fake(2), st=60)), dict(q=seq(fake(0), st=0)), dict(o=seq(fake(5), sh=-64)),
    dict(beta=gate(None)), dict(beta=gate(fake(4) + 2)), dict(g=gate(fake(3), st=-1)), dict(g=gate(None)),
    dict(beta=gate(fake(4), sb=1 << 41)), dict(B=1 << 20, H=1 << 20)])
def test_forward_refuses(lib, bad):
    assert forward(lib, **bad) == INVALID


def test_forward_refuses_outputs_on_top(lib):
    for i, name in ((0, "q"), (1, "k"), (2, "v")):
        assert forward(lib, o=seq(fake(i) + 1024)) == INVALID, name
    assert forward(lib, o=seq(fake(3))) == INVALID and forward(lib, o=seq(fake(4) + 256)) == INVALID
    assert forward(lib, S=fake(0)) == INVALID and forward(lib, S=fake(5)) == INVALID
    assert forward(lib, S=fake(9), S0=fake(9) + 64) == INVALID and forward(lib, o=seq(fake(5), sb=64)) == INVALID
    # a gate of stride 0 is the one value that it is
    assert forward(lib, g=gate(fake(5) + 16, 0, 0, 0)) == INVALID


def test_other_dims_and_empty(lib):
    for d in (0, 16, 48, 100, 256):
        assert forward(lib, d=d) == UNSUPPORTED
        assert lib.vla_delta_scratch_bytes(1, 1, 1, 100, d) == 0
    assert forward(lib, B=0) == OK and forward(lib, H=0, S=None) == OK


def test_scratch(lib):
    """E, two states a block of 64 tokens (32 in fp32) and one more, the rows' shares of the gates' gradients."""
    for dtype, span in ((0, 32), (1, 64)):
        for b, h, t, d in ((1, 1, 1, 32), (2, 3, 64, 96), (1, 4, 65, 128)):
            blocks = -(-t // span)
            parts = [b * h * t * d] + [b * h * (blocks + 1) * d * d] * 2 + [b * h * (d // 16) * t] * 3
            assert lib.vla_delta_scratch_bytes(dtype, b, h, t, d) == sum(-(-4 * n // 256) * 256 for n in parts)
    assert lib.vla_delta_scratch_bytes(1, 1, 1, 0, 64) == 0 and lib.vla_delta_scratch_bytes(2, 1, 1, 8, 64) == 0


def backward(lib, do="s", dq="s", dk="s", dv="s", dg="s", db="s", g="s", S0=None, dS=None, dS0=None, d=D, dtype=1, scratch=fake(20), nb=None):
    nb = lib.vla_delta_scratch_bytes(dtype, B, H, T, d) if nb is None else nb
    return lib.vla_delta_backward(seq(fake(0)), seq(fake(1)), seq(fake(2)), pick(do, 3, seq), dtype, B, H, T, d, pick(g, 4, gate),
                                  gate(fake(5)), 1.0, None, P(S0), P(dS), pick(dq, 6, seq), pick(dk, 7, seq), pick(dv, 8, seq),
                                  pick(dg, 9, gate), pick(db, 10, gate), P(dS0), P(scratch), nb, None, None)


def test_backward_refuses(lib):
    need = lib.vla_delta_scratch_bytes(1, B, H, T, D)
    for bad in (dict(do=None), dict(dq=seq(fake(6) + 2)), dict(dtype=-1, nb=0), dict(dS0=fake(11), S0=fake(11)), dict(dS0=fake(11), dS=fake(11)),
                dict(dS=fake(11) + 4), dict(scratch=None), dict(nb=need - 1), dict(scratch=fake(20) + 16), dict(db=None),
                dict(dg=gate(fake(9), 0, 0, 0)), dict(db=gate(fake(10), st=0)), dict(dg=gate(None)),
                # on top of an input, another output or the scratch
                dict(dq=seq(fake(0))), dict(dk=seq(fake(6))), dict(dv=seq(fake(3))), dict(dg=gate(fake(4))), dict(db=gate(fake(9))),
                dict(dS0=fake(6)), dict(scratch=fake(2)), dict(dv=seq(fake(20) + 512))):
        assert backward(lib, **bad) == INVALID, bad
    assert backward(lib, d=80, nb=0) == UNSUPPORTED


def test_step_refuses(lib):
    def call(q=fake(0), states=fake(5), B=2, H=2, d=64, N=4, slots=None, o=fake(6), scale=1.0, dtype=0, g=fake(3), beta=fake(4)):
        return lib.vla_delta_step(P(q), P(fake(1)), P(fake(2)), dtype, B, H, d, P(g), P(beta), scale, P(states), N, P(slots), P(o),
                                  None, None)
    for bad in (dict(q=None), dict(q=fake(0) + 4), dict(states=None), dict(N=1), dict(N=-1), dict(slots=fake(7) + 2),
                dict(scale=float("inf")), dict(dtype=9), dict(beta=None), dict(beta=fake(4) + 1), dict(g=fake(3) + 2), dict(B=-3),
                dict(o=fake(0)), dict(o=fake(5) + 64), dict(states=fake(1)), dict(o=fake(4)), dict(slots=fake(6))):
        assert call(**bad) == INVALID, bad
    assert call(d=65) == UNSUPPORTED and call(B=0) == OK


def test_qk_norm_refuses(lib):
    def fwd(q="s", k="s", yq="s", yk="s", wq=None, wk=None, shared=0, unit=0, eps=1e-6, freqs=fake(4), rot=32, pos=None, sb=0, rq=fake(6),
            rk=fake(7), d=D, t=T, dtype=0):
        return lib.vla_qk_norm(pick(q, 0, seq), pick(k, 1, seq), dtype, B, H, t, d, P(wq), P(wk), shared, unit, eps, P(freqs), rot, P(pos),
                               sb, pick(yq, 2, seq), pick(yk, 3, seq), P(rq), P(rk), None)
    for bad in (dict(q=None), dict(yk=seq(fake(3) + 4)), dict(wq=fake(8) + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(rot=8), dict(rot=-16), dict(rot=80), dict(freqs=None), dict(freqs=fake(4) + 4), dict(pos=fake(5) + 2),
                dict(pos=fake(5), sb=-1), dict(rq=fake(6) + 1), dict(dtype=3), dict(t=-1),
                # on top of another's rows, partly on top of its own, statistics on rows, rows on what is read
                dict(yq=seq(fake(1))), dict(yk=seq(fake(0))), dict(yq=seq(fake(0) + 16)), dict(yk=seq(fake(2) + 64)), dict(rq=fake(0)),
                dict(rk=fake(6)), dict(rq=fake(3)), dict(yq=seq(fake(4))), dict(pos=fake(2) + 128, sb=T), dict(wk=fake(3) + 64)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(d=33) == UNSUPPORTED and fwd(t=0) == OK

    def bwd(dq="s", dk="s", dwq=None, dwk=None, scratch=None, nb=0, rq=fake(6), rot=32, d=D):
        return lib.vla_qk_norm_backward(seq(fake(0)), seq(fake(1)), seq(fake(2)), seq(fake(3)), 0, B, H, T, d, None, None, 0, 0, P(fake(4)), rot,
                                        None, 0, P(rq), P(fake(7)), pick(dq, 8, seq), pick(dk, 9, seq), P(dwq), P(dwk), P(scratch), nb, None)
    need = lib.vla_qk_norm_scratch_bytes(B, H, T, D)
    assert need > 0 and need % (2 * B * H * D * 4) == 0 and lib.vla_qk_norm_scratch_bytes(B, H, T, 63) == 0
    both = dict(dwq=fake(10), dwk=fake(11))
    for bad in (dict(dq=None), dict(rq=None), dict(dwq=fake(10)), dict(dwk=fake(11)), dict(**both), dict(rot=24),
                dict(scratch=fake(12), nb=need - 1, **both), dict(scratch=fake(12) + 4, nb=need, **both),
                dict(dq=seq(fake(1))), dict(dq=seq(fake(3))), dict(dk=seq(fake(0))), dict(dk=seq(fake(8))), dict(dq=seq(fake(6))),
                dict(scratch=fake(2), nb=need, **both), dict(scratch=fake(12), nb=need, dwq=fake(10), dwk=fake(10) + 64)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(d=31) == UNSUPPORTED


def test_binding_refuses():
    x, g = torch.zeros(1, 2, 3, 64), torch.zeros(1, 2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_delta_forward(x, x, x, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_delta_backward(x, x, x, g, g, 1.0, None, x)
    with pytest.raises(ValueError):
        vla.vla_delta_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g[..., 0], g[..., 0], torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError, match="bfloat16"):
        vla.vla_delta_forward(x.half(), x.half(), x.half(), g, g)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_qk_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        vla.vla_qk_norm_backward(x, x, x, x, (g, g))
    for rot in (0, 8, -16, 24):
        with pytest.raises(ValueError):
            vla.vla_rotation_frequencies(rot, device="cpu")
    f = vla.vla_rotation_frequencies(32, 100.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (16,) and float(f[0]) == 1.0 and abs(float(f[8]) - 0.1) < 1e-15
