"""Calls at the edges of include/vla_layer.h's contract that are refused before any CUDA work, and host helpers."""
import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest

from sherman_morrison_memory_gb300 import _binding, build

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
MB = 1 << 20


def fake(i):
    """Addresses far apart, never read: every call here is refused first."""
    return (i + 1) << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(build.LIB):
        build.build()
    return _binding.load_library()


# ---- arrays on top of each other ----------------------------------------------------------------------------------

B, H, T, D = 2, 3, 40, 64


def seq(ptr, rows="heads", extra=0):
    sb, sh, st = (H * T * D, T * D, D) if rows == "heads" else (T * H * D + extra, D, H * D)
    return ctypes.byref(_binding._Seq(ptr, sb, sh, st))


def forward(lib, q=fake(0), k=fake(1), v=fake(2), o=fake(3), S0=fake(4), S=fake(5), g=fake(6), n=None, dtype=0, T_=T,
            o_seq=None):
    return lib.vla_decay_forward(seq(q), seq(k), seq(v), dtype, B, H, T_, D, P(g), 1.0, P(n), P(S0), o_seq or seq(o), P(S),
                                 None, 0, None, None)


@pytest.mark.parametrize("dtype", [0, 1])
def test_forward_refuses_outputs_on_top(lib, dtype):
    rows, es = B * H * T * D, (4, 2)[dtype]
    for x in (0, 1, 2):
        for off in (0, 16, es * (rows - D), es * (D - rows)):
            assert forward(lib, o=fake(x) + off, dtype=dtype) == INVALID
    assert forward(lib, o=fake(5), dtype=dtype) == INVALID and forward(lib, o=fake(4) + 1024, dtype=dtype) == INVALID
    assert forward(lib, S=fake(4) + 16, dtype=dtype) == INVALID and forward(lib, S=fake(1), dtype=dtype) == INVALID
    assert forward(lib, S=fake(4) + 16, dtype=dtype, T_=0) == INVALID
    assert forward(lib, g=fake(5) + 64, dtype=dtype) == INVALID and forward(lib, n=fake(3) + 64, dtype=dtype) == INVALID
    # the same memory in another order, and rows of o on top of each other
    assert forward(lib, o_seq=seq(fake(0), "tokens"), dtype=dtype) == INVALID
    for st in ((H * T * D, T * D, D - 8), (H * T * D, T * D - D, D), (T * D, T * D, D), (8, T * D, D)):
        assert forward(lib, o_seq=ctypes.byref(_binding._Seq(fake(3), *st)), dtype=dtype) == INVALID


def test_backward_refuses_outputs_on_top(lib):
    def call(dq=fake(8), dk=fake(9), dv=fake(10), S0=fake(4), dS=fake(5), dS0=fake(7), T_=T):
        return lib.vla_decay_backward(seq(fake(0)), seq(fake(1)), seq(fake(2)), seq(fake(3)), 0, B, H, T_, D, P(fake(6)),
                                      1.0, None, P(S0), P(dS), seq(dq), seq(dk), seq(dv), P(dS0), None, 0, None, None)
    for x in (0, 1, 2, 3, 4, 5):
        for name in ("dq", "dk", "dv", "dS0"):
            assert call(**{name: fake(x)}) == INVALID and call(**{name: fake(x) + 4096}) == INVALID
    assert call(dq=fake(9)) == INVALID and call(dk=fake(10) + 16) == INVALID and call(dv=fake(7)) == INVALID
    assert call(dS0=fake(4) + 16, T_=0) == INVALID and call(dS0=fake(5) - 16, T_=0) == INVALID


def test_step_refuses_outputs_on_top(lib):
    N = 7

    def call(o=fake(3), states=fake(4), q=fake(0), slots=None, dtype=0):
        return lib.vla_decay_step(P(q), P(fake(1)), P(fake(2)), dtype, B, H, D, P(fake(5)), 1.0, P(states), N, P(slots),
                                  P(o), None, None)
    for dtype in (0, 1):
        for x in (0, 1, 2, 5):
            assert call(o=fake(x), dtype=dtype) == INVALID
        assert call(o=fake(0) + (4, 2)[dtype] * (B * H * D - 8), dtype=dtype) == INVALID
        assert call(o=fake(4) + 4 * N * H * D * D - 64, dtype=dtype) == INVALID
        assert call(q=fake(4) + 4 * N * H * D * D - 64, dtype=dtype) == INVALID
        assert call(slots=fake(3) + 16, dtype=dtype) == INVALID


def test_norm_refuses_outputs_on_top(lib):
    def fwd(y=fake(1), mean=fake(2), rstd=fake(3), w=fake(4), rows="heads"):
        return lib.vla_head_norm(seq(fake(0)), 0, B, H, T, D, P(w), None, 0, 1e-5, seq(y, rows), P(mean), P(rstd), None)
    # in place only as the same rows
    assert fwd(y=fake(0), rows="tokens") == INVALID and fwd(y=fake(0) + 4 * D) == INVALID
    assert fwd(mean=fake(3)) == INVALID and fwd(mean=fake(0)) == INVALID and fwd(rstd=fake(1) + 64) == INVALID
    assert fwd(w=fake(1)) == INVALID

    def bwd(dx=fake(2), dw=fake(3), db=fake(4), mean=fake(5), rstd=fake(6), scratch=fake(7), rows="heads"):
        return lib.vla_head_norm_backward(seq(fake(0)), seq(fake(1)), 0, B, H, T, D, None, 0, P(mean), P(rstd), seq(dx, rows),
                                          P(dw), P(db), P(scratch), MB, None)
    assert bwd(dx=fake(0), rows="tokens") == INVALID and bwd(dx=fake(1) - 4 * D) == INVALID
    assert bwd(dw=fake(4)) == INVALID and bwd(dw=fake(0)) == INVALID and bwd(db=fake(2)) == INVALID
    assert bwd(mean=fake(2)) == INVALID and bwd(scratch=fake(6)) == INVALID and bwd(scratch=fake(1)) == INVALID


def test_state_cache_refuses_outputs_on_top(lib):
    N, rows = 5, 96

    def store(x=fake(0), codes=fake(1), scales=fake(2), slots=None, bits=8):
        return lib.vla_state_store(P(x), B, rows, D, bits, P(codes), P(scales), N, P(slots), None, None)

    def load(x=fake(0), codes=fake(1), scales=fake(2), slots=None, bits=8):
        return lib.vla_state_load(P(codes), P(scales), N, P(slots), B, rows, D, bits, P(x), None, None)
    for bits in (8, 4):
        for f in (store, load):
            assert f(x=fake(1), bits=bits) == INVALID and f(x=fake(2), bits=bits) == INVALID
            assert f(x=fake(1) + N * rows * D * bits // 8 - 16, bits=bits) == INVALID
        assert store(scales=fake(1) + 64, bits=bits) == INVALID
        assert store(slots=fake(1) + 64, bits=bits) == INVALID and load(slots=fake(0) + 64, bits=bits) == INVALID


SHIM = r"""
#include "vla_overlap.h"
using namespace vla_layer;
extern "C" int overlap_of(const long long* a, const long long* b) {
    auto r = [](const long long* v) {
        return Region{(uintptr_t)v[0], v[1], {v[2], v[3], v[4]}, {(int)v[5], (int)v[6], (int)v[7]}};
    };
    return (overlap(r(a), r(b)) ? 1 : 0) | (overlaps_itself(r(a)) ? 2 : 0);
}
"""


@pytest.fixture(scope="module")
def overlap_of(tmp_path_factory):
    cxx = shutil.which("g++") or pytest.skip("no g++")
    where = tmp_path_factory.mktemp("overlap")
    src, out = where / "shim.cpp", where / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o", str(out)], check=True)
    fn = ctypes.CDLL(str(out)).overlap_of
    return lambda a, b: fn((ctypes.c_longlong * 8)(*a), (ctypes.c_longlong * 8)(*b))


def bytes_of(r):
    """Every row's bytes, one list a row."""
    p, row, s0, s1, s2, n0, n1, n2 = r
    return [range(p + i * s0 + j * s1 + k * s2, p + i * s0 + j * s1 + k * s2 + row)
            for i, j, k in itertools.product(range(n0), range(n1), range(n2))]


def test_overlap_against_all_bytes(overlap_of):
    """Strides in any order, nested or not, interleaved arrays: as the sets of bytes have it."""
    rng = random.Random(0)
    seen = {0: 0, 1: 0, 2: 0, 3: 0}
    for _ in range(6000):
        row = rng.choice([4, 8])
        if rng.random() < 0.5:  # slices of one buffer, in one of its orders
            n = [rng.randint(1, 4) for _ in range(3)]
            wide = row * rng.randint(1, 3)
            order = rng.sample(range(3), 3)
            st, at = [0, 0, 0], wide
            for i in order:
                st[i] = at
                at *= n[i]
            a = (1000 + rng.randrange(0, wide, 4), row, *st, *n)
            b = (1000 + rng.randrange(0, wide, 4), row, *(st if rng.random() < 0.7 else rng.sample(st, 3)), *n)
        else:
            a, b = ((1000 + 4 * rng.randint(0, 60), row, *(4 * rng.randint(1, 24) for _ in range(3)),
                     *(rng.randint(1, 4) for _ in range(3))) for _ in range(2))
        x, y = bytes_of(a), bytes_of(b)
        flat = [c for r in x for c in r]
        want = (1 if set(flat) & {c for r in y for c in r} else 0) | (2 if len(set(flat)) < len(flat) else 0)
        assert overlap_of(a, b) == want, (a, b)
        seen[want] += 1
    assert min(seen.values()) > 100


def test_overlap_at_real_sizes(overlap_of):
    """dq, dk and dv as slices of one [B, T, 3, H, d] buffer, larger than 2^31 bytes; the same buffer in other orders."""
    b, t, h, row = 16, 65537, 32, 256
    st = (t * 3 * h * row, row, 3 * h * row)
    one = lambda i, st=st: (1 << 40) + i * h * row  # noqa: E731
    for i, j in itertools.product(range(3), range(3)):
        assert overlap_of((one(i), row, *st, b, h, t), (one(j), row, *st, b, h, t)) == (1 if i == j else 0)
    assert overlap_of((one(0), row, *st, b, h, t), (one(0) + row - 16, row, *st, b, h, t)) == 1
    # [B, H, T, d] in one half of the memory, [B, T, H, d] in the other
    heads, tokens = (h * t * row, t * row, row), (h * t * row, row, h * row)
    assert overlap_of((1 << 40, row, *heads, b, h, t), ((1 << 40) + b * h * t * row, row, *tokens, b, h, t)) == 0
    assert overlap_of((1 << 40, row, *heads, b, h, t), (1 << 40, row, *tokens, b, h, t)) == 1
