"""Norm and rotation of queries and keys on the GPU against their fp64 forms."""
import pytest
import torch

import delta_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import seqs

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def weights(kind, H, d, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(50 + seed)
    shape = {"none": None, "shared": (d,), "heads": (H, d)}[kind]
    return [None if shape is None else 1 + 0.3 * torch.randn(*shape, generator=gen, device="cuda") for _ in range(2)]


def check(q, k, gq, gk, w, unit, freqs, pos, eps=1e-6, got=None, back=None):
    B, H, T, d = q.shape
    (yq, yk), stats = got if got is not None else vla.vla_qk_norm(q, k, *w, eps, unit=unit, freqs=freqs, positions=pos)
    (dq, dk), dw = back if back is not None else vla.vla_qk_norm_backward(gq, gk, q, k, stats, *w, unit=unit, freqs=freqs, positions=pos)
    p = torch.arange(T)[None].expand(B, T) if pos is None else pos.cpu().expand(B, T)
    half = R.HALF[q.dtype] if q.dtype == BF else 0.0
    # rstd: d / 16 + 4 sums, its root and quotient (2 units); the weight, the turn's cosine, sine and sum
    u = (d // 16 + 4 + 2 + 8) * R.U
    # an angle is a product of two float64 values and a constant, each and here its own rounded by 2^-53 of it
    if freqs is not None:
        u = u + 4 * 2.0 ** -53 * (p.double().abs() * float(freqs.abs().max()))[:, None, :, None]
    most = u if isinstance(u, float) else float(u.max())
    for x, g, wt, y, s, dx, dwt in ((q, gq, w[0], yq, stats[0], dq, dw[0]), (k, gk, w[1], yk, stats[1], dk, dw[1])):
        assert y.dtype == dx.dtype == q.dtype
        x6 = x.detach().double().cpu().requires_grad_()
        w6 = None if wt is None else wt.double().cpu().requires_grad_()
        y6, r6 = R.qk(x6, w6, unit, eps, None if freqs is None else freqs.cpu(), p)
        (y6 * g.double().cpu()).sum().backward()
        row = lambda a: a.detach().norm(dim=-1, keepdim=True)  # noqa: E731
        assert bool(((y.double().cpu() - y6.detach()).abs() <= half * y6.detach().abs() + u * row(y6) + 1e-30).all())
        assert bool(((s.double().cpu() - r6.detach()).abs() <= most * r6.detach()).all())
        # dx is a difference of p and its share along n: both are at most |w dz| rstd
        size = r6.detach()[..., None] * row(g.double().cpu()) * (1.0 if wt is None else float(wt.abs().max()))
        assert bool(((dx.double().cpu() - x6.grad).abs() <= half * x6.grad.abs() + 4 * u * size + 1e-30).all())
        if wt is None:
            assert dwt is None
        else:
            n = row(y6) + (x6.detach() * r6.detach()[..., None]).abs()
            terms = (g.double().cpu().norm(dim=-1, keepdim=True) * n).sum((0, 1, 2) if wt.dim() == 1 else (0, 2))
            assert dwt.shape == wt.shape
            assert bool(((dwt.double().cpu() - w6.grad).abs() <= (2 * most + (16 + T // 16) * R.U) * terms).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1, 32), (2, 3, 5, 64), (1, 5, 67, 96), (2, 9, 33, 128), (1, 4, 20, 96), (3, 2, 300, 32)])
@pytest.mark.parametrize("kind", ["none", "shared", "heads"])
def test_norm_and_rotation(B, H, T, d, kind, dtype):
    q, k, gq, gk = seqs(4, B, H, T, d, dtype, seed=T + d)
    w = weights(kind, H, d)
    for rot in (0, 16, d // 2 // 16 * 16, d):
        for unit in (False, True):
            freqs = vla.vla_rotation_frequencies(rot) if rot else None
            check(q, k, gq, gk, w, unit, freqs, None)
    pos = torch.randint(-100, 1 << 20, (B, T), device="cuda", dtype=torch.int32)
    check(q, k, gq, gk, w, False, vla.vla_rotation_frequencies(d, 500.0), pos)
    check(q, k, gq, gk, w, False, vla.vla_rotation_frequencies(16), pos[0].contiguous())


@pytest.mark.parametrize("d", [32, 96, 128])
def test_far_positions(d):
    """The ends of the positions' range: angles lose nothing."""
    B, H, T = 1, 2, 6
    q, k, gq, gk = seqs(4, B, H, T, d, F32)
    pos = torch.tensor([[0, 1, -1, (1 << 31) - 1, -(1 << 31), 123456789]], dtype=torch.int32, device="cuda")
    check(q, k, gq, gk, (None, None), False, vla.vla_rotation_frequencies(d), pos)
    # frequencies of more than a turn a position, against time, and 0
    freqs = torch.tensor([7.0, -0.3, 0.0, 1e-9, 3.0, 100.0, -6.5, 0.7], dtype=torch.float64, device="cuda")
    check(q, k, gq, gk, (None, None), True, freqs, pos)
    # ... and hardly any, either way
    freqs = torch.tensor([-1e-20, 1e-20, -1e-17, -1e-12, 3e-12, -2.0 ** -40, -0.0, -1e-10], dtype=torch.float64, device="cuda")
    check(q, k, gq, gk, (None, None), True, freqs, pos)


def test_a_frequency_that_is_not_finite():
    q, k = seqs(2, 1, 1, 3, 64, F32)
    freqs = vla.vla_rotation_frequencies(32)
    freqs[2] = float("inf")
    (y, _), _ = vla.vla_qk_norm(q, k, freqs=freqs)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[2, 18]] = True
    assert torch.isnan(y[..., bad]).all() and torch.isfinite(y[..., ~bad]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 96])
def test_strides_and_in_place(d, dtype):
    """Slices of one projection's output, results in its order or on top of it."""
    B, H, T = 2, 3, 50
    proj = torch.randn(B, T, 3, H, d, device="cuda").to(dtype)
    q, k, v = (proj[:, :, i].transpose(1, 2) for i in range(3))
    gq, gk = seqs(2, B, H, T, d, dtype, seed=2, rows="tokens")
    w, freqs = weights("heads", H, d), vla.vla_rotation_frequencies(32)
    kw = dict(unit=True, freqs=freqs)
    want = vla.vla_qk_norm(q, k, *w, **kw)
    check(q, k, gq, gk, w, True, freqs, None, got=want)
    frame = torch.full((B, T + 2, 2, H, d), 5.0, dtype=dtype, device="cuda")
    outs = tuple(frame[:, 1:T + 1, i].transpose(1, 2) for i in range(2))
    (yq, yk), _ = vla.vla_qk_norm(q, k, *w, out=outs, **kw)
    assert yq is outs[0] and torch.equal(yq, want[0][0]) and torch.equal(yk, want[0][1])
    assert (frame[:, 0] == 5).all() and (frame[:, T + 1] == 5).all()
    back = vla.vla_qk_norm_backward(gq, gk, q, k, want[1], *w, **kw)
    g2 = [x.clone() for x in (gq, gk)]
    got = vla.vla_qk_norm_backward(*g2, q, k, want[1], *w, out=tuple(g2), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got[0] + got[1], back[0] + back[1]))
    keep = v.clone()
    x = proj.clone()
    q, k = (x[:, :, i].transpose(1, 2) for i in range(2))
    vla.vla_qk_norm(q, k, *w, out=(q, k), **kw)
    assert torch.equal(q, want[0][0]) and torch.equal(k, want[0][1]) and torch.equal(x[:, :, 2].transpose(1, 2), keep)
    odd = torch.randn(B, H, T, d + 3, device="cuda").to(dtype)[..., 3:]
    check(odd, odd, gq, gk, w, False, None, None)


def test_zero_rows_and_empty_sizes():
    z = torch.zeros(1, 2, 3, 64, device="cuda")
    (y, _), (r, _) = vla.vla_qk_norm(z, z, unit=True, eps=1e-6)
    assert (y == 0).all() and float((r - 1e3).abs().max()) <= 1e3 * 4 * R.U
    e = torch.empty(0, 2, 3, 64, device="cuda")
    w = torch.ones(2, 64, device="cuda")
    (y, _), stats = vla.vla_qk_norm(e, e, w, w)
    assert y.shape == e.shape
    (dq, _), (dw, dw2) = vla.vla_qk_norm_backward(e, e, e, e, stats, w, w)
    assert dq.shape == e.shape and (dw == 0).all() and (dw2 == 0).all() and dw.shape == w.shape


@pytest.mark.parametrize("kind", ["shared", "heads"])
def test_many_rows(kind):
    """Several tiles a block and several blocks a head, the same bits each time, in a graph and on another stream."""
    B, H, T, d = 2, 6, 9000, 96
    q, k, gq, gk = seqs(4, B, H, T, d, BF, seed=1)
    w, freqs = weights(kind, H, d), vla.vla_rotation_frequencies(96)

    def call(q, k, stream=None):
        y, stats = vla.vla_qk_norm(q, k, *w, freqs=freqs, stream=stream)
        g, dw = vla.vla_qk_norm_backward(gq, gk, q, k, stats, *w, freqs=freqs, stream=stream)
        return (*y, *stats, *g, *dw)

    want = call(q, k)
    check(q, k, gq, gk, w, False, freqs, None, got=(want[:2], want[2:4]), back=(want[4:6], want[6:]))
    torch.cuda.synchronize()
    got = call(q, k, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call(q2, k2)
    q2.copy_(q), k2.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, res))


def test_rows_far_apart():
    """Sequences more than 2^31 elements apart."""
    d, T, far = 64, 20, (1 << 31) + 4096
    buf = torch.empty(far + T * d, dtype=BF, device="cuda")
    x = buf.as_strided((2, 1, T, d), (far, T * d, d, 1))
    q, k, gq, gk = seqs(4, 2, 1, T, d, BF)
    x.copy_(k)
    check(q, x, gq, gk, (None, None), False, None, None)
    x.copy_(gk)
    check(q, k, gq, x, weights("heads", 1, d), True, vla.vla_rotation_frequencies(64), None)


def test_streams_and_graphs():
    """Calls on two streams at once give the same bits each time, and a captured pair of calls follows its inputs."""
    freqs = vla.vla_rotation_frequencies(64)

    def call(x, w):
        y, stats = vla.vla_qk_norm(x[0], x[1], *w, freqs=freqs)
        return *y, *stats, *(t for pair in vla.vla_qk_norm_backward(x[2], x[3], x[0], x[1], stats, *w, freqs=freqs) for t in pair)

    sets = [(seqs(4, 2, 6, 700, 64, BF, seed=s), weights(kind, 6, 64, s)) for s, kind in ((1, "heads"), (2, "shared"))]
    want = [call(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(call(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
    held = [x.clone() for x in sets[0][0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(held, sets[0][1])
    for s in (1, 0):
        for a, b in zip(held, sets[s][0]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call(sets[s][0], sets[0][1])))
