"""The gated delta rule on the GPU against its fp64 form (delta_ref.py): sizes at
the kernels' tile and block edges, carried states, padded batches, strides, gates
from none to total, streams and graphs."""
import pytest
import torch

import delta_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import seqs, state_like

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def unit(x):
    return (x.float() / x.float().norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(x.dtype)


def inputs(n, B, H, T, d, dtype, seed=0, rows="heads"):
    """q, k (unit rows), v and, of four, dO."""
    q, k, *rest = seqs(n, B, H, T, d, dtype, seed, rows)
    return [unit(q), unit(k), *rest]


def gates(B, H, T, seed=0):
    """Heads from hardly any decay to strong ones; a token that forgets all; beta from 0 to 1."""
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    rate = torch.exp2(torch.linspace(-9, 2, H, device="cuda"))[:, None]
    g = -rate * torch.rand(B, H, T, generator=gen, device="cuda")
    beta = torch.rand(B, H, T, generator=gen, device="cuda")
    if T > 2:
        g[:, :, T // 2] = float("-inf")
        beta[:, :, T // 3], beta[:, :, T // 3 + 1] = 0.0, 1.0
    return g, beta


def check_forward(q, k, v, g, beta, scale, state, lengths=None, got=None, more=1):
    B, H, T, d = q.shape
    o, S = got if got is not None else vla.vla_delta_forward(q, k, v, g, beta, scale, state, lengths=lengths, check=True)
    ro, rS, mag = R.delta(q, k, v, g, beta, scale, state, lengths)
    assert o.dtype == q.dtype and S.dtype == F32
    e = more * R.roundings(T, d) * R.U
    R.assert_normwise(S, rS, e, "S")
    if q.dtype == BF:
        R.assert_rounded(o, ro, mag, T, "o")
    else:
        R.assert_normwise(o, ro, e, "o")
    return o, S


def check_backward(q, k, v, g, beta, scale, state, do, dS, lengths=None, got=None, more=1):
    B, H, T, d = q.shape
    (dq, dk, dv), (dg, db), dS0 = got if got is not None else vla.vla_delta_backward(q, k, v, g, beta, scale, state, do, dS,
                                                                                     lengths=lengths, check=True)
    ref, (mq, mk, mb) = R.delta_grads(q, k, v, g, beta, scale, state, do, dS, lengths)
    e = 2 * more * R.roundings(T, d) * R.U  # through both recurrences
    for name, x, r, m in (("dq", dq, ref[0], mq), ("dk", dk, ref[1], mk), ("dv", dv, ref[2], 0 * mq)):
        assert x.dtype == q.dtype
        if q.dtype == BF:
            R.assert_rounded(x, r, m, T, name)
        else:
            R.assert_normwise(x, r, e, name)
    # dbeta is a scalar product of R k and e, each within e of its own size: (x + a) . (y + b) - x . y is at most
    # (|a| / |x| + |b| / |y|) |x| |y| to first order, however much of x . y cancels
    off = (db.double().cpu() - ref[4]).norm(dim=-1)
    assert torch.isfinite(db).all() and bool((off <= e * (ref[4].norm(dim=-1) + mb.norm(dim=-1)) + 1e-30).all()), ("dbeta", off, mb)
    R.assert_normwise(dS0, ref[5], e, "dS0")
    if g is None:
        assert dg is None
        return
    # a sum over the tokens of a block of o . dO - v . dV, which are larger than what is left of them
    o = R.delta(q, k, v, g, beta, scale, state, lengths)[0]
    live = torch.ones(B, 1, T) if lengths is None else (torch.arange(T)[None] < lengths.cpu()[:, None]).double()[:, None]
    terms = (((o * do.double().cpu()).nan_to_num(0, 0, 0).norm(dim=-1) + (v.double().cpu() * ref[2]).nan_to_num(0, 0, 0).norm(dim=-1)) * live).norm(dim=-1)
    off = (dg.double().cpu() - ref[3]).norm(dim=-1)
    assert torch.isfinite(dg).all() and bool((off <= e * (ref[3].norm(dim=-1) + 8 * terms) + 1e-30).all()), ("dg", off, terms)


SIZES = [(1, 1, 1, 32), (2, 3, 2, 64), (1, 4, 31, 96), (2, 2, 32, 128), (1, 3, 33, 32), (3, 1, 63, 64), (1, 5, 64, 96),
         (2, 4, 65, 128), (1, 2, 127, 64), (1, 4, 128, 32), (2, 3, 129, 96), (1, 4, 200, 128)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_forward(B, H, T, d, dtype):
    q, k, v = inputs(3, B, H, T, d, dtype, seed=T + d)
    g, beta = gates(B, H, T)
    check_forward(q, k, v, g, beta, 1.0, None)
    check_forward(q, k, v, g, beta, -0.3, state_like(B, H, d, 1))
    check_forward(q, k, v, None, beta, 0.5, state_like(B, H, d, 1))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_backward(B, H, T, d, dtype):
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=T + d + 1)
    g, beta = gates(B, H, T)
    check_backward(q, k, v, g, beta, 1.0, None, do, None)
    check_backward(q, k, v, g, beta, 0.4, state_like(B, H, d, 1), do, state_like(B, H, d, 2))
    check_backward(q, k, v, None, beta, 0.4, None, do, state_like(B, H, d, 2))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(513, 32), (777, 64), (1024, 96), (1153, 128)])
def test_longer_sequences(T, d, dtype):
    q, k, v, do = inputs(4, 1, 2, T, d, dtype, seed=T)
    g, beta = gates(1, 2, T)
    S0, dS = state_like(1, 2, d, 3), state_like(1, 2, d, 4)
    check_forward(q, k, v, g, beta, d ** -0.5, S0)
    check_backward(q, k, v, g, beta, d ** -0.5, S0, do, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d,lengths", [(70, 64, [70, 0, 1, 69]), (130, 128, [64, 65, 130, 129]), (33, 96, [32, 33, 5, 0]),
                                         (300, 32, [300, 0, 257, 63]), (200, 128, [1, 200, 96, -4])])
def test_padded_batches(T, d, lengths, dtype):
    """Rows behind a sequence's end hold NaN and Inf: nothing of them is seen, and their results are zero."""
    B, H = len(lengths), 2
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=d)
    g, beta = gates(B, H, T)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    clean = [x.clone() for x in (q, k, v, do, g, beta)]
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (do, float("-inf")), (g, float("nan")), (beta, float("inf"))):
        for b, m in enumerate(lengths):
            x[b, :, max(0, m):] = bad
    S0, dS = state_like(B, H, d, 5), state_like(B, H, d, 6)
    got = vla.vla_delta_forward(q, k, v, g, beta, 0.5, S0, lengths=n, check=True)
    check_forward(*clean[:3], *clean[4:], 0.5, S0, n, got)
    back = vla.vla_delta_backward(q, k, v, g, beta, 0.5, S0, do, dS, lengths=n, check=True)
    check_backward(*clean[:3], *clean[4:], 0.5, S0, clean[3], dS, n, back)
    for x in (got[0], *back[0], *back[1]):
        for b, m in enumerate(lengths):
            assert (x[b, :, max(0, m):] == 0).all()
    for b, m in enumerate(lengths):
        if m <= 0:
            assert torch.equal(got[1][b], S0[b]) and torch.equal(back[2][b], dS[b])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 96, 128])
def test_strides(d, dtype):
    """Token-order inputs, outputs and gates, slices of wider rows and of longer sequences, broadcast gates and keys."""
    B, H, T = 2, 3, 77
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=3, rows="tokens")
    q, k = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (q, k))
    g, beta = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in gates(B, H, T))
    out = torch.full((B, T, H, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
    S = torch.empty(B, H, d, d, device="cuda")
    o, _ = vla.vla_delta_forward(q, k, v, g, beta, 1.0, out=(out, S), check=True)
    assert o is out
    check_forward(q, k, v, g, beta, 1.0, None, None, (o, S))
    grads = [torch.full((B, T, H, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(3)]
    dgates = torch.full((B, T, 2, H + 2), 7.0, device="cuda")
    dg, db = (dgates[:, :, i, 1:H + 1].transpose(1, 2) for i in range(2))
    got = vla.vla_delta_backward(q, k, v, g, beta, 1.0, None, do, out=(*grads, dg, db, S), check=True)
    check_backward(q, k, v, g, beta, 1.0, None, do, None, None, got)
    assert (dgates[..., 0] == 7).all() and (dgates[..., H + 1] == 7).all()
    wide = torch.randn(B, H, T + 9, 2 * d + 16, device="cuda").to(dtype)
    v2, q2 = wide[:, :, 4:T + 4, 8:d + 8], wide[:, :, :T, d + 16:]
    odd = unit(torch.randn(B, H, T, d + 3, device="cuda").to(dtype)[..., 3:])
    before = wide.clone()
    flat = (torch.full((H, 1), -0.02, device="cuda").expand(B, H, T), torch.full((1,), 0.4, device="cuda").expand(B, H, T))
    check_forward(q2, odd, v2, *flat, 1.0, None)
    check_backward(q2, odd, v2, *flat, 1.0, None, do, None)
    assert torch.equal(before, wide)
    check_forward(q, k[:, :1].expand(B, H, T, d), v, g, beta, 1.0, None)


def test_padding_between_rows_is_left_alone():
    B, H, T, d = 2, 2, 70, 64
    q, k, v, do = inputs(4, B, H, T, d, BF, seed=8)
    g, beta = gates(B, H, T)
    frame = torch.full((B, H, T + 5, d + 16), 3.0, dtype=BF, device="cuda")
    grads = [frame.clone() for _ in range(3)]
    S = torch.empty(B, H, d, d, device="cuda")
    inner = lambda x: x[:, :, 2:T + 2, 8:d + 8]  # noqa: E731
    n = torch.tensor([70, 20], dtype=torch.int32, device="cuda")
    vla.vla_delta_forward(q, k, v, g, beta, lengths=n, out=(inner(frame), S))
    vla.vla_delta_backward(q, k, v, g, beta, 1.0, None, do, lengths=n,
                           out=(*map(inner, grads), torch.empty_like(g), torch.empty_like(g), S))
    torch.cuda.synchronize()
    for x in (frame, *grads):
        assert (inner(x) != 3.0).any()
        inner(x).fill_(3.0)
        assert (x == 3.0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_far_apart(dtype):
    """Sequences and gates more than 2^31 elements apart."""
    d, T = 64, 40
    far = (1 << 31) + 4096
    buf = torch.empty(far + T * d, dtype=dtype, device="cuda")
    x = buf.as_strided((2, 1, T, d), (far, T * d, d, 1))
    q, k, v, do = inputs(4, 2, 1, T, d, dtype)
    g, beta = gates(2, 1, T)
    x.copy_(k)
    check_forward(q, x, v, g, beta, 1.0, None)
    check_backward(q, x, v, g, beta, 1.0, None, do, None)
    x.zero_()
    S = torch.empty(2, 1, d, d, device="cuda")
    vla.vla_delta_forward(q, k, v, g, beta, out=(x, S), check=True)
    check_forward(q, k, v, g, beta, 1.0, None, None, (x, S))
    del buf, x
    wide = torch.empty(far + T, device="cuda")
    b2 = wide.as_strided((2, 1, T), (far, T, 1))
    b2.copy_(beta)
    check_forward(q, k, v, g, b2, 1.0, None)


def test_empty_sizes():
    S0 = state_like(3, 2, 64, 1)
    q = torch.empty(3, 2, 0, 64, device="cuda")
    e = torch.empty(3, 2, 0, device="cuda")
    o, S = vla.vla_delta_forward(q, q, q, e, e, 1.0, S0)
    assert o.shape == q.shape and torch.equal(S, S0)
    assert (vla.vla_delta_forward(q, q, q, None, e)[1] == 0).all()
    (dq, _, _), (dg, db), dS0 = vla.vla_delta_backward(q, q, q, e, e, 1.0, None, q, S0)
    assert dq.shape == q.shape and dg.shape == db.shape == (3, 2, 0) and torch.equal(dS0, S0)
    q, e = torch.empty(0, 2, 5, 64, device="cuda"), torch.empty(0, 2, 5, device="cuda")
    assert vla.vla_delta_forward(q, q, q, e, e)[1].shape == (0, 2, 64, 64)
    assert vla.vla_delta_backward(q, q, q, e, e)[2].shape == (0, 2, 64, 64)
    assert vla.vla_delta_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], e[:, :, 0], e[:, :, 0], S0).shape == (0, 2, 64)


def test_nothing_comes_back():
    """No gradient of o or of the state: zeros."""
    q, k, v = inputs(3, 1, 2, 50, 64, BF)
    g, beta = gates(1, 2, 50)
    grads, (dg, db), dS0 = vla.vla_delta_backward(q, k, v, g, beta, check=True)
    assert all((x == 0).all() for x in (*grads, dg, db, dS0))


def test_chunks_carry_on():
    """A prompt in pieces, the state carried in place, then single tokens: as one sequence."""
    B, H, T, d = 2, 3, 150, 96
    q, k, v = inputs(3, B, H, T, d, F32, seed=9)
    g, beta = gates(B, H, T)
    S = torch.zeros(B, H, d, d, device="cuda")
    parts = []
    for t0, t1 in ((0, 64), (64, 65), (65, 140)):
        x = [s[:, :, t0:t1] for s in (q, k, v, g, beta)]
        o, S2 = vla.vla_delta_forward(*x, 0.2, S, out=(torch.empty(B, H, t1 - t0, d, device="cuda"), S))
        assert S2 is S
        parts.append(o)
    for t in range(140, T):
        parts.append(vla.vla_delta_step(*(s[:, :, t] for s in (q, k, v, g, beta)), S, 0.2).unsqueeze(2))
    check_forward(q, k, v, g, beta, 0.2, None, None, (torch.cat(parts, 2), S))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_few_heads_and_many_give_the_same_bits(d, dtype):
    """Heads whose rows are spread over several blocks, and heads of a block each; and each time the same bits."""
    B, H, T = 5, 32, 100
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=d)
    g, beta = gates(B, H, T)
    n = torch.tensor([100, 99, 64, 33, 1], dtype=torch.int32, device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)

    def call(x, n):
        q, k, v, do, g, beta, S0, dS = x
        o, S = vla.vla_delta_forward(q, k, v, g, beta, 0.3, S0, lengths=n, check=True)
        grads, gg, dS0 = vla.vla_delta_backward(q, k, v, g, beta, 0.3, S0, do, dS, lengths=n, check=True)
        return (o, S, *grads, *gg, dS0)

    every = (q, k, v, do, g, beta, S0, dS)
    want = call(every, n)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(want, call(every, n)))
    for b, h, m in ((0, 0, 1), (2, 7, 2), (1, 0, 12), (3, 20, 12)):
        part = call([x[b:b + 1, h:h + m] for x in every], n[b:b + 1])
        assert all(torch.equal(x[b:b + 1, h:h + m], y) for x, y in zip(want, part))
    pick = slice(None, None, 9)
    part = lambda x: x[:, pick]  # noqa: E731
    check_forward(*map(part, (q, k, v, g, beta)), 0.3, part(S0), n, tuple(map(part, want[:2])))
    check_backward(*map(part, (q, k, v, g, beta)), 0.3, part(S0), part(do), part(dS), n,
                   (tuple(map(part, want[2:5])), tuple(map(part, want[5:7])), part(want[7])))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 128])
def test_keys_that_repeat(d, dtype):
    """One key for all tokens: with beta 1 and no decay, a token leaves nothing of the ones before it."""
    B, H, T = 1, 2, 90
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=d)
    k = torch.zeros_like(k)
    k[..., 3] = 1
    beta = torch.ones(B, H, T, device="cuda")
    o, S = vla.vla_delta_forward(q, k, v, None, beta, check=True)
    want = torch.zeros(B, H, d, d, dtype=torch.float64)
    want[..., 3] = v[:, :, -1].double().cpu()
    R.assert_normwise(S, want, R.roundings(T, d) * R.U, "S")
    # (1 + N)^-1 has as many terms as tokens in a chunk
    check_forward(q, k, v, None, beta, 1.0, None, None, (o, S), more=4)
    check_backward(q, k, v, None, beta, 1.0, None, do, None, more=4)
    g = torch.full((B, H, T), -0.1, device="cuda")
    check_forward(q, k, v, g, 0.5 * beta, 1.0, state_like(B, H, d, 1), more=4)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gates_at_their_ends(dtype):
    """-inf and values below it in effect, 0, a head that grows; beta 0 leaves the memory as it is."""
    B, H, T, d = 1, 4, 80, 64
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=1)
    g = torch.zeros(B, H, T, device="cuda")
    g[:, 0], g[:, 1], g[:, 2], g[:, 3] = float("-inf"), 0.0, -1000.0, 0.01
    g[:, 0, 40:], g[:, 2, 20:60] = -0.001, -0.02
    beta = torch.rand(B, H, T, device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    check_forward(q, k, v, g, beta, 0.5, S0)
    check_backward(q, k, v, g, beta, 0.5, S0, do, dS)
    none = torch.zeros(B, H, T, device="cuda")
    o, S = vla.vla_delta_forward(q, k, v, None, none, 1.0, S0, check=True)
    assert torch.equal(S, S0)
    grads, (_, db), dS0 = vla.vla_delta_backward(q, k, v, None, none, 1.0, S0, do, dS, check=True)
    assert (grads[2] == 0).all() and (grads[1] == 0).all() and (db != 0).any()


@pytest.mark.parametrize("H", [1, 200])
def test_slow_decays_over_long_sequences(H):
    """One write, then nothing: the state decays by the same factor thousands of times."""
    d, T = 32, 65536
    g = -torch.logspace(-6, -4, H).cuda()[None, :, None].expand(1, H, T)
    k, v = (torch.zeros(1, H, T, d, dtype=BF, device="cuda") for _ in range(2))
    beta = torch.zeros(1, H, T, device="cuda")
    k[:, :, 0], v[:, :, 0] = (x[:, :, 0] for x in seqs(2, 1, H, 1, d, BF))
    beta[:, :, 0] = 1
    S = vla.vla_delta_forward(k, k, v, g, beta, check=True)[1].double().cpu()
    want = (torch.exp(g[:, :, 0].double().cpu() * (T - 1))[..., None, None]
            * (v[:, :, 0, :, None].double() * k[:, :, 0, None, :].double()).cpu())
    # T / 32 products, each off by at most half a step on its own: six times their standard deviation; the factors'
    # own roundings do not add up, but a chunk's sum of g is rounded (2^-24 of 0.0032 a chunk at most)
    bound = (6 * (T / 32 / 12) ** 0.5 + 8) * 2 * R.U + T / 32 * 0.0032 * R.U
    assert float(((S - want).abs() / want.abs().clamp(min=1e-30)).max()) <= bound


def test_gradients_against_differences():
    """The loss is linear in q, v and the state, and quadratic at most in one token's k, g's factor or beta."""
    B, H, T, d = 1, 2, 90, 32
    q, k, v, do = inputs(4, B, H, T, d, F32, seed=11)
    g, beta = gates(B, H, T)
    g = g.clamp(min=-5)
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    (dq, dk, dv), (dg, db), dS0 = vla.vla_delta_backward(q, k, v, g, beta, 0.3, S0, do, dS)

    def loss(q, k, v, g, beta, S0):
        o, S, _ = R.delta(q, k, v, g, beta, 0.3, S0)
        return float((o * do.double().cpu()).sum() + (S * dS.double().cpu()).sum())

    args = [x.double().cpu() for x in (q, k, v, g, beta, S0)]
    for i, grad in enumerate((dq, dk, dv, dg, db, dS0)):
        x = args[i]
        for t in (0, 31, 32, T - 1):
            step = torch.randn(x.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
            if i != 5:
                keep = torch.zeros(x.shape, dtype=torch.float64)
                keep[:, :, t] = 1
                step = step * keep
            h = 2.0 ** -17  # differences in 64 bits: h^2 of the third derivative, 2^-53 / h of the loss
            plus, minus = list(args), list(args)
            plus[i], minus[i] = x + h * step, x - h * step
            diff = (loss(*plus) - loss(*minus)) / (2 * h)
            want = float((grad.double().cpu() * step).sum())
            size = float((grad.double().cpu() * step).abs().sum())
            assert abs(diff - want) <= 1e-5 * size + 1e-6, (i, t, diff, want)


def test_non_finite_results_are_recorded():
    """A NaN stays in its head, and behind its block of 64 tokens' start (in o), before its end (in gradients)."""
    q, k, v, do = inputs(4, 1, 2, 200, 64, BF)
    g, beta = gates(1, 2, 200)
    vla.vla_get_last_device_status()
    k2 = k.clone()
    k2[0, 1, 150, 3] = float("inf")
    with pytest.raises(vla.VLAError) as e:
        vla.vla_delta_forward(q, k2, v, g, beta, check=True)
    assert e.value.status == 5 and e.value.detail[1] == 1
    o, S = vla.vla_delta_forward(q, k2, v, g, beta)
    assert torch.isfinite(o[0, 0]).all() and torch.isfinite(o[0, 1, :128]).all() and not torch.isfinite(o[0, 1, 150:]).all()
    assert torch.isfinite(S[0, 0]).all() and not torch.isfinite(S[0, 1]).all()
    assert vla.vla_get_last_device_status()[0] == 5 and vla.vla_get_last_device_status()[0] == 0
    do2 = do.clone()
    do2[0, 1, 20, 5] = float("nan")
    grads, gg, dS0 = vla.vla_delta_backward(q, k, v, g, beta, 1.0, None, do2)
    assert vla.vla_get_last_device_status()[0] == 5
    for x in (*grads, *gg):
        assert torch.isfinite(x[0, 0]).all() and torch.isfinite(x[0, 1, 64:]).all()
    assert not torch.isfinite(grads[0][0, 1, 20]).all() and torch.isfinite(dS0[0, 0]).all()
    # one value of v touches its coordinate of the state alone
    v2 = v.clone()
    v2[0, 1, 150, 3] = float("nan")
    o, S = vla.vla_delta_forward(q, k, v2, g, beta)
    rest = [i for i in range(64) if i != 3]
    assert torch.isfinite(o[..., rest]).all() and torch.isfinite(S[:, :, rest]).all()
    assert vla.vla_get_last_device_status()[0] == 5


@pytest.mark.parametrize("d", [64, 128])
def test_streams_and_graphs(d):
    """Calls on two streams at once, and a captured call replayed on new inputs."""
    B, H, T = 1, 4, 300
    sets = [(*inputs(4, B, H, T, d, BF, seed=s), *gates(B, H, T, s)) for s in (1, 2)]
    S0 = state_like(B, H, d, 1)

    def call(x, stream=None):
        q, k, v, do, g, beta = x
        return (vla.vla_delta_forward(q, k, v, g, beta, 0.1, S0, stream=stream),
                vla.vla_delta_backward(q, k, v, g, beta, 0.1, S0, do, S0, stream=stream))

    want = [call(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [call(x, s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()

    def same(a, b):
        if isinstance(a, torch.Tensor):
            return torch.equal(a, b)
        return all(same(x, y) for x, y in zip(a, b))

    assert same(want, got)
    ins = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call(ins)
    for x, w in zip(sets, want):
        for a, b in zip(ins, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert same(w, res)


# ---- single tokens ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_step(d, dtype):
    B, H, N = 5, 3, 9
    q, k, v = (x[:, :, 0] for x in inputs(3, B, H, 1, d, dtype, seed=d))
    g, beta = (x[:, :, 0] for x in gates(B, H, 1))
    g[0, 0], beta[2, 1] = float("-inf"), 0.0
    pool = state_like(N, H, d, 1)
    before = pool.clone()
    slots = torch.tensor([7, -1, 0, 3, 8], dtype=torch.int32, device="cuda")
    o = vla.vla_delta_step(q, k, v, g, beta, pool, 0.7, slots=slots, check=True)
    live = [0, 2, 3, 4]
    at = slots[live].long()
    pick = lambda x: x[live].unsqueeze(2)  # noqa: E731
    ro, rS, _ = R.delta(*map(pick, (q, k, v, g, beta)), 0.7, before[at])
    e = R.roundings(1, d) * R.U
    R.assert_normwise(pool[at], rS, e, "S")
    if dtype == BF:
        R.assert_rounded(o[live].unsqueeze(2), ro, 0 * ro, 1, "o")
    else:
        R.assert_normwise(o[live].unsqueeze(2), ro, e, "o")
    assert (o[1] == 0).all()
    rest = [i for i in range(N) if i not in (7, 0, 3, 8)]
    assert torch.equal(pool[rest], before[rest])
    # no decay, and slots by number
    pool = before.clone()
    vla.vla_delta_step(q, k, v, None, beta, pool, 0.7, check=True)
    _, rS, _ = R.delta(*(x.unsqueeze(2) for x in (q, k, v)), None, beta.unsqueeze(2), 0.7, before[:B])
    R.assert_normwise(pool[:B], rS, e, "S")


def test_step_bad_slots():
    """A slot out of range or used twice: the first use counts, the others are idle rows and recorded."""
    B, H, d, N = 4, 2, 64, 3
    q, k, v = (x[:, :, 0] for x in inputs(3, B, H, 1, d, F32))
    g, beta = (x[:, :, 0] for x in gates(B, H, 1))
    pool = state_like(N, H, d, 1)
    before = pool.clone()
    vla.vla_get_last_device_status()
    slots = torch.tensor([1, 3, 1, 2], dtype=torch.int32, device="cuda")
    o = vla.vla_delta_step(q, k, v, g, beta, pool, slots=slots)
    st, detail = vla.vla_get_last_device_status()
    assert st == vla._binding.VLA_ERR_BAD_SLOT and detail in ((4, 1, 3), (4, 2, 1))
    good, use = before.clone(), [0, 3]
    want = vla.vla_delta_step(*(x[use] for x in (q, k, v, g, beta)), good, slots=slots[use], check=True)
    assert torch.equal(pool, good) and torch.equal(o[use], want) and (o[[1, 2]] == 0).all()
    with pytest.raises(vla.VLAError):
        vla.vla_delta_step(q, k, v, g, beta, pool, slots=slots, check=True)


def test_long_pool():
    """Slots behind 2^31 values."""
    H, d = 4, 128
    N = (1 << 31) // (H * d * d) + 3
    pool = torch.zeros(N, H, d, d, device="cuda")
    q, k, v = (x[:, :, 0] for x in inputs(3, 2, H, 1, d, BF))
    g, beta = (x[:, :, 0] for x in gates(2, H, 1))
    slots = torch.tensor([N - 1, 0], dtype=torch.int32, device="cuda")
    S = torch.zeros(2, H, d, d, device="cuda")
    o = vla.vla_delta_step(q, k, v, g, beta, pool, slots=slots, check=True)
    assert torch.equal(o, vla.vla_delta_step(q, k, v, g, beta, S, check=True))
    assert torch.equal(pool[[N - 1, 0]], S) and not pool[1:N - 1].any()


def test_step_in_a_graph():
    """Captured once and replayed: each replay goes one token on."""
    B, H, d = 3, 2, 96
    q, k, v = inputs(3, B, H, 4, d, BF, seed=6)
    g, beta = gates(B, H, 4)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool = state_like(5, H, d, 3)
    want = pool.clone()
    outs = [vla.vla_delta_step(*(x[:, :, t] for x in (q, k, v, g, beta)), want, slots=slots) for t in range(4)]
    token = [x[:, :, 0].clone() for x in (q, k, v, g, beta)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = vla.vla_delta_step(*token, pool, slots=slots)
    for t in range(4):
        for a, b in zip(token, (q, k, v, g, beta)):
            a.copy_(b[:, :, t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, outs[t])
    assert torch.equal(pool, want)


# ---- together ------------------------------------------------------------------------------------------------------

def test_training_step_together():
    """Norm and rotation, the rule, the readout's norm, and back through all of them: against autograd in 64 bits."""
    B, H, T, d = 2, 3, 100, 64
    q, k, v, dy = seqs(4, B, H, T, d, F32, seed=4)
    g, beta = gates(B, H, T)
    g = g.clamp(min=-5)
    wq, wk, wy = (1 + 0.1 * torch.randn(H, d, device="cuda") for _ in range(3))
    freqs = vla.vla_rotation_frequencies(32)
    scale = d ** -0.5

    kw = dict(unit=True, freqs=freqs)
    (yq, yk), stats = vla.vla_qk_norm(q, k, wq, wk, 1e-6, **kw)
    o, S = vla.vla_delta_forward(yq, yk, v, g, beta, scale, check=True)
    y, ystats = vla.vla_head_norm(o, wy)
    do, dwy, _ = vla.vla_head_norm_backward(dy, o, ystats, wy)
    (dyq, dyk, dv), (dg, db), _ = vla.vla_delta_backward(yq, yk, v, g, beta, scale, None, do, check=True)
    (dq, dk), (dwq, dwk) = vla.vla_qk_norm_backward(dyq, dyk, q, k, stats, wq, wk, **kw)

    leaves = [x.double().cpu().requires_grad_() for x in (q, k, v, g, beta, wq, wk, wy)]
    q6, k6, v6, g6, b6, wq6, wk6, wy6 = leaves
    pos = torch.arange(T)[None].expand(B, T)
    xq, xk = (R.qk(x, w, True, 1e-6, freqs.cpu(), pos)[0] for x, w in ((q6, wq6), (k6, wk6)))
    M = torch.zeros(B, H, d, d, dtype=torch.float64)
    rows = []
    for t in range(T):
        M = torch.exp(g6[:, :, t])[..., None, None] * M
        M = M + (b6[:, :, t, None] * (v6[:, :, t] - (M @ xk[:, :, t, :, None])[..., 0]))[..., :, None] * xk[:, :, t, None, :]
        rows.append(scale * (M @ xq[:, :, t, :, None])[..., 0])
    o6 = torch.stack(rows, 2)
    c = o6 - o6.mean(-1, keepdim=True)
    y6 = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * wy6[:, None]
    (y6 * dy.double().cpu()).sum().backward()
    R.assert_normwise(S, M.detach(), 2 * R.roundings(T, d) * R.U, "S")
    # early rows of o are small beside the norm's eps and the errors of what went into them: the norm divides by them
    R.assert_normwise(y, y6.detach(), 1e-4, "y")
    for name, x, leaf in zip(("dq", "dk", "dv", "dg", "dbeta"), (dq, dk, dv, dg, db), leaves):
        R.assert_normwise(x, leaf.grad, 1e-4, name)
    for name, x, leaf in zip(("dwq", "dwk", "dwy"), (dwq, dwk, dwy), leaves[5:]):
        R.assert_normwise(x[None], leaf.grad[None], 1e-4, name)


def test_serving_together():
    """A padded prompt, its states parked in 8 bits and brought back into other rows, then tokens: as without parking
    up to the codes' steps."""
    B, H, T, d = 3, 2, 60, 64
    q, k, v = seqs(3, B, H, T + 1, d, BF, seed=7)
    g, beta = gates(B, H, T + 1)
    n = torch.tensor([60, 31, 7], dtype=torch.int32, device="cuda")
    freqs = vla.vla_rotation_frequencies(64)
    (yq, yk), _ = vla.vla_qk_norm(q[:, :, :T], k[:, :, :T], unit=True, freqs=freqs)
    _, S = vla.vla_delta_forward(yq, yk, v[:, :, :T], g[:, :, :T], beta[:, :, :T], lengths=n, check=True)
    codes, scales = vla.vla_state_cache(8, (H, d, d), 8)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    vla.vla_state_store(S, codes, scales, slots, check=True)
    pool = vla.vla_state_load(codes, scales, slots, check=True)
    assert float((pool - S).abs().max()) <= float(scales.max()) * 0.501
    (tq, tk), _ = vla.vla_qk_norm(q[:, :, T:], k[:, :, T:], unit=True, freqs=freqs, positions=n[:, None].contiguous())
    token = [x[:, :, 0] for x in (tq, tk)] + [v[:, :, T], g[:, :, T], beta[:, :, T]]
    base = pool.double().cpu()
    o = vla.vla_delta_step(*token, pool, check=True)
    ro, rS, _ = R.delta(*(x.unsqueeze(2) for x in token), 1.0, base)
    R.assert_normwise(pool, rS, R.roundings(1, d) * R.U, "S")
    R.assert_rounded(o.unsqueeze(2), ro, 0 * ro, 1, "o")


# ---- waits ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_a_wait_that_runs_out_is_reported(d):
    """The last chunk's loads kept back: the waits give up, the status says so, and the calls behind are right."""
    B, H, T = 1, 3, 300
    q, k, v, do = inputs(4, B, H, T, d, BF, seed=d)
    g, beta = gates(B, H, T)
    vla.vla_get_last_device_status()
    for _ in range(2):
        with pytest.raises(vla.VLAError) as e:
            vla.vla_delta_forward(q, k, v, g, beta, check=True, wait_limit_us=2000, test_stall_producer=True)
        assert e.value.status == vla.VLA_ERR_TIMEOUT
        check_forward(q, k, v, g, beta, 1.0, None)
        with pytest.raises(vla.VLAError) as e:
            vla.vla_delta_backward(q, k, v, g, beta, 1.0, None, do, check=True, wait_limit_us=2000, test_stall_producer=True)
        assert e.value.status == vla.VLA_ERR_TIMEOUT
        check_backward(q, k, v, g, beta, 1.0, None, do, None)


def test_calls_without_waits_do_not_stall():
    """fp32 calls and short ones have no waits: the option changes nothing."""
    for dtype, T in ((F32, 300), (BF, 64)):
        q, k, v, do = inputs(4, 1, 2, T, 64, dtype)
        g, beta = gates(1, 2, T)
        kw = dict(check=True, wait_limit_us=2000, test_stall_producer=True)
        check_forward(q, k, v, g, beta, 1.0, None, None, vla.vla_delta_forward(q, k, v, g, beta, **kw))
        check_backward(q, k, v, g, beta, 1.0, None, do, None, None, vla.vla_delta_backward(q, k, v, g, beta, 1.0, None, do, **kw))


@pytest.mark.parametrize("d,H,T", [(32, 24, 200), (64, 24, 200), (96, 24, 200), (128, 24, 200), (128, 12, 200),
                                   (32, 24, 20), (64, 24, 20), (96, 24, 40), (128, 24, 1)])
def test_more_heads_than_sms(d, H, T):
    """One block or several an SM, lengths at every edge of a chunk, the same bits each time."""
    B = 9
    q, k, v, do = inputs(4, B, H, T, d, BF, seed=d)
    g, beta = gates(B, H, T)
    n = torch.tensor([200, 199, 193, 192, 191, 129, 64, 9, 1], dtype=torch.int32, device="cuda").clamp(max=T)
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)

    def call():
        o, S = vla.vla_delta_forward(q, k, v, g, beta, 0.2, S0, lengths=n, check=True)
        grads, gg, dS0 = vla.vla_delta_backward(q, k, v, g, beta, 0.2, S0, do, dS, lengths=n, check=True)
        return (o, S, *grads, *gg, dS0)

    want = call()
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(want, call()))
    pick = slice(None, None, 7)
    part = lambda x: x[:, pick]  # noqa: E731
    check_forward(*map(part, (q, k, v, g, beta)), 0.2, part(S0), n, tuple(map(part, want[:2])))
    check_backward(*map(part, (q, k, v, g, beta)), 0.2, part(S0), part(do), part(dS), n,
                   (tuple(map(part, want[2:5])), tuple(map(part, want[5:7])), part(want[7])))
