"""The operators of include/vla_layer.h on the GPU against their fp64 forms
(layer_ref.py): sizes at the kernels' tile and segment edges, carried states,
padded batches, strides, decays from none to total, streams and graphs."""
import pytest
import torch

import layer_ref as R
import sherman_morrison_memory_gb300 as vla

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def seqs(n, B, H, T, d, dtype, seed=0, rows="heads"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(n):
        if rows == "tokens":
            out.append(torch.randn(B, T, H, d, generator=gen, device="cuda").to(dtype).transpose(1, 2))
        else:
            out.append(torch.randn(B, H, T, d, generator=gen, device="cuda").to(dtype))
    return out


def state_like(B, H, d, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, H, d, d, generator=gen, device="cuda")


def decays(H):
    """From almost none to strong ones, and 0, -inf and a growing head where there are heads for them."""
    g = -torch.exp2(torch.linspace(-9, 1, H, dtype=torch.float64))
    if H >= 3:
        g[0], g[1] = 0.0, float("-inf")
    if H >= 4:
        g[2] = 0.003
    return g.float().cuda()


def check_forward(q, k, v, g, scale, state, lengths, got=None):
    B, H, T, d = q.shape
    o, S = got if got is not None else vla.vla_decay_forward(q, k, v, g, scale, state, lengths=lengths, check=True)
    ro, rS = R.decay(q, k, v, g, scale, state, lengths)
    mo, mS = R.decay(q.abs(), k.abs(), v.abs(), g, abs(scale), None if state is None else state.abs(), lengths)
    assert o.dtype == q.dtype and S.dtype == F32
    R.assert_within(o, ro, R.seq_bound(ro, mo, q.dtype, T, d, g), "o")
    R.assert_within(S, rS, R.state_bound(mS, q.dtype, T, d, g), "S")
    return o, S


def check_backward(q, k, v, g, scale, state, do, dS, lengths, got=None):
    B, H, T, d = q.shape
    (dq, dk, dv), dS0 = got if got is not None else vla.vla_decay_backward(q, k, v, g, scale, state, do, dS,
                                                                           lengths=lengths, check=True)
    ref = R.decay_grads(q, k, v, g, scale, state, do, dS, lengths)
    a = lambda x: None if x is None else x.abs()  # noqa: E731
    mag = R.decay_grads(a(q), a(k), a(v), g, abs(scale), a(state), a(do), a(dS), lengths)
    for name, x, r, m in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, mag):
        assert x.dtype == q.dtype
        R.assert_within(x, r, R.seq_bound(r, m, q.dtype, T, d, g), name)
    R.assert_within(dS0, ref[3], R.state_bound(mag[3], q.dtype, T, d, g), "dS0")


# ---- linear attention with a decay --------------------------------------------------------------------------------

SIZES = [(1, 1, 1, 32), (2, 3, 2, 64), (1, 4, 31, 96), (2, 2, 32, 128), (1, 3, 33, 32), (3, 1, 63, 64), (1, 5, 64, 96),
         (2, 4, 65, 128), (1, 2, 127, 64), (1, 4, 128, 32), (2, 3, 129, 96), (1, 4, 200, 128)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_decay_forward(B, H, T, d, dtype):
    q, k, v = seqs(3, B, H, T, d, dtype, seed=T + d)
    g = decays(H)
    check_forward(q, k, v, g, 1.0, None, None)
    check_forward(q, k, v, g, -0.3, state_like(B, H, d, 1), None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_decay_backward(B, H, T, d, dtype):
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=T + d + 1)
    g = decays(H)
    check_backward(q, k, v, g, 1.0, None, do, None, None)
    check_backward(q, k, v, g, 0.4, state_like(B, H, d, 1), do, state_like(B, H, d, 2), None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(513, 32), (777, 64), (1024, 96), (1153, 128)])
def test_decay_in_segments(T, d, dtype):
    """Few heads of long sequences: cut into segments that run side by side."""
    q, k, v, do = seqs(4, 1, 2, T, d, dtype, seed=T)
    g = torch.tensor([-0.002, -0.3], device="cuda")
    S0, dS = state_like(1, 2, d, 3), state_like(1, 2, d, 4)
    check_forward(q, k, v, g, d ** -0.5, S0, None)
    check_backward(q, k, v, g, d ** -0.5, S0, do, dS, None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d,lengths", [(70, 64, [70, 0, 1, 69]), (130, 128, [64, 65, 130, 129]), (33, 96, [32, 33, 5, 0]),
                                         (900, 32, [900, 0, 257, 513]), (700, 128, [1, 700, 256, -4])])
def test_padded_batches(T, d, lengths, dtype):
    """Rows behind a sequence's end hold NaN and Inf: nothing of them is seen, and their results are zero."""
    B, H = len(lengths), 2
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=d)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    clean = [x.clone() for x in (q, k, v, do)]
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (do, float("-inf"))):
        for b, m in enumerate(lengths):
            x[b, :, max(0, m):] = bad
    for x, c in zip(clean, (q, k, v, do)):
        x[~torch.isfinite(c)] = 0
    g = torch.tensor([-0.01, -0.5], device="cuda")
    S0, dS = state_like(B, H, d, 5), state_like(B, H, d, 6)
    got = vla.vla_decay_forward(q, k, v, g, 0.5, S0, lengths=n, check=True)
    check_forward(*clean[:3], g, 0.5, S0, n, got)
    back = vla.vla_decay_backward(q, k, v, g, 0.5, S0, do, dS, lengths=n, check=True)
    check_backward(*clean[:3], g, 0.5, S0, clean[3], dS, n, back)
    for x in (got[0], *back[0]):
        for b, m in enumerate(lengths):
            assert (x[b, :, max(0, m):] == 0).all()
    for b, m in enumerate(lengths):
        if m <= 0:
            assert torch.equal(got[1][b], S0[b]) and torch.equal(back[1][b], dS[b])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 96, 128])
def test_strides(d, dtype):
    """Token-order inputs and outputs, slices of wider rows and of longer sequences, odd offsets (copied)."""
    B, H, T = 2, 3, 77
    g = decays(H)
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=3, rows="tokens")
    out = torch.full((B, T, H, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
    S = torch.empty(B, H, d, d, device="cuda")
    o, _ = vla.vla_decay_forward(q, k, v, g, 1.0, out=(out, S), check=True)
    assert o is out
    check_forward(q, k, v, g, 1.0, None, None, (o, S))
    wide = torch.randn(B, H, T + 9, 2 * d + 16, device="cuda").to(dtype)
    q2, k2 = wide[:, :, 4:T + 4, 8:d + 8], wide[:, :, :T, d + 16:]
    odd = torch.randn(B, H, T, d + 3, device="cuda").to(dtype)[..., 3:]
    before = wide.clone()
    check_forward(q2, k2, odd, g, 1.0, None, None)
    check_backward(q2, k2, odd, g, 1.0, None, do, None, None)
    assert torch.equal(before, wide)
    # one key head for all, as a broadcast view
    check_forward(q, k[:, :1].expand(B, H, T, d), v, g, 1.0, None, None)


def test_padding_between_rows_is_left_alone():
    B, H, T, d = 2, 2, 70, 64
    q, k, v, do = seqs(4, B, H, T, d, BF, seed=8)
    g = decays(H)
    frame = torch.full((B, H, T + 5, d + 16), 3.0, dtype=BF, device="cuda")
    grads = [frame.clone() for _ in range(3)]
    o = frame[:, :, 2:T + 2, 8:d + 8]
    S = torch.empty(B, H, d, d, device="cuda")
    vla.vla_decay_forward(q, k, v, g, out=(o, S))
    vla.vla_decay_backward(q, k, v, g, 1.0, None, do, out=(*(x[:, :, 2:T + 2, 8:d + 8] for x in grads), S))
    torch.cuda.synchronize()
    for x in (frame, *grads):
        inner = x[:, :, 2:T + 2, 8:d + 8]
        assert (inner != 3.0).any()
        x = x.clone()
        x[:, :, 2:T + 2, 8:d + 8] = 3.0
        assert (x == 3.0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_far_apart(dtype):
    """Sequences more than 2^31 elements apart."""
    d, T = 64, 40
    far = (1 << 31) + 4096
    buf = torch.empty(far + T * d, dtype=dtype, device="cuda")
    x = buf.as_strided((2, 1, T, d), (far, T * d, d, 1))
    q, k, v = seqs(3, 2, 1, T, d, dtype)
    x.copy_(k)
    g = decays(1)
    check_forward(q, x, v, g, 1.0, None, None)
    x.zero_()
    vla.vla_decay_forward(q, k, v, g, out=(x, torch.empty(2, 1, d, d, device="cuda")), check=True)
    check_forward(q, k, v, g, 1.0, None, None, (x, vla.vla_decay_forward(q, k, v, g)[1]))


def test_empty_sizes():
    g = decays(2)
    S0 = state_like(3, 2, 64, 1)
    q = torch.empty(3, 2, 0, 64, device="cuda")
    o, S = vla.vla_decay_forward(q, q, q, g, 1.0, S0)
    assert o.shape == q.shape and torch.equal(S, S0)
    assert (vla.vla_decay_forward(q, q, q, g)[1] == 0).all()
    (dq, _, _), dS0 = vla.vla_decay_backward(q, q, q, g, 1.0, None, q, S0)
    assert dq.shape == q.shape and torch.equal(dS0, S0)
    e = torch.empty(0, 2, 5, 64, device="cuda")
    assert vla.vla_decay_forward(e, e, e, g)[1].shape == (0, 2, 64, 64)
    y, _ = vla.vla_head_norm(e)
    assert y.shape == e.shape
    w = torch.ones(2, 64, device="cuda")
    dx, dw, db = vla.vla_head_norm_backward(e, e, (e[..., 0], e[..., 0]), w)
    assert (dw == 0).all() and (db == 0).all() and dw.shape == (2, 64)
    assert vla.vla_decay_step(e[:, :, 0], e[:, :, 0], e[:, :, 0], g, S0).shape == (0, 2, 64)


def test_chunks_carry_on():
    """A prompt in pieces, the state carried in place, then single tokens: as one sequence."""
    B, H, T, d = 2, 3, 150, 96
    q, k, v = seqs(3, B, H, T, d, F32, seed=9)
    g = decays(H)
    S = torch.zeros(B, H, d, d, device="cuda")
    parts = []
    for t0, t1 in ((0, 64), (64, 65), (65, 140)):
        x = [s[:, :, t0:t1] for s in (q, k, v)]
        o, S2 = vla.vla_decay_forward(*x, g, 0.2, S, out=(torch.empty(B, H, t1 - t0, d, device="cuda"), S))
        assert S2 is S
        parts.append(o)
    for t in range(140, T):
        parts.append(vla.vla_decay_step(*(s[:, :, t] for s in (q, k, v)), g, S, 0.2).unsqueeze(2))
    check_forward(q, k, v, g, 0.2, None, None, (torch.cat(parts, 2), S))


def test_gradients_against_differences():
    """The loss is linear in each of q, k, v and the state, so that central differences are exact."""
    B, H, T, d = 1, 2, 90, 32
    q, k, v, do = (x.double().float() for x in seqs(4, B, H, T, d, F32, seed=11))
    g = torch.tensor([-0.02, -0.4], device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    (dq, dk, dv), dS0 = vla.vla_decay_backward(q, k, v, g, 0.3, S0, do, dS)

    def loss(q, k, v, S0):
        o, S = vla.vla_decay_forward(q, k, v, g, 0.3, S0)
        return float((o.double() * do.double()).sum() + (S.double() * dS.double()).sum())

    args = [q, k, v, S0]
    for i, grad in enumerate((dq, dk, dv, dS0)):
        x = args[i]
        step = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").round()
        plus, minus = list(args), list(args)
        plus[i], minus[i] = x + step, x - step
        diff = (loss(*plus) - loss(*minus)) / 2
        want = float((grad.double() * step.double()).sum())
        # every output is within gamma of its magnitude; the losses sum them against do and dS
        o_m, S_m = R.decay(*(a.abs() + step.abs() if j == i else a.abs() for j, a in enumerate(args[:3])), g, 0.3,
                           S0.abs() + step.abs() if i == 3 else S0.abs())
        total = float((o_m * do.abs().double().cpu()).sum() + (S_m * dS.abs().double().cpu()).sum())
        assert abs(diff - want) <= 2 * R.gamma(T, d, g) * total, (i, diff, want)


def test_non_finite_results_are_recorded():
    q, k, v = seqs(3, 1, 2, 50, 64, BF)
    g = decays(2)
    k[0, 1, 20, 3] = float("inf")
    vla.vla_get_last_device_status()
    with pytest.raises(vla.VLAError) as e:
        vla.vla_decay_forward(q, k, v, g, check=True)
    assert e.value.status == 5 and e.value.detail[1] == 1
    o, _ = vla.vla_decay_forward(q, k, v, g)
    assert torch.isfinite(o[0, 0]).all() and torch.isfinite(o[0, 1, :20]).all()
    assert vla.vla_get_last_device_status()[0] == 5 and vla.vla_get_last_device_status()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_streams_and_graphs(d):
    """Calls on two streams at once, and a captured call replayed on new inputs."""
    B, H, T = 1, 4, 700
    g = decays(H)
    sets = [seqs(4, B, H, T, d, BF, seed=s) for s in (1, 2)]
    S0 = state_like(B, H, d, 1)
    want = [(vla.vla_decay_forward(*x[:3], g, 0.1, S0), vla.vla_decay_backward(*x[:3], g, 0.1, S0, x[3], S0)) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for x, s in zip(sets, streams):
        got.append((vla.vla_decay_forward(*x[:3], g, 0.1, S0, stream=s),
                    vla.vla_decay_backward(*x[:3], g, 0.1, S0, x[3], S0, stream=s)))
    torch.cuda.synchronize()

    def same(a, b):
        if isinstance(a, torch.Tensor):
            return torch.equal(a, b)
        return all(same(x, y) for x, y in zip(a, b))

    assert same(want, got)
    inputs = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = (vla.vla_decay_forward(*inputs[:3], g, 0.1, S0),
               vla.vla_decay_backward(*inputs[:3], g, 0.1, S0, inputs[3], S0))
    for x, w in zip(sets, want):
        for a, b in zip(inputs, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert same(w, res)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H", [1, 200])
def test_slow_decays_over_long_sequences(H, dtype):
    """One write, then nothing: the state decays by the same factor thousands of times (in segments and in one piece)."""
    d, T = 32, 65536
    g = -torch.logspace(-6, -4, H).cuda()
    k, v = (torch.zeros(1, H, T, d, dtype=dtype, device="cuda") for _ in range(2))
    k[:, :, 0], v[:, :, 0] = (x[:, :, 0] for x in seqs(2, 1, H, 1, d, dtype))
    S = vla.vla_decay_forward(k, k, v, g, check=True)[1].double().cpu()
    want = torch.exp(g.double().cpu() * (T - 1))[None, :, None, None] * (v[:, :, 0, :, None].double() * k[:, :, 0, None, :].double()).cpu()
    # T / 32 products, each off by at most half a step on its own: six times their standard deviation, and the
    # factors' own roundings, which do not add up (bf16: the write itself in three exact parts)
    bound = (6 * (T / 32 / 12) ** 0.5 + 8) * 2 * R.U
    assert float(((S - want).abs() / want.abs().clamp(min=1e-30)).max()) <= bound


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,T,d", [(1, 155, 700, 64), (2, 80, 1025, 32), (1, 56, 1500, 128)])
def test_whole_waves_and_the_rest(B, H, T, d, dtype):
    """A few heads more than fill the SMs: those are cut into segments, the others not."""
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=d)
    g = -torch.exp2(torch.linspace(-9, 0, H)).cuda()
    n = torch.full((B,), T - 3, dtype=torch.int32, device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    fwd = vla.vla_decay_forward(q, k, v, g, 0.2, S0, lengths=n, check=True)
    bwd = vla.vla_decay_backward(q, k, v, g, 0.2, S0, do, dS, lengths=n, check=True)
    pick = torch.tensor([0, H // 2, H - 4, H - 1])
    part = lambda x: x[:, pick]  # noqa: E731
    check_forward(part(q), part(k), part(v), g[pick], 0.2, part(S0), n, tuple(part(x) for x in fwd))
    check_backward(part(q), part(k), part(v), g[pick], 0.2, part(S0), part(do), part(dS), n,
                   (tuple(part(x) for x in bwd[0]), part(bwd[1])))


@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_more_heads_than_sms(d):
    """Several blocks an SM one after another, lengths at every edge of a chunk, the same bits each time."""
    B, H, T = 9, 24, 200
    q, k, v, do = seqs(4, B, H, T, d, BF, seed=d)
    g = -torch.exp2(torch.linspace(-8, 0, H)).cuda()
    n = torch.tensor([200, 199, 193, 192, 191, 129, 64, 9, 1], dtype=torch.int32, device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    fwd = vla.vla_decay_forward(q, k, v, g, 0.2, S0, lengths=n, check=True)
    bwd = vla.vla_decay_backward(q, k, v, g, 0.2, S0, do, dS, lengths=n, check=True)
    for _ in range(20):
        o, S = vla.vla_decay_forward(q, k, v, g, 0.2, S0, lengths=n)
        grads, dS0 = vla.vla_decay_backward(q, k, v, g, 0.2, S0, do, dS, lengths=n)
        assert torch.equal(o, fwd[0]) and torch.equal(S, fwd[1]) and torch.equal(dS0, bwd[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, bwd[0]))
    # every third head against the definition
    pick = slice(None, None, 3)
    part = lambda x: x[:, pick]  # noqa: E731
    check_forward(part(q), part(k), part(v), g[pick], 0.2, part(S0), n, tuple(part(x) for x in fwd))
    check_backward(part(q), part(k), part(v), g[pick], 0.2, part(S0), part(do), part(dS), n,
                   (tuple(part(x) for x in bwd[0]), part(bwd[1])))


# ---- single tokens ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_step(d, dtype):
    B, H, N = 5, 3, 9
    q, k, v = (x[:, :, 0] for x in seqs(3, B, H, 1, d, dtype, seed=d))
    g = decays(H)
    pool = state_like(N, H, d, 1)
    before = pool.clone()
    slots = torch.tensor([7, -1, 0, 3, 8], dtype=torch.int32, device="cuda")
    o = vla.vla_decay_step(q, k, v, g, pool, 0.7, slots=slots, check=True)
    live = [0, 2, 3, 4]
    at = slots[live].long()
    ro, rS = R.decay(*(x[live].unsqueeze(2) for x in (q, k, v)), g, 0.7, before[at])
    mo, mS = R.decay(*(x[live].unsqueeze(2).abs() for x in (q, k, v)), g, 0.7, before[at].abs())
    e = R.gamma(1, d, g)
    half = R.HALF[dtype] if dtype == BF else 0.0  # the one rounding of a bf16 result
    R.assert_within(o[live].unsqueeze(2), ro, e * mo + half * ro.abs() + 1e-30, "o")
    R.assert_within(pool[at], rS, e * mS + 1e-30, "S")
    assert (o[1] == 0).all()
    rest = [i for i in range(N) if i not in (7, 0, 3, 8)]
    assert torch.equal(pool[rest], before[rest])


def test_step_bad_slots():
    """A slot out of range or used twice: the first use counts, the others are idle rows and recorded."""
    B, H, d, N = 4, 2, 64, 3
    q, k, v = (x[:, :, 0] for x in seqs(3, B, H, 1, d, F32))
    g = decays(H)
    pool = state_like(N, H, d, 1)
    before = pool.clone()
    vla.vla_get_last_device_status()
    slots = torch.tensor([1, 3, 1, 2], dtype=torch.int32, device="cuda")
    o = vla.vla_decay_step(q, k, v, g, pool, slots=slots)
    st, detail = vla.vla_get_last_device_status()
    assert st == vla._binding.VLA_ERR_BAD_SLOT and detail in ((4, 1, 3), (4, 2, 1))
    good = before.clone()
    want = vla.vla_decay_step(q[[0, 3]], k[[0, 3]], v[[0, 3]], g, good, slots=slots[[0, 3]], check=True)
    assert torch.equal(pool, good) and torch.equal(o[[0, 3]], want) and (o[[1, 2]] == 0).all()
    with pytest.raises(vla.VLAError):
        vla.vla_decay_step(q, k, v, g, pool, slots=slots, check=True)


def test_long_pools():
    """Slots behind 2^31 values: stepped, stored and read."""
    H, d = 4, 128
    N = (1 << 31) // (H * d * d) + 3
    pool = torch.zeros(N, H, d, d, device="cuda")
    codes, scales = vla.vla_state_cache(N, (H, d, d), 8)
    q, k, v = (x[:, :, 0] for x in seqs(3, 2, H, 1, d, BF))
    g = decays(H)
    slots = torch.tensor([N - 1, 0], dtype=torch.int32, device="cuda")
    S = torch.zeros(2, H, d, d, device="cuda")
    o = vla.vla_decay_step(q, k, v, g, pool, slots=slots, check=True)
    assert torch.equal(o, vla.vla_decay_step(q, k, v, g, S, check=True))
    assert torch.equal(pool[[N - 1, 0]], S) and not pool[1:N - 1].any()
    vla.vla_state_store(S, codes, scales, slots, check=True)
    assert torch.equal(vla.vla_state_load(codes, scales, slots, check=True).cpu(), R.store(S, 8)[0])
    assert not codes[1:N - 1].any()


def test_serving_calls_in_a_graph():
    """Step, store and load captured once and replayed: each replay goes one token on."""
    B, H, d = 3, 2, 96
    q, k, v = seqs(3, B, H, 4, d, BF, seed=6)
    g = decays(H)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool = torch.zeros(5, H, d, d, device="cuda")
    codes, scales = vla.vla_state_cache(3, (H, d, d), 8)
    x = [torch.empty(B, H, d, dtype=BF, device="cuda") for _ in range(3)]
    vla.vla_decay_step(*(s[:, :, 0] for s in (q, k, v)), g, pool.clone(), slots=slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = vla.vla_decay_step(*x, g, pool, 0.3, slots=slots)
        vla.vla_state_store(pool[2:], codes, scales)
        back = vla.vla_state_load(codes, scales)
    pool.zero_()
    outs = []
    for t in range(4):
        for a, s in zip(x, (q, k, v)):
            a.copy_(s[:, :, t])
        graph.replay()
        outs.append(o.clone())
        assert torch.equal(back.cpu(), R.store(pool[2:], 8)[0])
    check_forward(q, k, v, g, 0.3, None, None, (torch.stack(outs, 2), pool[slots.long()]))


# ---- layer norm of the readout ------------------------------------------------------------------------------------

NORMS = [(1, 1, 1, 32), (2, 3, 5, 64), (1, 2, 127, 96), (2, 2, 128, 128), (3, 5, 129, 96), (1, 4, 600, 32)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("weights", ["none", "heads", "shared", "no bias"])
@pytest.mark.parametrize("B,H,T,d", NORMS)
def test_head_norm(B, H, T, d, weights, dtype):
    x, dy = seqs(2, B, H, T, d, dtype, seed=T)
    x = (x.float() * 2 + 3).to(dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    shape = (d,) if weights == "shared" else (H, d)
    w = None if weights == "none" else torch.randn(shape, generator=gen, device="cuda")
    b = None if weights in ("none", "no bias") else torch.randn(shape, generator=gen, device="cuda")
    eps = 1e-5
    y, (mean, rstd) = vla.vla_head_norm(x, w, b, eps)
    ry, rm, rr = R.norm(x, w, b, eps)
    # fp32: a mean of d values, its differences, their squares' mean, an rsqrt (2 ulp) and three more roundings
    peak = x.double().abs().amax(-1).cpu()
    e = (d + 16) * R.U
    R.assert_within(mean, rm, e * peak, "mean")
    # a difference is off by e peak: the variance by 2 e peak / sigma and its own d roundings, rstd by half of that
    off = e * (1 + peak * rr)
    R.assert_within(rstd, rr, off * rr, "rstd")
    n = R.norm(x, None, None, eps)[0]
    wa = torch.ones(d, dtype=torch.float64) if w is None else w.double().abs().cpu()
    wa = wa.view(1, -1 if wa.dim() == 2 else 1, 1, d)
    by = ((off[..., None] * (n.abs() + 1)) * wa + 4 * R.U * ry.abs() + 2 * R.U * (n.abs() * wa))
    R.assert_within(y, ry, by + (R.HALF[dtype] * (ry.abs() + by) if dtype == BF else 0) + 1e-30, "y")
    dx, dw, db = vla.vla_head_norm_backward(dy, x, (mean, rstd), w)
    rdx, rdw, rdb, mdw, mdb, n, _ = R.norm_grads(dy, x, w, eps)
    rows = B * T * (H if weights == "shared" else 1)
    # n carries the statistics' error; then products and a sum over the rows
    en = float((off[..., None] * (n.abs() + 1)).max())
    assert dw.shape == shape and db.shape == shape
    R.assert_within(db, rdb, (rows + 8) * R.U * mdb + 1e-30, "db")
    R.assert_within(dw, rdw, (rows + 8) * R.U * mdw + en * mdb + 1e-30, "dw")
    gm = (dy.double().abs().cpu() * wa)
    top = gm.amax(-1, keepdim=True) * (1 + n.abs().amax(-1, keepdim=True)) ** 2
    bx = rr[..., None] * top * (3 * en + (2 * d + 16) * R.U)
    R.assert_within(dx, rdx, bx + (R.HALF[dtype] * (rdx.abs() + bx) if dtype == BF else 0) + 1e-30, "dx")


def test_head_norm_in_token_order_and_in_place():
    B, H, T, d = 2, 3, 140, 96
    x, dy = seqs(2, B, H, T, d, BF, seed=2)
    w, b = torch.randn(H, d, device="cuda"), torch.randn(H, d, device="cuda")
    y, stats = vla.vla_head_norm(x, w, b)
    rows = torch.empty(B, T, H, d, dtype=BF, device="cuda").transpose(1, 2)
    y2, _ = vla.vla_head_norm(x.transpose(1, 2).contiguous().transpose(1, 2), w, b, out=rows)
    assert y2 is rows and torch.equal(y, y2)
    dx, dw, db = vla.vla_head_norm_backward(dy, x, stats, w)
    again = vla.vla_head_norm_backward(dy, x, stats, w, out=dy)
    assert again[0] is dy and all(torch.equal(p, r) for p, r in zip((dx, dw, db), again))
    y3, _ = vla.vla_head_norm(x, w, b, out=x)
    assert y3 is x and torch.equal(y, x)


def test_head_norm_of_a_constant_row():
    """No spread: rstd = 1 / sqrt(eps), y = bias; a shift of all values changes nothing."""
    x = torch.full((1, 2, 3, 64), 5.0, device="cuda")
    b = torch.randn(2, 64, device="cuda")
    y, (mean, rstd) = vla.vla_head_norm(x, None, b, 1e-4)
    assert torch.equal(y, b[None, :, None].expand_as(y)) and (mean == 5).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=2.0 ** -22)


def test_head_norm_gradients_against_differences():
    B, H, T, d = 1, 2, 7, 32
    x, dy = (s.double() for s in seqs(2, B, H, T, d, F32, seed=5))
    w = torch.randn(H, d, device="cuda")
    xf, dyf = x.float(), dy.float()
    _, stats = vla.vla_head_norm(xf, w, None, 1e-3)
    dx, dw, db = vla.vla_head_norm_backward(dyf, xf, stats, w)
    loss = lambda x, w: float((R.norm(x, w, None, 1e-3)[0] * dyf.double().cpu()).sum())  # noqa: E731
    for i in range(3):
        gen = torch.Generator(device="cuda").manual_seed(i)
        sx = torch.randn(x.shape, generator=gen, device="cuda").double()
        h = 1e-4
        diff = (loss(xf.double() + h * sx, w) - loss(xf.double() - h * sx, w)) / (2 * h)
        want = float((dx.double() * sx).sum())
        # h^2 times third derivatives, which are below 100 per row here, and fp32 in dx
        assert abs(diff - want) <= 100 * h * h * B * H * T * d + 1e-5 * float((dx.double() * sx).abs().sum())
        sw = torch.randn(w.shape, generator=gen, device="cuda")
        diff = loss(xf, w + sw) - loss(xf, w)  # linear in w
        assert abs(diff - float((dw.double() * sw.double()).sum())) <= 1e-5 * float((dw.abs().double() * sw.abs()).sum() + 1)


# ---- quantised cache of states ------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("B,shape", [(1, (32,)), (3, (5, 64)), (2, (3, 96, 96)), (5, (2, 128, 128)), (4, (7, 32, 32))])
def test_store_and_load(B, shape, bits):
    gen = torch.Generator(device="cuda").manual_seed(B)
    N = B + 3
    x = torch.randn(B, *shape, generator=gen, device="cuda") * torch.exp(3 * torch.randn(B, *shape[:-1], 1, generator=gen, device="cuda"))
    x[0].view(-1)[:32] = 0
    codes, scales = vla.vla_state_cache(N, shape, bits)
    slots = torch.randperm(N, generator=gen, device="cuda")[:B].to(torch.int32)
    vla.vla_state_store(x, codes, scales, slots, check=True)
    want, scale = R.store(x, bits)
    assert torch.equal(vla.vla_state_load(codes, scales, slots, check=True).cpu(), want)
    assert torch.equal(scales[slots.long()].cpu(), scale)
    # within half a step of what was stored
    step = scale.repeat_interleave(32, -1).view(want.shape)
    assert ((want.double() - x.double().cpu()).abs() <= step.double() / 2 + 2.0 ** -22 * x.abs().double().cpu()).all()
    free = [i for i in range(N) if i not in slots.tolist()]
    assert not codes[free].any() and not scales[free].any()
    # repeats, a fresh state for a negative slot, all slots in order
    pick = torch.tensor([int(slots[0])] * 2 + [-1], dtype=torch.int32, device="cuda")
    y = vla.vla_state_load(codes, scales, pick, check=True).cpu()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[0]) and (y[2] == 0).all()
    every = vla.vla_state_load(codes, scales, check=True)
    assert torch.equal(every[slots.long()].cpu(), want)


@pytest.mark.parametrize("bits", [8, 4])
def test_codes_next_to_a_border(bits):
    """Values on, just below and just above the middle between two codes, at scales that are no powers of two."""
    top = 127 if bits == 8 else 7
    rows = []
    gen = torch.Generator().manual_seed(0)
    for i in range(64):
        s = float(torch.rand((), generator=gen) + 0.5) * 10.0 ** (i % 7 - 3)
        s = float(torch.tensor(s * top).float().double() / top)
        mid = (torch.randint(-top, top, (30,), generator=gen).double() + 0.5) * s
        mid = mid.float()
        mid[0::3] = torch.nextafter(mid[0::3], torch.tensor(float("inf")))
        mid[1::3] = torch.nextafter(mid[1::3], torch.tensor(float("-inf")))
        rows.append(torch.cat((torch.tensor([s * top, 0.0]).float(), mid)))
    x = torch.stack(rows).view(8, 8 * 32).view(8, 2, 128).cuda()
    codes, scales = vla.vla_state_cache(8, (2, 128), bits)
    vla.vla_state_store(x, codes, scales, check=True)
    want, scale = R.store(x, bits)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(vla.vla_state_load(codes, scales).cpu(), want)


@pytest.mark.parametrize("bits", [8, 4])
def test_extreme_groups(bits):
    """The largest and smallest values, and groups with NaN and Inf (read back as NaN, recorded)."""
    x = torch.ones(1, 6, 64, device="cuda")
    x[0, 0, :32] = 3.4e38
    x[0, 1, :32] = 1e-39
    x[0, 2, 5] = float("nan")
    x[0, 3, 40] = float("-inf")
    x[0, 4, :32] = 1e-30
    x[0, 4, 32:] = -0.0
    codes, scales = vla.vla_state_cache(1, (6, 64), bits)
    vla.vla_get_last_device_status()
    vla.vla_state_store(x, codes, scales)
    assert vla.vla_get_last_device_status()[0] == 5
    y = vla.vla_state_load(codes, scales).cpu()
    bad = torch.zeros(1, 6, 64, dtype=torch.bool)
    bad[0, 2, :32] = bad[0, 3, 32:] = True
    assert torch.isnan(y[bad]).all()
    clean = torch.where(bad, torch.zeros(()), x.cpu())
    assert torch.equal(y[~bad], R.store(clean, bits)[0][~bad])


def test_store_bad_slots():
    x = state_like(4, 2, 32, 1)
    codes, scales = vla.vla_state_cache(3, (2, 32, 32), 8)
    vla.vla_get_last_device_status()
    vla.vla_state_store(x, codes, scales, torch.tensor([2, -1, 2, 9], dtype=torch.int32, device="cuda"))
    assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_BAD_SLOT
    y = vla.vla_state_load(codes, scales).cpu()
    assert torch.equal(y[2], R.store(x[:1], 8)[0][0]) and not y[:2].any()
    z = vla.vla_state_load(codes, scales, torch.tensor([2, 3, -7], dtype=torch.int32, device="cuda")).cpu()
    assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_BAD_SLOT
    assert torch.equal(z[0], y[2]) and not z[1:].any()


def test_cache_of_the_recurrence_states():
    """vla_forward's S, A and z^key through the cache: parked, brought back, carried on."""
    B, H, T, d = 2, 3, 40, 64
    q, k, v, u = seqs(4, B, H, T, d, F32, seed=4)
    _, state = vla.vla_forward(q, k, v, u, check=True)
    back = []
    for x in state:
        codes, scales = vla.vla_state_cache(B, tuple(x.shape[1:]), 8)
        vla.vla_state_store(x, codes, scales, check=True)
        back.append(vla.vla_state_load(codes, scales, check=True))
        assert torch.equal(back[-1].cpu(), R.store(x, 8)[0])
    vla.vla_forward(q, k, v, u, state=tuple(back), check=True)


# ---- together -----------------------------------------------------------------------------------------------------

def test_training_step_together():
    """Scan, norm, loss, the norm's and the scan's gradients, against fp64 autograd of the definitions."""
    B, H, T, d = 2, 3, 100, 64
    q, k, v, dy = seqs(4, B, H, T, d, F32, seed=21)
    g = torch.tensor([-0.01, -0.1, -1.0], device="cuda")
    w = torch.rand(H, d, device="cuda") + 0.5
    eps = 0.1
    o, S = vla.vla_decay_forward(q, k, v, g, 0.2)
    y, stats = vla.vla_head_norm(o, w, None, eps)
    do, dw, _ = vla.vla_head_norm_backward(dy, o, stats, w)
    (dq, dk, dv), _ = vla.vla_decay_backward(q, k, v, g, 0.2, None, do)
    leaves = [x.double().cpu().requires_grad_() for x in (q, k, v, w)]
    t = torch.arange(T)
    D = torch.where(t[:, None] >= t, torch.exp(g.double().cpu()[:, None, None] * (t[:, None] - t).clamp(min=0)), 0.0)
    ro = 0.2 * ((leaves[0] @ leaves[1].transpose(-1, -2)) * D) @ leaves[2]
    rn = (ro - ro.mean(-1, keepdim=True)) / torch.sqrt(ro.var(-1, correction=0, keepdim=True) + eps)
    loss = (rn * leaves[3][None, :, None] * dy.double().cpu()).sum()
    ref = torch.autograd.grad(loss, leaves)
    for name, x, r in zip("qkvw", (dq, dk, dv, dw), ref):
        # fp32 through four operators, each within about (T + 2 d) u of its magnitudes, which cancel by less than 10
        assert float((x.double().cpu() - r).norm() / r.norm()) <= 40 * (T + 2 * d) * R.U, name


def test_serving_together():
    """Prompt, park in 8 bits, resume in another row, next tokens over a pool: each step from the stored state."""
    B, H, T, d = 3, 2, 80, 128
    q, k, v = seqs(3, B, H, T, d, BF, seed=31)
    g = torch.tensor([-0.02, -0.2], device="cuda")
    n = torch.tensor([80, 33, 0], dtype=torch.int32, device="cuda")
    _, S = vla.vla_decay_forward(q, k, v, g, 0.1, lengths=n, check=True)
    codes, scales = vla.vla_state_cache(6, (H, d, d))
    at = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    vla.vla_state_store(S, codes, scales, at, check=True)
    pool = torch.zeros(4, H, d, d, device="cuda")
    rows = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    pool[rows.long()] = vla.vla_state_load(codes, scales, at, check=True)
    parked = R.store(S, 8)[0]
    q1, k1, v1 = seqs(3, B, H, 2, d, BF, seed=32)
    o = torch.stack([vla.vla_decay_step(q1[:, :, t], k1[:, :, t], v1[:, :, t], g, pool, 0.1, slots=rows, check=True)
                     for t in range(2)], 2)
    check_forward(q1, k1, v1, g, 0.1, parked, None, (o, pool[rows.long()]))
