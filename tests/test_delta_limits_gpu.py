"""The gated delta rule on the GPU where its numbers are at their ends: results that are rounded to bf16, heads that
grow, decays that leave next to nothing, states of one sign, strong corrections; and every number of rows that a block
may have."""
import math

import pytest
import torch

import delta_ref as R
import sherman_morrison_memory_gb300 as vla
from test_delta_gpu import BF, F32, check_backward, check_forward, gates, inputs
from test_layer_gpu import state_like

pytestmark = pytest.mark.gpu


# ---- the definition, and the sizes of what a block of tokens adds up -------------------------------------------------

def by_blocks(q, k, v, g, beta, scale, do, state=None, dS=None):
    """By the definition in 64 bits: dq, dk, dv, dg, dbeta, dS0; the magnitudes of dk's terms that have dV in them; the
    magnitudes of all terms of dq, dk and dv, as a block of 64 tokens has them (factors as large as its heads grow); and
    |R k| |e| of dbeta's scalar products."""
    q, k, v, g, beta, do = (x.double().cpu() for x in (q, k, v, g, beta, do))
    B, H, T, d = q.shape
    S, G = (torch.zeros(B, H, d, d, dtype=torch.float64) if x is None else x.double().cpu() for x in (state, dS))
    Ds, es, Ss, starts, ends = [], [], [], [], {}
    for t in range(T):
        if t % R.BLOCK == 0:
            starts.append(S)
        D = torch.exp(g[:, :, t])[..., None, None] * S
        e = v[:, :, t] - (D @ k[:, :, t, :, None])[..., 0]
        S = D + (beta[:, :, t, None] * e)[..., :, None] * k[:, :, t, None, :]
        Ds.append(D), es.append(e), Ss.append(S)
    dq, dk, dv, size_v = (torch.zeros_like(q) for _ in range(4))
    dg, db, mb = (torch.zeros_like(g) for _ in range(3))
    for t in reversed(range(T)):
        if t == T - 1 or (t + 1) % R.BLOCK == 0:
            ends[t // R.BLOCK] = G
        D, e, b = Ds[t], es[t], beta[:, :, t, None]
        dq[:, :, t] = scale * (do[:, :, t, None, :] @ Ss[t])[..., 0, :]
        G = G + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
        du = (G @ k[:, :, t, :, None])[..., 0]
        size_v[:, :, t] = b * (G.abs() @ k[:, :, t, :, None].abs())[..., 0]
        db[:, :, t], mb[:, :, t] = (du * e).sum(-1), du.norm(dim=-1) * e.norm(dim=-1)
        dv[:, :, t] = b * du
        dk[:, :, t] = ((b * e)[..., None, :] @ G - dv[:, :, t, None, :] @ D)[..., 0, :]
        G = G - dv[:, :, t, :, None] * k[:, :, t, None, :]
        dg[:, :, t] = (G * D).sum((-1, -2))
        G = torch.exp(g[:, :, t])[..., None, None] * G
    by_dv, size_q, size_k = (torch.zeros_like(q) for _ in range(3))
    for m, S0 in enumerate(starts):
        at = slice(m * R.BLOCK, min(T, (m + 1) * R.BLOCK))
        c = g[:, :, at].clamp(min=-300).cumsum(-1)  # exp(-300) is nothing beside these bounds
        w = torch.exp((c[..., :, None] - c[..., None, :]).tril()).tril()
        u = beta[:, :, at, None] * torch.stack(es[at], 2).abs()
        near, far = torch.exp(c)[..., None], torch.exp(c[..., -1:] - c)[..., None]
        qa, ka, oa, va = (x[:, :, at].abs() for x in (q, k, do, dv))
        M, X = w * (va @ u.transpose(-1, -2)), abs(scale) * w * (oa @ u.transpose(-1, -2))
        by_dv[:, :, at] = near * (va @ S0.abs()) + M @ ka + M.transpose(-1, -2) @ ka
        size_q[:, :, at] = abs(scale) * near * (oa @ S0.abs()) + X @ ka
        size_k[:, :, at] = by_dv[:, :, at] + far * (u @ ends[m].abs()) + X.transpose(-1, -2) @ qa
    return (dq, dk, dv, dg, db, G), by_dv, (size_q, size_k, size_v), mb


def assert_by_token(x, ref, size, rounds, what, once=0.0):
    """Each token on its own: fp32 sums of terms whose magnitudes are ``size``; a bf16 result rounded once, of terms in two
    parts (each within 2^-16 and without the products of the small ones), those in ``once`` of a value rounded to bf16."""
    x, dtype = x.detach().double().cpu(), x.dtype
    assert torch.isfinite(x).all(), f"{what}: not finite"
    bound = rounds * R.U * (size + ref.abs()).amax(-1, keepdim=True) + 1e-36
    if dtype == BF:
        bound = bound + 2.0 ** -8 * (ref.abs() + 1.01 * once) + 2.0 ** -14 * size
    worst = float(((x - ref).abs() / bound).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


# ---- bf16 results ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,d", [(1, 32), (20, 64), (64, 96), (50, 128), (65, 32), (150, 64), (200, 96), (140, 128)])
def test_bf16_results_are_rounded_once(T, d):
    """o, dq and dv are fp32 results up to their own rounding, and so is dk but for dv, which it takes as it was written."""
    B, H = 2, 3
    q, k, v, do = inputs(4, B, H, T, d, BF, seed=T + d)
    g, beta = gates(B, H, T)
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    n = 4 * R.roundings(T, d)
    ro, _, mag = R.delta(q, k, v, g, beta, 0.4, S0)
    o, _ = vla.vla_delta_forward(q, k, v, g, beta, 0.4, S0, check=True)
    assert_by_token(o, ro, mag, n, "o")
    ref, by_dv, size, _ = by_blocks(q, k, v, g, beta, 0.4, do, S0, dS)
    (dq, dk, dv), _, _ = vla.vla_delta_backward(q, k, v, g, beta, 0.4, S0, do, dS, check=True)
    assert_by_token(dq, ref[0], size[0], 2 * n, "dq")
    assert_by_token(dk, ref[1], size[1], 2 * n, "dk", by_dv)
    assert_by_token(dv, ref[2], size[2], 2 * n, "dv")


# ---- heads that grow ----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(33, 64), (64, 64), (64, 128), (192, 32), (192, 64), (192, 96), (192, 128)])
def test_growing_heads(T, d, dtype):
    """A factor of e^1.5 a token: of 32 tokens that is e^48, of the 64 that a bf16 call's gradients take together e^96, which
    float32 does not hold, of values so small that every result is finite."""
    B, H = 1, 2
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=T + d)
    v, do = (1e-10 * v.float()).to(dtype), (1e-5 * do.float()).to(dtype)
    beta = gates(B, H, T)[1]
    g = torch.full((B, H, T), 1.5, device="cuda")
    if T > 64:  # one block grows, the one behind it shrinks by as much
        g[:, :, :64], g[:, :, 128:] = 0.0, -1.5
    ro, rS, mag = R.delta(q, k, v, g, beta, 0.5)
    ref, by_dv, size, mb = by_blocks(q, k, v, g, beta, 0.5, do)
    assert all(float(x.abs().max()) < 1e38 for x in (ro, rS, *ref))
    # as where nothing grows (a rounding grows as what it is a rounding of does); the exponents of up to 96 are off by half a step
    n = 4 * R.roundings(T, d) + 2 * 96
    o, S = vla.vla_delta_forward(q, k, v, g, beta, 0.5, check=True)
    assert_by_token(o, ro, mag, n, "o")
    R.assert_normwise(S, rS, n * R.U, "S")
    (dq, dk, dv), (dg, db), dS0 = vla.vla_delta_backward(q, k, v, g, beta, 0.5, None, do, check=True)
    for name, x, r, s, once in zip(("dq", "dk", "dv"), (dq, dk, dv), ref, size, (0.0, by_dv, 0.0)):
        assert_by_token(x, r, s, 2 * n, name, once)
    R.assert_normwise(dS0, ref[5], 2 * n * R.U, "dS0")
    off = (db.double().cpu() - ref[4]).norm(dim=-1)
    assert torch.isfinite(db).all() and bool((off <= 2 * n * R.U * (ref[4].norm(dim=-1) + mb.norm(dim=-1))).all()), ("dbeta", off)
    terms = ((ro * do.double().cpu()).norm(dim=-1) + (v.double().cpu() * ref[2]).norm(dim=-1)).norm(dim=-1)
    off = (dg.double().cpu() - ref[3]).norm(dim=-1)
    assert torch.isfinite(dg).all() and bool((off <= 2 * n * R.U * (ref[3].norm(dim=-1) + 8 * terms)).all()), ("dg", off, terms)


# ---- decays that leave next to nothing ----------------------------------------------------------------------------

STRONG = {BF: -6.0, F32: -2.0}  # below it, dlog_decay is the sum of what the decay multiplies


def across(q, k, v, g, beta, scale, state, do, dS, dv):
    """What log_decay's gradient is a sum of, a token at a time, [B, H, T] each: the magnitudes of all terms that cross
    the decay, and the 2-norm of those with dV in them, which a bf16 call takes as it was written."""
    q, k, v, g, beta, do = (x.double().cpu() for x in (q, k, v, g, beta, do))
    B, H, T, d = q.shape
    S = state.double().cpu()
    starts, us = [], []
    for t in range(T):
        if t % R.BLOCK == 0:
            starts.append(S)
        S = torch.exp(g[:, :, t])[..., None, None] * S
        us.append(beta[:, :, t, None] * (v[:, :, t] - (S @ k[:, :, t, :, None])[..., 0]))
        S = S + us[t][..., :, None] * k[:, :, t, None, :]
    G, ends = dS.double().cpu(), {}
    for t in reversed(range(T)):
        if t == T - 1 or (t + 1) % R.BLOCK == 0:
            ends[t // R.BLOCK] = G
        G = torch.exp(g[:, :, t])[..., None, None] * (G + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
                                                      - dv[:, :, t, :, None] * k[:, :, t, None, :])
    size, once = torch.zeros_like(g), torch.zeros_like(g)
    late = lambda x, i: x.flip(i).cumsum(i).flip(i)  # noqa: E731
    for m, S0 in enumerate(starts):
        at = slice(m * R.BLOCK, min(T, (m + 1) * R.BLOCK))
        c = g[:, :, at].clamp(min=-256).cumsum(-1)
        n = c.shape[-1]
        w = torch.exp((c[..., :, None] - c[..., None, :]).tril()).tril(-1)
        near, far = torch.exp(c)[..., None], torch.exp(c[..., -1:] - c)[..., None]
        u = torch.stack(us[at], 2).abs()
        qa, ka, oa, va = (x[:, :, at].abs() for x in (q, k, abs(scale) * do, dv))
        R1, kk = ends[m].abs(), (k[:, :, at] @ k[:, :, at].transpose(-1, -2)).abs()
        qk = (q[:, :, at] @ k[:, :, at].transpose(-1, -2)).abs()
        # S0[x][y]: every token from t on; R1[x][y]: every one before t
        by_S = late((near * oa)[..., :, None] * qa[..., None, :], 2) * S0.abs()[:, :, None]
        by_R = (far * u)[..., :, None] * ka[..., None, :]
        by_R = (by_R.cumsum(2) - by_R) * R1[:, :, None]
        t = torch.arange(n)
        before = (t[None, :] < t[:, None]).double()                    # [t][j]: j before t
        pair = (w * kk)[:, :, None] * before[None, None, :, None, :]   # [t][i][j]
        by_V = (near * (ka @ S0.abs().transpose(-1, -2)))[:, :, None] + pair @ u[:, :, None]
        by_V = by_V * va[:, :, None] * (1 - before)[None, None, :, :, None]
        by_X = ((w * (oa @ u.transpose(-1, -2)) * qk)[:, :, None] * before[None, None, :, None, :]
                * (1 - before)[None, None, :, :, None]).sum((-1, -2))
        whole = torch.exp(c[..., -1:]) * (R1 * S0.abs()).sum((-1, -2))[..., None]
        size[:, :, at] = by_S.sum((-1, -2)) + by_R.sum((-1, -2)) + by_V.sum((-1, -2)) + by_X + whole
        once[:, :, at] = torch.sqrt((by_V ** 2).sum((-1, -2)))
    return size, once


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(40, 64), (64, 32), (130, 64), (130, 96), (100, 128)])
def test_gradients_of_strong_decays(T, d, dtype):
    """Heads of one decay from slow to total, and one with such tokens among slow ones: dlog_decay keeps its digits where
    the decay leaves little, and is 0 where it leaves nothing."""
    rates = [-0.01, -1.0, -5.0, -9.5, -10.5, -16.0, -20.0, -30.0, -80.0, -256.0, -1e4, float("-inf"), 0.0]
    B, H = 1, len(rates)
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=T + d)
    g = torch.tensor(rates, device="cuda")[None, :, None].repeat(B, 1, T)
    g[:, -1] = -0.02
    g[:, -1, 5::7], g[:, -1, 9::16], g[:, -1, 31::33] = -12.0, -25.0, float("-inf")
    beta = gates(B, H, T)[1]
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    got = vla.vla_delta_backward(q, k, v, g, beta, 0.4, S0, do, dS, check=True)
    (dx, (dg, db), dS0), held = got, [h for h, rate in enumerate(rates) if rate > -50]  # whose states float32 holds
    part = lambda x: x[:, held]  # noqa: E731
    check_backward(*map(part, (q, k, v, g, beta)), 0.4, *map(part, (S0, do, dS)), None,
                   (tuple(map(part, dx)), (part(dg), part(db)), part(dS0)))
    ref = R.delta_grads(q, k, v, g, beta, 0.4, S0, do, dS)[0]
    size, once = across(q, k, v, g, beta, 0.4, S0, do, dS, ref[2])
    dg, g = dg.double().cpu(), g.double().cpu()
    strong = g < STRONG[dtype]
    e = 2 * R.roundings(T, d) * R.U
    bound = e * size
    if dtype == BF:  # terms in two parts; dV's roundings, each within 2^-8 and as often up as down: six times their deviation
        bound = bound + 2.0 ** -14 * size + 6 * 2.0 ** -8 / math.sqrt(3) * once
    off = (dg - ref[3]).abs()
    assert bool((off <= bound + 1e-37)[strong].all()), float((off / (bound + 1e-37))[strong].max())
    assert (dg[g <= -256] == 0).all()
    limit = 0.1 if dtype == BF else 2e-3  # these bounds are far below the gradients themselves
    for h, rate in enumerate(rates):
        if -81 < rate < STRONG[dtype]:
            assert float(off[:, h].norm()) <= limit * float(ref[3][:, h].norm()), (rate, float(off[:, h].norm() / ref[3][:, h].norm()))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_strong_decays_of_padded_batches(d, dtype):
    """Strong and total decays at random among slow ones, without a state, in sequences of several lengths whose rows behind
    the end are NaN; and the same gate for all tokens, read from one value."""
    lengths, H, T = [130, 65, 64, 1], 2, 130
    B = len(lengths)
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=d)
    g, beta = gates(B, H, T)
    pick = torch.rand(B, H, T, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda")
    g = torch.where(pick < 0.2, -15.0, torch.where(pick < 0.25, float("-inf"), 0.05 * g.clamp(min=-4.0)))
    none, dS = torch.zeros(B, H, d, d, device="cuda"), state_like(B, H, d, 2)
    for x in (g, beta, do):
        for b, n in enumerate(lengths):
            x[b, :, n:] = float("nan")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    dg = vla.vla_delta_backward(q, k, v, g, beta, 0.4, None, do, dS, lengths=n, check=True)[1][0].double().cpu()
    e = 2 * R.roundings(T, d) * R.U
    for b, m in enumerate(lengths):
        x = [y[b:b + 1, :, :m] for y in (q, k, v, g, beta)]
        ref = R.delta_grads(*x, 0.4, none[b:b + 1], do[b:b + 1, :, :m], dS[b:b + 1])[0]
        size, once = across(*x, 0.4, none[b:b + 1], do[b:b + 1, :, :m], dS[b:b + 1], ref[2])
        bound = e * size
        if dtype == BF:
            bound = bound + 2.0 ** -14 * size + 6 * 2.0 ** -8 / math.sqrt(3) * once
        off, strong = (dg[b:b + 1, :, :m] - ref[3]).abs(), x[3].cpu() < STRONG[dtype]
        assert bool((off <= bound + 1e-37)[strong].all()), (b, off, bound)
        assert (dg[b:b + 1, :, :m][x[3].cpu() == float("-inf")] == 0).all() and (dg[b, :, 0] == 0).all() and (dg[b, :, m:] == 0).all()
    flat = torch.full((1,), -9.0, device="cuda").expand(B, H, T)
    args = (q, k, v, flat, beta.nan_to_num(0), 0.4, None, do.nan_to_num(0), dS)
    a = vla.vla_delta_backward(*args, lengths=n, check=True)
    b = vla.vla_delta_backward(*args[:3], flat.contiguous(), *args[4:], lengths=n, check=True)
    assert torch.equal(a[1][0], b[1][0]) and torch.equal(a[0][1], b[0][1])


# ---- states of one sign -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T", [64, 96])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_sums_of_one_sign(d, T):
    """A state and keys of one sign, of which one token takes what it reads: the sum over d coordinates is cut off by
    2^-23 at most with every 16 of them, always towards zero, and by nothing else."""
    B, H = 1, 3
    gen = torch.Generator(device="cuda").manual_seed(d)
    S0 = 1 + torch.rand(B, H, d, d, generator=gen, device="cuda")
    k_in = 1 + torch.rand(B, H, T, d, generator=gen, device="cuda")
    k_in = (k_in / k_in.norm(dim=-1, keepdim=True)).to(BF)
    v, beta = torch.zeros(B, H, T, d, dtype=BF, device="cuda"), torch.zeros(B, H, T, device="cuda")
    beta[:, :, 7] = 1
    S = vla.vla_delta_forward(k_in, k_in, v, None, beta, 1.0, S0, check=True)[1].double().cpu()
    x, k = S0.double().cpu(), k_in.double().cpu()[:, :, 7]
    read = (x @ k[..., None])[..., 0]
    want = x - read[..., :, None] * k[..., None, :]
    # d / 16 sums cut off, and half a step each of their joining, of E, of the two ends of the product and of the new state
    bound = (2 * (d // 16) + 6) * R.U * read[..., :, None] * k[..., None, :] + 2 * R.U * x
    # ... and back: without a gradient of o the state's gradient goes the same way
    dS0 = vla.vla_delta_backward(k_in, k_in, v, None, beta, 1.0, None, v, S0, check=True)[2].double().cpu()
    for name, y in (("S", S), ("dS0", dS0)):
        worst = float(((y - want).abs() / bound).max())
        assert worst <= 1.0, (name, worst)
        # what is cut off is between 0 and 2^-23 of a sum, a half of that in the mean
        mean = float(((y - want) / (R.U * read[..., :, None] * k[..., None, :])).mean())
        assert abs(mean) <= d // 16, (name, mean)


# ---- strong corrections -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d", [(64, 32), (100, 64), (129, 96), (200, 128)])
def test_corrections_beyond_one(T, d, dtype):
    """beta in (1, 2] on unit keys, and keys of length 1.4 with beta up to 1: the update still stretches nothing."""
    B, H = 2, 3
    q, k, v, do = inputs(4, B, H, T, d, dtype, seed=T)
    g, beta = gates(B, H, T)
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    check_forward(q, k, v, g, 1 + beta, 0.4, S0, more=4)
    check_backward(q, k, v, g, 1 + beta, 0.4, S0, do, dS, more=4)
    check_forward(q, k, v, None, torch.full_like(beta, 2.0), 0.4, S0, more=4)
    long = (1.4 * k.float()).to(dtype)
    check_forward(q, long, v, g, beta, 0.4, S0, more=4)
    check_backward(q, long, v, g, beta, 0.4, S0, do, dS, more=4)


# ---- rows of a block ----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_every_number_of_rows(d, dtype):
    """Calls of as many heads as give a block each number of rows of S that there is on the warp-level path: a head's bits
    are the same in all of them, and right."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most, T = (64 if d == 128 else d), 64 if dtype == BF else 70

    def rows_of(heads):  # the rule: halved while all blocks run at once
        rows = most
        while rows % 32 == 0 and heads * (d // (rows // 2)) <= sms:
            rows //= 2
        return rows

    counts = {rows_of(h): h for h in range(sms + 1, 0, -1)}  # the fewest heads of each
    assert set(counts) == {most >> i for i in range(3) if (most >> i) >= 16 and (i == 0 or (most >> (i - 1)) % 32 == 0)}
    H = max(counts.values())
    q, k, v, do = inputs(4, 1, H, T, d, dtype, seed=d)
    g, beta = gates(1, H, T)
    S0, dS = state_like(1, H, d, 1), state_like(1, H, d, 2)

    def call(n):
        x = [y[:, :n] for y in (q, k, v, do, g, beta, S0, dS)]
        o, S = vla.vla_delta_forward(*x[:3], *x[4:6], 0.3, x[6], check=True)
        grads, gg, dS0 = vla.vla_delta_backward(*x[:3], *x[4:6], 0.3, x[6], x[3], x[7], check=True)
        return (o, S, *grads, *gg, dS0)

    want = call(H)
    for n in counts.values():
        got = call(n)
        assert all(torch.equal(a[:, :n], b) for a, b in zip(want, got)), n
    part = lambda x: x[:, :H:max(1, H // 8)]  # noqa: E731
    check_forward(*map(part, (q, k, v, g, beta)), 0.3, part(S0), None, tuple(map(part, want[:2])))
    check_backward(*map(part, (q, k, v, g, beta)), 0.3, part(S0), part(do), part(dS), None,
                   (tuple(map(part, want[2:5])), tuple(map(part, want[5:7])), part(want[7])))
