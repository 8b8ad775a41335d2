"""The gated delta rule on the GPU where its numbers are at their ends: results that are rounded to bf16, heads that
grow."""
import pytest
import torch

import delta_ref as R
import sherman_morrison_memory_gb300 as vla
from test_delta_gpu import BF, F32, gates, inputs
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
