"""fp64 forms of the operators in include/vla_layer.h for the tests, from their
definitions, a token or a group at a time (torch on the CPU), and the bounds on
what the kernels may be off.

Bounds are elementwise. M, the same sum taken over the terms' magnitudes, scales
every rounding that a term goes through on the way; u = 2^-24.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def decay(q, k, v, g, scale=1.0, state=None, lengths=None):
    """(o, S) of the recurrence, token by token; inputs of any type, [B, H, T, d]."""
    q, k, v, g = (x.double().cpu() for x in (q, k, v, g))
    B, H, T, d = q.shape
    lam = torch.exp(g)[None, :, None, None]
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if state is None else state.double().cpu().clone()
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    o = torch.zeros(B, H, T, d, dtype=torch.float64)
    for t in range(T):
        on = t < n
        if not on.any():
            break
        S[on] = lam * S[on] + v[on, :, t, :, None] * k[on, :, t, None, :]
        o[on, :, t] = scale * torch.einsum("bhij,bhj->bhi", S[on], q[on, :, t])
    return o, S


def decay_grads(q, k, v, g, scale, state, do, dS, lengths=None):
    """(dq, dk, dv, dS0) by the reverse recurrence, token by token."""
    q, k, v, g, do = (x.double().cpu() for x in (q, k, v, g, do))
    B, H, T, d = q.shape
    lam = torch.exp(g)[None, :, None, None]
    zero = torch.zeros(B, H, d, d, dtype=torch.float64)
    S = zero.clone() if state is None else state.double().cpu().clone()
    R = zero.clone() if dS is None else dS.double().cpu().clone()
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    dq, dk, dv = (torch.zeros(B, H, T, d, dtype=torch.float64) for _ in range(3))
    for t in range(T):
        on = t < n
        S[on] = lam * S[on] + v[on, :, t, :, None] * k[on, :, t, None, :]
        dq[on, :, t] = scale * torch.einsum("bhij,bhi->bhj", S[on], do[on, :, t])
    for t in reversed(range(T)):
        on = t < n
        R[on] = R[on] + scale * do[on, :, t, :, None] * q[on, :, t, None, :]
        dk[on, :, t] = torch.einsum("bhij,bhi->bhj", R[on], v[on, :, t])
        dv[on, :, t] = torch.einsum("bhij,bhj->bhi", R[on], k[on, :, t])
        R[on] = lam * R[on]
    return dq, dk, dv, R


def gamma(T, d, g):
    """Roundings a term of a decayed sum can meet in fp32: the dot product's d,
    the sums over the tokens and over the state's columns (T + d), and its decay.
    A power of it comes from one exp (within 2 ulp) of a rounded angle, which is
    |g| n u off, and from at most T / 32 products of such powers."""
    fin = g[torch.isfinite(g)].abs()
    gmax = float(fin.max()) if fin.numel() else 0.0
    # a term whose decay's angle is over 100 is below 2^-144 of the others
    return (T + 2 * d + 8 + 6 * (T // 32 + 2) + min(gmax * T, 100.0)) * U


def seq_bound(ref, mag, dtype, T, d, g):
    """Output rows: fp32 sums; for bf16 the pair products and the state are
    rounded to bf16 on their way (each term meets one of them) and so is the
    result."""
    e = gamma(T, d, g) * mag
    if dtype == torch.bfloat16:
        e = e + HALF[dtype] * (1.01 * mag + ref.abs())
    return e + 1e-30


def state_bound(mag, dtype, T, d, g):
    """States: fp32 sums; bf16 inputs are decayed in two bf16 parts, whose rest
    is 2^-16 of a term."""
    return (gamma(T, d, g) + (2.0 ** -16 if dtype == torch.bfloat16 else 0.0)) * mag + 1e-30


def assert_within(x, ref, bound, what):
    x = x.detach().double().cpu()
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    assert torch.isfinite(x).all(), f"{what}: not finite"
    over = (x - ref).abs() / bound
    if over.numel():
        worst = float(over.max())
        assert worst <= 1.0, f"{what}: {worst:.3g} of the bound at {torch.nonzero(over == over.max())[0].tolist()}"


def norm(x, w, b, eps):
    x = x.double().cpu()
    H, d = x.shape[1], x.shape[3]
    per = lambda p, e: torch.full((1, 1, 1, d), e, dtype=torch.float64) if p is None else p.double().cpu().view(
        1, -1 if p.dim() == 2 else 1, 1, d)  # noqa: E731
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = 1 / torch.sqrt((c * c).mean(-1) + eps)
    return c * rstd[..., None] * per(w, 1.0) + per(b, 0.0), mean, rstd


def norm_grads(dy, x, w, eps):
    """(dx, dw, db, magnitudes of the sums dw and db)"""
    dy, x = dy.double().cpu(), x.double().cpu()
    d = x.shape[3]
    _, mean, rstd = norm(x, None, None, eps)
    n = (x - mean[..., None]) * rstd[..., None]
    g = dy * (1.0 if w is None else w.double().cpu().view(1, -1 if w.dim() == 2 else 1, 1, d))
    dx = rstd[..., None] * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    dims = (0, 1, 2) if w is not None and w.dim() == 1 else (0, 2)
    return dx, (dy * n).sum(dims), dy.sum(dims), (dy * n).abs().sum(dims), dy.abs().sum(dims), n, rstd


def store(x, bits):
    """Values a cache gives back for x: codes times scales, and the scales."""
    top = 127 if bits == 8 else 7
    y = x.double().cpu().unflatten(-1, (-1, 32))
    scale = (y.abs().amax(-1) / top).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros(()), scale)
    s = scale.double()[..., None]
    c = torch.where(s > 0, torch.round(y / torch.where(s > 0, s, torch.ones((), dtype=torch.float64))), 0.0)
    c = c.clamp(-top, top)
    return (c.float() * scale[..., None]).flatten(-2), scale
