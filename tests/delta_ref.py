"""fp64 forms of the gated delta rule and of the norm and rotation of queries and
keys for the tests, from their definitions (torch on the CPU), and the bounds on
what the kernels may be off.

fp32 results are held normwise, a head at a time. Where keys have length 1 at
most, 0 <= beta <= 1 and decays are not above 1, a token's update is a contraction
of every row of the state, so that roundings add up but do not grow. A value meets
one addition for every 16 coordinates of a product (the tensor cores cut those
off, by 2^-23 at most), and with every chunk of 32 tokens that it lives through the
product with the decay and the sum.

bf16 results are held element by element: half a step for the result, and for
each term that meets one rounding on its way half a step of it.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CHUNK, BLOCK = 32, 64  # tokens whose pairs a bf16 call takes together: forward, gradients


def roundings(T, d):
    """Of 2^-24 each, that a value of an fp32 result meets one after another."""
    return 2 * (d // 16) + 16 + 3 * (T // CHUNK + 1)


def _in(x):
    return None if x is None else x.detach().double().cpu()


def delta(q, k, v, g, beta, scale=1.0, state=None, lengths=None):
    """(o, S, magnitude of o's terms that are rounded once) of the recurrence, token by token."""
    q, k, v, g, beta, state = (_in(x) for x in (q, k, v, g, beta, state))
    B, H, T, d = q.shape
    g = torch.zeros(B, H, T, dtype=torch.float64) if g is None else g
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if state is None else state.clone()
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    o, mag = torch.zeros(B, H, T, d, dtype=torch.float64), torch.zeros(B, H, T, d, dtype=torch.float64)
    # |S| as the chunk finds it and |u_j| |k_j . q_t| of its tokens, decayed
    for t in range(T):
        on = (t < n)[:, None, None, None]
        if t % CHUNK == 0:
            start, near, us, ks = S.abs(), torch.ones(B, H, 1, dtype=torch.float64), [], []
        a = torch.exp(g[:, :, t])[..., None, None]
        D = a * S
        u = beta[:, :, t, None] * (v[:, :, t] - (D @ k[:, :, t, :, None])[..., 0])
        S = torch.where(on, D + u[..., :, None] * k[:, :, t, None, :], S)
        near = near * a[..., 0]
        us, ks = [x * a[..., 0] for x in us] + [u.abs()], ks + [k[:, :, t]]
        ot = scale * (S @ q[:, :, t, :, None])[..., 0]
        m = near * (start @ q[:, :, t, :, None].abs())[..., 0]
        m = m + sum(x * (y * q[:, :, t]).sum(-1, keepdim=True).abs() for x, y in zip(us, ks))
        o[:, :, t] = torch.where(on[..., 0], ot, 0.0)
        mag[:, :, t] = torch.where(on[..., 0], abs(scale) * m, 0.0)
    return o, S, mag


def delta_grads(q, k, v, g, beta, scale, state, do, dS, lengths=None):
    """dq, dk, dv, dg, dbeta, dS0 by the reverse recurrence, the magnitudes of dq's and dk's terms that are rounded
    once, and |R k| |e| of dbeta's scalar products."""
    q, k, v, g, beta, state, do, dS = (_in(x) for x in (q, k, v, g, beta, state, do, dS))
    B, H, T, d = q.shape
    g = torch.zeros(B, H, T, dtype=torch.float64) if g is None else g
    n = torch.full((B,), T) if lengths is None else lengths.cpu().long().clamp(0, T)
    live = (torch.arange(T)[None] < n[:, None])[:, None]
    q, k, v, do = (torch.where(live[..., None], x, 0.0) for x in (q, k, v, do))
    g, beta = (torch.where(live, x, 0.0) for x in (g, beta))
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if state is None else state.clone()
    R = torch.zeros_like(S) if dS is None else dS.clone()
    Ds, es, Ss, starts, ends = [], [], [], [], [None] * (-(-T // BLOCK))
    for t in range(T):
        if t % BLOCK == 0:
            starts.append(S)
        D = torch.exp(g[:, :, t])[..., None, None] * S
        e = v[:, :, t] - (D @ k[:, :, t, :, None])[..., 0]
        S = D + (beta[:, :, t, None] * e)[..., :, None] * k[:, :, t, None, :]
        Ds.append(D), es.append(e), Ss.append(S)
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    dg, db, mb = (torch.zeros_like(g) for _ in range(3))
    for t in reversed(range(T)):
        if t == T - 1 or (t + 1) % BLOCK == 0:
            ends[t // BLOCK] = R
        D, e, S = Ds[t], es[t], Ss[t]
        dq[:, :, t] = scale * (do[:, :, t, None, :] @ S)[..., 0, :]
        R = R + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
        du = (R @ k[:, :, t, :, None])[..., 0]
        db[:, :, t] = (du * e).sum(-1)
        mb[:, :, t] = du.norm(dim=-1) * e.norm(dim=-1)
        dv[:, :, t] = beta[:, :, t, None] * du
        dk[:, :, t] = ((beta[:, :, t, None] * e)[..., None, :] @ R - dv[:, :, t, None, :] @ D)[..., 0, :]
        R = R - dv[:, :, t, :, None] * k[:, :, t, None, :]
        dg[:, :, t] = (R * D).sum((-1, -2))
        R = torch.exp(g[:, :, t])[..., None, None] * R
    mq, mk = torch.zeros_like(q), torch.zeros_like(q)
    for m, (S0, R1) in enumerate(zip(starts, ends)):
        at = slice(m * BLOCK, min(T, (m + 1) * BLOCK))
        G = g[:, :, at].clamp(min=-300).cumsum(-1)  # exp(-300) is nothing beside these bounds
        w = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0)).tril(-1)
        u = beta[:, :, at, None].abs() * torch.stack(es[at], 2).abs()
        near, far = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None]
        pairs = w * (dv[:, :, at].abs() @ u.transpose(-1, -2))
        mq[:, :, at] = abs(scale) * near * (do[:, :, at].abs() @ S0.abs())
        mk[:, :, at] = (far * (u @ R1.abs()) + near * (dv[:, :, at].abs() @ S0.abs()) + pairs @ k[:, :, at].abs()
                        + pairs.transpose(-1, -2) @ k[:, :, at].abs())
    zero = lambda x: torch.where(live if x.dim() == 3 else live[..., None], x, 0.0)  # noqa: E731
    return (zero(dq), zero(dk), dv, zero(dg), zero(db), R), (mq, mk, zero(mb))


def assert_normwise(x, ref, limit, what):
    """x of ref, a head (the first two dimensions) at a time, in the 2-norm."""
    x = x.detach().double().cpu()
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    assert torch.isfinite(x).all(), f"{what}: not finite"
    if not x.numel():
        return
    off = (x - ref).flatten(2).norm(dim=-1)
    size = ref.flatten(2).norm(dim=-1)
    worst = float((off / size.clamp(min=1e-30)).max())
    assert bool((off <= limit * size).all()), f"{what}: {worst:.3g} of the result, limit {limit:.3g}"


def assert_rounded(x, ref, mag, T, what):
    """A bf16 result: its own rounding, one of each term, and fp32 sums."""
    x = x.detach().double().cpu()
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    assert torch.isfinite(x).all(), f"{what}: not finite"
    if not x.numel():
        return
    size = ref.flatten(2).abs().amax(-1)[..., None, None] + mag.flatten(2).amax(-1)[..., None, None]
    bound = 2.0 ** -8 * (ref.abs() + 1.01 * mag) + 4 * roundings(T, ref.shape[-1]) * U * size + 1e-30
    worst = float(((x - ref).abs() / bound).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def qk(x, w, unit, eps, freqs, pos):
    """y of a differentiable x in 64 bits, and rstd; x on the CPU, [B, H, T, d]."""
    d = x.shape[-1]
    rstd = 1 / torch.sqrt((x * x).sum(-1) / (1 if unit else d) + eps)
    z = x * rstd[..., None]
    if w is not None:
        z = z * (w if w.dim() == 1 else w[:, None])
    if freqs is None:
        return z, rstd
    m = freqs.shape[0]
    a = (pos.double()[..., None] * freqs)[:, None]
    lo, hi = z[..., :m], z[..., m:2 * m]
    return torch.cat((lo * torch.cos(a) - hi * torch.sin(a), hi * torch.cos(a) + lo * torch.sin(a), z[..., 2 * m:]), -1), rstd
