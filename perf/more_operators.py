"""Cases of the operators of a layer whose heads correct their memories: the norm and position rotation of queries and
keys, and the gated delta rule over prompts, for training, and for single tokens.

``own`` false: the plain forms, in elementary torch operations. ``own`` true: the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64  # tokens that the plain form of the delta rule takes at a time
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a batch of prompts, the sizes of the benchmark's workload
        dict(name="delta_prompt_d96", kind="prompt", B=8, H=16, T=4096, d=96, dtype="bf16", rows="heads", state=False, ragged=False),
        # one long context: few heads, each a long chain
        dict(name="delta_long_d128", kind="prompt", B=1, H=32, T=32768, d=128, dtype="bf16", rows="tokens", state=False, ragged=False),
        # padded prompts of several lengths that continue earlier turns, fp32
        dict(name="delta_ragged_f32_d64", kind="prompt", B=5, H=8, T=1021, d=64, dtype="f32", rows="tokens", state=True, ragged=True),
        # gradients of a training step
        dict(name="delta_train_d64", kind="train", B=4, H=8, T=4096, d=64, dtype="bf16", rows="heads", state=False, ragged=False),
        # gradients through a carried state, projections in token order, odd length
        dict(name="delta_train_state_d128", kind="train", B=2, H=32, T=4095, d=128, dtype="bf16", rows="tokens", state=True, ragged=False),
        # a small fp32 model with padded sequences
        dict(name="delta_train_ragged_f32_d32", kind="train", B=3, H=5, T=777, d=32, dtype="f32", rows="heads", state=True, ragged=True),
        # one user's next token: latency
        dict(name="delta_step_one_d128", kind="step", B=1, H=32, d=128, dtype="bf16", slots=1),
        # a server's batch of next tokens over a pool of states
        dict(name="delta_step_pool_d96", kind="step", B=256, H=16, d=96, dtype="bf16", slots=300),
        # queries and keys of a long prompt, from the projection's order to the heads'
        dict(name="qk_prompt_d128", kind="qk", B=1, H=32, T=32768, d=128, dtype="bf16", rot=128, unit=False, weight="heads", train=False, rows="tokens", at="far"),
        # a training step: forward, then the gradients, with one weight for all heads
        dict(name="qk_train_d96", kind="qk", B=8, H=16, T=4096, d=96, dtype="bf16", rot=96, unit=False, weight="shared", train=True, rows="tokens", at="start"),
        # unit rows for a delta rule, half of each rotated, fp32, an odd length
        dict(name="qk_train_unit_f32_d64", kind="qk", B=3, H=8, T=1021, d=64, dtype="f32", rot=32, unit=True, weight="none", train=True, rows="heads", at="start"),
        # the next tokens of a batch, each at its own position: latency
        dict(name="qk_token_d128", kind="qk", B=64, H=32, T=1, d=128, dtype="bf16", rot=128, unit=False, weight="heads", train=False, rows="tokens", at="far"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "train", "step", "qk", "qk"])
    d = rng.choice([32, 64, 96, 128])
    H = rng.randint(1, 32)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = rng.choice(["heads", "tokens"])
    if kind == "step":
        B = _log(rng, 1, 128)
        return dict(kind=kind, B=B, H=H, d=d, dtype=dtype, slots=B + rng.randint(0, 40))
    T = _log(rng, 1, 16384)
    B = max(1, min(rng.randint(1, 8), (1 << 25) // (T * H * d)))
    if kind == "qk":
        return dict(kind=kind, B=B, H=H, T=T, d=d, dtype=dtype, rot=rng.choice([0, 16, d // 2, d, d]), unit=rng.random() < 0.4,
                    weight=rng.choice(["none", "shared", "heads"]), train=rng.random() < 0.6, rows=rows,
                    at=rng.choice(["start", "far"]))
    return dict(kind=kind, B=B, H=H, T=T, d=d, dtype=dtype, rows=rows, state=rng.random() < 0.5, ragged=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind, B, H, d, dt = case["kind"], case["B"], case["H"], case["d"], DT[case["dtype"]]
    in_order = case.get("rows") == "tokens"

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def sequence(T, unit=False, size=1.0):
        """[B, H, T, d]; "tokens": a view of a projection's output, [B, T, H, d] in memory."""
        x = normal(B, T, H, d) if in_order else normal(B, H, T, d)
        if unit:
            x /= torch.sqrt((x * x).sum(-1, keepdim=True))
        x = (x * size).to(dt)
        return x.transpose(1, 2) if in_order else x

    def gates(T):
        """Log decays and writing strengths [B, H, T] as a layer's projections give them: heads from slow to fast."""
        rate = torch.exp2(torch.linspace(-8, 0, H, device=dev))
        x, y = (normal(B, T, H) for _ in range(2))
        g, beta = -rate * torch.log1p(torch.exp(x)), 1 / (1 + torch.exp(-y))
        g, beta = g.transpose(1, 2), beta.transpose(1, 2)
        return (g, beta) if in_order else (g.contiguous(), beta.contiguous())

    s = dict(case)
    if kind in ("prompt", "train"):
        T = case["T"]
        s["q"], s["k"], s["v"] = sequence(T, unit=True), sequence(T, unit=True), sequence(T)
        s["g"], s["beta"] = gates(T)
        s["scale"] = d ** -0.5
        s["state"] = 0.3 * normal(B, H, d, d) if case["state"] else None
        if kind == "train":
            s["grad_o"] = sequence(T)
            s["grad_state"] = 0.3 * normal(B, H, d, d) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            n[0] = T
            s["lengths"] = n
    elif kind == "step":
        N = case["slots"]
        s["q"], s["k"], s["v"] = (sequence(1, unit=u)[:, :, 0] for u in (True, True, False))
        s["g"], s["beta"] = (x[:, :, 0].contiguous() for x in gates(1))
        s["scale"] = d ** -0.5
        s["pool"] = 0.3 * normal(N, H, d, d)
        s["slots"] = torch.randperm(N, generator=gen, device=dev)[:B].to(torch.int32)
    else:
        T, rot = case["T"], case["rot"]
        s["q"], s["k"] = sequence(T, size=3.0), sequence(T, size=0.5)
        shape = {"none": None, "shared": (d,), "heads": (H, d)}[case["weight"]]
        s["wq"], s["wk"] = (None if shape is None else 1 + 0.1 * normal(*shape) for _ in range(2))
        s["freqs"] = None
        if rot:
            s["freqs"] = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        s["positions"] = None
        if case["at"] == "far":  # each sequence goes on from its own place
            first = torch.randint(0, 1 << 20, (B, 1), generator=gen, device=dev, dtype=torch.int32)
            s["positions"] = first + torch.arange(T, device=dev, dtype=torch.int32)
        if case["train"]:
            s["grad_q"], s["grad_k"] = sequence(T), sequence(T)
    return s


def run(s):
    return (_own if own else _plain)(s)


# ---------------------------------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import sherman_morrison_memory_gb300 as vla

    kind = s["kind"]
    if kind == "prompt":
        o, S = vla.vla_delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["state"], lengths=s["lengths"])
        return {"o": o, "S": S}
    if kind == "train":
        (dq, dk, dv), (dg, dbeta), dS0 = vla.vla_delta_backward(
            s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["state"], s["grad_o"], s["grad_state"], lengths=s["lengths"])
        return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dS0": dS0}
    if kind == "step":
        o = vla.vla_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["scale"], slots=s["slots"])
        return {"o": o, "pool": s["pool"]}
    (yq, yk), stats = vla.vla_qk_norm(s["q"], s["k"], s["wq"], s["wk"], EPS, unit=s["unit"], freqs=s["freqs"], positions=s["positions"])
    got = {"yq": yq, "yk": yk}
    if s["train"]:
        (dq, dk), (dwq, dwk) = vla.vla_qk_norm_backward(s["grad_q"], s["grad_k"], s["q"], s["k"], stats, s["wq"], s["wk"],
                                                        unit=s["unit"], freqs=s["freqs"], positions=s["positions"])
        got.update(dq=dq, dk=dk)
        if s["wq"] is not None:
            got.update(dwq=dwq, dwk=dwk)
    return got


# ---------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------
def _plain(s):
    kind = s["kind"]
    if kind in ("prompt", "train"):
        return _plain_sequences(s)
    if kind == "step":
        at, q, k, v = s["slots"].long(), s["q"].float(), s["k"].float(), s["v"].float()
        S = s["pool"][at] * torch.exp(s["g"])[..., None, None]
        u = s["beta"][..., None] * (v - (S @ k[..., None])[..., 0])
        S = S + u[..., :, None] * k[..., None, :]
        s["pool"][at] = S
        return {"o": ((S @ q[..., None])[..., 0] * s["scale"]).to(s["q"].dtype), "pool": s["pool"]}
    turn = _turns(s)
    yq, rq = _plain_norm(s["q"], s["wq"], s["unit"], turn)
    yk, rk = _plain_norm(s["k"], s["wk"], s["unit"], turn)
    got = {"yq": yq, "yk": yk}
    if s["train"]:
        dq, dwq = _plain_norm_backward(s["grad_q"], s["q"], rq, s["wq"], s["unit"], turn)
        dk, dwk = _plain_norm_backward(s["grad_k"], s["k"], rk, s["wk"], s["unit"], turn)
        got.update(dq=dq, dk=dk)
        if s["wq"] is not None:
            got.update(dwq=dwq, dwk=dwk)
    return got


def _turns(s):
    """cos and sin [B, 1, T, rot / 2] of the tokens' angles (the angles in 64 bits), or None."""
    if s["freqs"] is None:
        return None
    pos = torch.arange(s["T"], device=s["q"].device)[None] if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None, :, None] * s["freqs"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, turn, sign):
    if turn is None:
        return x
    cos, sin = turn
    h = cos.shape[-1]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((a * cos - sign * b * sin, b * cos + sign * a * sin, x[..., 2 * h:]), -1)


def _weight(w, x):
    return 1.0 if w is None else w if w.dim() == 1 else w[:, None]


def _plain_norm(x, w, unit, turn):
    z = x.float()
    rstd = torch.rsqrt((z * z).sum(-1, keepdim=True) / (1 if unit else x.shape[-1]) + EPS)
    return _turn(z * rstd * _weight(w, x), turn, 1).to(x.dtype), rstd


def _plain_norm_backward(grad, x, rstd, w, unit, turn):
    z, dn = x.float(), _turn(grad.float(), turn, -1)
    xn = z * rstd
    gw = dn * _weight(w, x)
    dx = (gw - xn * (gw * xn).sum(-1, keepdim=True) / (1 if unit else x.shape[-1])) * rstd
    dw = None if w is None else (dn * xn).sum((0, 1, 2) if w.dim() == 1 else (0, 2))
    return dx.to(x.dtype), dw


def _inverse(L):
    """(1 + L)^-1 of a strictly lower triangle [..., C, C], C a power of two: blocks of twice the size each time."""
    i = torch.arange(L.shape[-1], device=L.device)
    T = torch.eye(L.shape[-1], device=L.device).expand_as(L)
    size = 1
    while size < L.shape[-1]:
        block = i // size
        T = T - T @ (L * ((block[:, None] % 2 == 1) & (block[:, None] - block == 1))) @ T
        size *= 2
    return T


def _plain_sequences(s):
    """A chunk of tokens as products of matrices; from chunk to chunk the recurrence leaves nothing but a loop."""
    dt, scale, dev = s["q"].dtype, s["scale"], s["q"].device
    B, H, T, d = s["q"].shape
    C = CHUNK
    n = -(-T // C)
    t = torch.arange(T, device=dev)
    count = torch.full((B,), T, device=dev) if s["lengths"] is None else s["lengths"].long()
    live = (t < count[:, None])[:, None]                                       # [B, 1, T]

    def chunks(x):
        x = torch.where(live if x.dim() == 3 else live[..., None], x.float(), 0.0)
        x = torch.nn.functional.pad(x, (0, n * C - T) if x.dim() == 3 else (0, 0, 0, n * C - T))
        return x.view(B, H, n, C, *x.shape[3:])

    q, k, v, g, beta = (chunks(s[x]) for x in ("q", "k", "v", "g", "beta"))
    i = torch.arange(C, device=dev)
    G = torch.cumsum(g.double(), -1)
    D = torch.exp(torch.where(i[:, None] >= i, G[..., :, None] - G[..., None, :], -math.inf)).float()
    near, far, whole = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None], torch.exp(G[..., -1]).float()
    pairs = (k @ k.transpose(-1, -2)) * D * (i[:, None] > i)
    inv = _inverse(beta[..., None] * pairs)
    own_u, w = (inv * beta[..., None, :]) @ v, (inv * beta[..., None, :]) @ (near * k)
    write = (far * k).transpose(-1, -2)
    M = torch.zeros(B, H, d, d, device=dev) if s["state"] is None else s["state"].transpose(-1, -2)
    before, u = torch.empty(B, H, n, d, d, device=dev), torch.empty(B, H, n, C, d, device=dev)
    for c in range(n):
        before[:, :, c] = M
        u[:, :, c] = own_u[:, :, c] - w[:, :, c] @ M
        M = whole[:, :, c, None, None] * M + write[:, :, c] @ u[:, :, c]
    P = scale * D * (q @ k.transpose(-1, -2))
    o = scale * near * (q @ before) + P @ u
    whole_rows = lambda x: x.reshape(B, H, n * C, *x.shape[4:])[:, :, :T]  # noqa: E731
    if s["kind"] == "prompt":
        return {"o": whole_rows(o).to(dt), "S": M.transpose(-1, -2).contiguous()}

    do = chunks(s["grad_o"])
    dM = torch.zeros(B, H, d, d, device=dev) if s["grad_state"] is None else s["grad_state"].transpose(-1, -2)
    from_o, add, take = P.transpose(-1, -2) @ do, (scale * near * q).transpose(-1, -2) @ do, (near * beta[..., None] * k).transpose(-1, -2)
    behind, dr = torch.empty_like(before), torch.empty_like(u)
    for c in reversed(range(n)):
        behind[:, :, c] = dM
        dr[:, :, c] = inv[:, :, c].transpose(-1, -2) @ (from_o[:, :, c] + far[:, :, c] * (k[:, :, c] @ dM))
        dM = whole[:, :, c, None, None] * dM + add[:, :, c] - take[:, :, c] @ dr[:, :, c]
    dv = beta[..., None] * dr
    error = v - near * (k @ before) - pairs @ u
    X = scale * D * (do @ u.transpose(-1, -2))
    Y = -(dv @ u.transpose(-1, -2)) * D * (i[:, None] > i)
    dq = scale * near * (do @ before.transpose(-1, -2)) + X @ k
    dk = X.transpose(-1, -2) @ q + far * (u @ behind.transpose(-1, -2)) - near * (dv @ before.transpose(-1, -2)) + Y @ k + Y.transpose(-1, -2) @ k
    # a log decay lies between its token and all that come before: pairs of tokens, tokens and the chunk's two states, the states
    pair = (X * (q @ k.transpose(-1, -2)) + Y * (k @ k.transpose(-1, -2))) * (i[:, None] > i)
    across = ((pair.cumsum(-1) - pair) * (i[:, None] >= i)).sum(-2)
    reads = scale * near * (q @ before) * do - near * (k @ before) * dv
    kept = far * (k @ behind) * u
    dg = (across + reads.sum(-1).flip(-1).cumsum(-1).flip(-1) + kept.sum(-1).cumsum(-1) - kept.sum(-1)
          + whole[..., None] * (behind * before).sum((-1, -2))[..., None])
    dg = torch.where(live, whole_rows(dg), 0.0)
    return {"dq": whole_rows(dq).to(dt), "dk": whole_rows(dk).to(dt), "dv": whole_rows(dv).to(dt), "dg": dg,
            "dbeta": whole_rows((dr * error).sum(-1)), "dS0": dM.transpose(-1, -2).contiguous()}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    kind, B, H, d = case["kind"], case["B"], case["H"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    if kind == "step":
        return {"bytes": B * H * (8 * d * d + 4 * d * es + 8), "flops": B * H * 7 * d * d}
    rows = B * H * case["T"]
    if kind == "qk":
        tensors = 8 if case["train"] else 4  # q, k and what comes of them; then two gradients read and two written
        weights = {"none": 0, "shared": d, "heads": H * d}[case["weight"]] * 4 * 2 * (2 if case["train"] else 1)
        return {"bytes": rows * tensors * d * es + weights, "flops": 2 * rows * d * (18 if case["train"] else 7)}
    states = B * H * d * d * 4
    if kind == "prompt":  # S k, S += u k^T and S q of each token
        return {"bytes": rows * (4 * d * es + 8) + states * (2 if case["state"] else 1), "flops": rows * 6 * d * d}
    # both again, dS k, two updates of dS, and the products of S and dS for dq and dk
    return {"bytes": rows * (7 * d * es + 16) + states * (3 if case["state"] else 1), "flops": rows * 16 * d * d}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "step":
        pool, o = s["pool"].double(), torch.zeros_like(s["q"], dtype=torch.float64)
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        for b, n in enumerate(s["slots"].tolist()):
            S = torch.einsum("h,hij->hij", torch.exp(s["g"][b].double()), pool[n])
            wrong = v[b] - torch.einsum("hij,hj->hi", S, k[b])
            pool[n] = S + torch.einsum("h,hi,hj->hij", s["beta"][b].double(), wrong, k[b])
            o[b] = s["scale"] * torch.einsum("hij,hj->hi", pool[n], q[b])
        return {"o": o, "pool": pool}
    if kind == "qk":
        (yq, dq, dwq), (yk, dk, dwk) = (_exact_norm(s, x) for x in "qk")
        got = {"yq": yq, "yk": yk}
        if s["train"]:
            got.update(dq=dq, dk=dk)
            if s["wq"] is not None:
                got.update(dwq=dwq, dwk=dwk)
        return got
    return _exact_sequences(s)


def _exact_norm(s, name):
    x, w, rot, d = s[name].double(), s["w" + name], s["rot"], s["d"]
    c = 1.0 if s["unit"] else 1.0 / d
    size = torch.sqrt(c * torch.einsum("bhti,bhti->bht", x, x) + EPS)[..., None]
    w = torch.ones(s["H"], d, dtype=torch.float64, device=x.device) if w is None else w.double().expand(s["H"], d)
    w = w[None, :, None]
    spin = None
    if rot:
        pos = torch.arange(s["T"], device=x.device).expand(s["B"], -1) if s["positions"] is None else s["positions"]
        spin = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), torch.einsum("bt,f->btf", pos.double(), s["freqs"])[:, None])

    def rotate(y, by):  # coordinates i and i + rot / 2 as one complex number
        if spin is None:
            return y
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * by
        return torch.cat((z.real, z.imag, y[..., rot:]), -1)

    y = rotate(x / size * w, spin)
    if not s["train"]:
        return y, None, None
    dz = rotate(s["grad_" + name].double(), None if spin is None else spin.conj())
    p = dz * w
    dx = p / size - c * x * torch.einsum("bhti,bhti->bht", p, x)[..., None] / size ** 3
    dw = torch.einsum("bhti,bhti->hi", dz, x / size)
    return y, dx, (dw.sum(0) if s["weight"] == "shared" else dw)


def _exact_sequences(s):
    """The recurrence and its reverse, token by token, all sequences side by side."""
    B, H, T, d = s["q"].shape
    dev, scale, train = s["q"].device, s["scale"], s["kind"] == "train"
    n = torch.full((B,), T, device=dev) if s["lengths"] is None else s["lengths"].long()
    live = (torch.arange(T, device=dev)[:, None] < n).view(T, B, 1, 1)
    seq = lambda x: torch.where(live, x.double().permute(2, 0, 1, 3).reshape(T, B, H, -1), 0.0)  # noqa: E731
    q, k, v = (seq(s[x]) for x in "qkv")
    a, beta = torch.exp(seq(s["g"][..., None])), seq(s["beta"][..., None])
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double()

    def token(S, t):
        """The state decayed to token t, and what it gets wrong about it."""
        S = a[t, :, :, :, None] * S
        return S, v[t] - (S @ k[t][..., None])[..., 0]

    o, kept, W = torch.empty_like(q), [], 64
    for t in range(T):
        if train and t % W == 0:
            kept.append(S)
        S, e = token(S, t)
        S = S + (beta[t] * e)[..., :, None] * k[t][..., None, :]
        if not train:
            o[t] = scale * (S @ q[t][..., None])[..., 0]
    back = lambda x: x.permute(1, 2, 0, 3).contiguous()  # noqa: E731
    if not train:
        return {"o": back(o), "S": S}
    do, R = seq(s["grad_o"]), torch.zeros_like(S) if s["grad_state"] is None else s["grad_state"].double()
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    dg, db = (torch.empty_like(a) for _ in range(2))
    for first in reversed(range(0, T, W)):
        states, S = [], kept[first // W]
        for t in range(first, min(T, first + W)):
            D, e = token(S, t)
            S = D + (beta[t] * e)[..., :, None] * k[t][..., None, :]
            states.append((D, e, S))
        for t in reversed(range(first, min(T, first + W))):
            D, e, S = states.pop()
            dq[t] = scale * (do[t][..., None, :] @ S)[..., 0, :]
            R = R + scale * do[t][..., :, None] * q[t][..., None, :]
            du = (R @ k[t][..., None])[..., 0]
            db[t] = (du * e).sum(-1, keepdim=True)
            dv[t] = beta[t] * du
            dk[t] = (((beta[t] * e)[..., None, :] @ R) - dv[t][..., None, :] @ D)[..., 0, :]
            R = R - dv[t][..., :, None] * k[t][..., None, :]
            dg[t] = (R * D).sum((-1, -2))[..., None] * live[t]
            R = a[t, :, :, :, None] * R
    return {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dg": back(dg)[..., 0], "dbeta": back(db)[..., 0], "dS0": R}
