"""Cases of the operators around the recurrence: linear attention with a decay per head (prompt, training, single
tokens), the layer norm of each head's readout, and the quantised cache of states.

``own`` false: the plain forms, in elementary torch operations. ``own`` true: the package's calls.
"""
import math

import torch

own = False

GROUP = 32  # values that share a scale in the quantised cache
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a batch of prompts at the head dimension of the benchmark's workload
        dict(name="prompt_d96", kind="prompt", B=8, H=16, T=4096, d=96, dtype="bf16", rows="heads", state=False, ragged=False),
        # one long context, few heads: the work has to be split along the sequence
        dict(name="prompt_long_d128", kind="prompt", B=1, H=32, T=65536, d=128, dtype="bf16", rows="heads", state=False, ragged=False),
        # padded prompts of several lengths that continue earlier turns, fp32
        dict(name="prompt_ragged_f32_d64", kind="prompt", B=5, H=8, T=1021, d=64, dtype="f32", rows="tokens", state=True, ragged=True),
        # gradients of a training step
        dict(name="train_d64", kind="train", B=4, H=8, T=4096, d=64, dtype="bf16", rows="heads", state=False, ragged=False),
        # gradients through a carried state, projections in token order, odd length
        dict(name="train_state_d128", kind="train", B=2, H=32, T=8191, d=128, dtype="bf16", rows="tokens", state=True, ragged=False),
        # a small fp32 model with padded sequences
        dict(name="train_ragged_f32_d32", kind="train", B=3, H=5, T=777, d=32, dtype="f32", rows="heads", state=True, ragged=True),
        # one user's next token: latency
        dict(name="step_one_d128", kind="step", B=1, H=32, d=128, dtype="bf16", slots=1),
        # a server's batch of next tokens over a pool of states
        dict(name="step_pool_d128", kind="step", B=256, H=32, d=128, dtype="bf16", slots=300),
        # the readout's norm over a long prompt, written in token order for the output projection
        dict(name="norm_prompt_d128", kind="norm", B=1, H=32, T=65536, d=128, dtype="bf16", train=False, bias=False),
        # the readout's norm in a training step: forward, then its gradients
        dict(name="norm_train_d96", kind="norm", B=8, H=16, T=4096, d=96, dtype="bf16", train=True, bias=True),
        # sequences parked in 8 bits and brought back into other batch rows
        dict(name="park_8bit_d128", kind="park", B=64, H=32, d=128, bits=8, slots=80),
        # shared prefixes read back from 4 bits, several sequences from the same slot
        dict(name="resume_4bit_d96", kind="resume", B=48, H=16, d=96, bits=4, slots=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "train", "train", "step", "norm", "park", "resume"])
    d = rng.choice([32, 64, 96, 128])
    H = rng.randint(1, 32)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("prompt", "train"):
        T = _log(rng, 1, 16384)
        B = max(1, min(rng.randint(1, 8), (1 << 25) // (T * H * d)))
        return dict(kind=kind, B=B, H=H, T=T, d=d, dtype=dtype, rows=rng.choice(["heads", "tokens"]),
                    state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if kind == "norm":
        T = _log(rng, 1, 32768)
        B = max(1, min(rng.randint(1, 8), (1 << 26) // (T * H * d)))
        return dict(kind=kind, B=B, H=H, T=T, d=d, dtype=dtype, train=rng.random() < 0.6, bias=rng.random() < 0.5)
    B = _log(rng, 1, 128)
    if kind == "step":
        return dict(kind=kind, B=B, H=H, d=d, dtype=dtype, slots=B + rng.randint(0, 40))
    return dict(kind=kind, B=min(B, 64), H=H, d=d, bits=rng.choice([8, 4]), slots=min(B, 64) + rng.randint(0, 20))


# ---------------------------------------------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------------------------------------------
def _decays(H, dev):
    """log of the decay of each head, from exp(-1/2) down to nearly none, spaced evenly in their logarithm."""
    h = torch.arange(H, dtype=torch.float64)
    return (-torch.exp2(-(1 + 8 * h / max(1, H - 1)))).to(device=dev, dtype=torch.float32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind, B, H, d = case["kind"], case["B"], case["H"], case["d"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def sequence(T, dtype, rows):
        """[B, H, T, d]; "tokens": a view of a projection's output, [B, T, H, d] in memory."""
        if rows == "tokens":
            return normal(B, T, H, d, dtype=dtype).transpose(1, 2)
        return normal(B, H, T, d, dtype=dtype)

    s = dict(case)
    if kind in ("prompt", "train"):
        T, dt = case["T"], DT[case["dtype"]]
        for name in ("q", "k", "v") + (("grad_o",) if kind == "train" else ()):
            s[name] = sequence(T, dt, case["rows"])
        s["log_decay"], s["scale"] = _decays(H, dev), d ** -0.5
        s["state"] = normal(B, H, d, d) if case["state"] else None
        s["grad_state"] = normal(B, H, d, d) if kind == "train" and case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            n[0] = T
            s["lengths"] = n
    elif kind == "step":
        dt, N = DT[case["dtype"]], case["slots"]
        s["q"], s["k"], s["v"] = (normal(B, H, d, dtype=dt) for _ in range(3))
        s["log_decay"], s["scale"] = _decays(H, dev), d ** -0.5
        s["pool"] = normal(N, H, d, d)
        s["slots"] = torch.randperm(N, generator=gen, device=dev)[:B].to(torch.int32)
    elif kind == "norm":
        dt = DT[case["dtype"]]
        s["x"] = (normal(B, H, case["T"], d) * 3 + 0.5).to(dt)
        s["weight"] = 1 + 0.1 * normal(H, d)
        s["bias"] = 0.1 * normal(H, d) if case["bias"] else None
        s["y"] = torch.empty(B, case["T"], H, d, device=dev, dtype=dt).transpose(1, 2)
        if case["train"]:
            s["grad_y"] = normal(B, case["T"], H, d, dtype=dt).transpose(1, 2)
    else:
        N, bits = case["slots"], case["bits"]
        # rows of a state differ in size, as its value channels do
        rows = torch.exp(normal(N, H, d, 1))
        if bits == 8:
            s["codes"] = torch.zeros(N, H, d, d, dtype=torch.int8, device=dev)
        else:
            s["codes"] = torch.zeros(N, H, d, d // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(N, H, d, d // GROUP, dtype=torch.float32, device=dev)
        if kind == "park":
            s["x"] = normal(B, H, d, d) * rows[:B]
            s["slots"] = torch.randperm(N, generator=gen, device=dev)[:B].to(torch.int32)
            s["back"] = s["slots"].flip(0).contiguous()
        else:
            _plain_store(normal(N, H, d, d) * rows, s["codes"], s["scales"], torch.arange(N, device=dev))
            s["slots"] = torch.randint(0, N, (B,), generator=gen, device=dev, dtype=torch.int32)
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
        o, S = vla.vla_decay_forward(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["state"], lengths=s["lengths"])
        return {"o": o, "S": S}
    if kind == "train":
        (dq, dk, dv), dS0 = vla.vla_decay_backward(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["state"],
                                                   s["grad_o"], s["grad_state"], lengths=s["lengths"])
        return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}
    if kind == "step":
        o = vla.vla_decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], s["scale"], slots=s["slots"])
        return {"o": o, "pool": s["pool"]}
    if kind == "norm":
        y, stats = vla.vla_head_norm(s["x"], s["weight"], s["bias"], EPS, out=s["y"])
        got = {"y": y, "mean": stats[0], "rstd": stats[1]}
        if s["train"]:
            dx, dw, db = vla.vla_head_norm_backward(s["grad_y"], s["x"], stats, s["weight"])
            got.update(dx=dx, dw=dw, db=db)
        return got
    if kind == "park":
        vla.vla_state_store(s["x"], s["codes"], s["scales"], s["slots"])
        return {"x": vla.vla_state_load(s["codes"], s["scales"], s["back"]), "scales": s["scales"]}
    return {"x": vla.vla_state_load(s["codes"], s["scales"], s["slots"])}


# ---------------------------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------------------------
def _pow(g, n):
    """exp(g n), g [H] and n a tensor of whole numbers >= 0: [H, *n.shape], the angle in 64 bits."""
    n = n.double()
    return torch.exp(g.double().view(-1, *(1,) * n.dim()) * n).float()


def _causal(a, b, c, g):
    """out_i = sum_{j <= i} exp(g (i - j)) (a_i . b_j) c_j, in chunks that a matrix of decays joins."""
    B, H, T, d = a.shape
    C = min(128, T)
    n = -(-T // C)
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).view(B, H, n, C, d) for x in (a, b, c))
    i = torch.arange(C, device=a.device)
    r = torch.arange(n, device=a.device)
    lag = i[:, None] - i[None]
    near = _pow(g, lag.clamp(min=0)) * (lag >= 0)                              # [H, C, C]
    o = ((a @ b.transpose(-1, -2)) * near[:, None]) @ c
    own_state = (c * _pow(g, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ b  # [B, H, n, d, d]
    gap = r[:, None] - r[None] - 1
    far = _pow(g, gap.clamp(min=0) * C) * (gap >= 0)                           # [H, n, n]
    before = (far @ own_state.reshape(B, H, n, d * d)).view(B, H, n, d, d)
    o = o + (a @ before.transpose(-1, -2)) * _pow(g, i + 1)[:, None, :, None]
    return o.reshape(B, H, n * C, d)[:, :, :T]


def _plain(s):
    kind = s["kind"]
    if kind in ("prompt", "train"):
        dt, g, scale = s["q"].dtype, s["log_decay"], s["scale"]
        B, H, T, d = s["q"].shape
        t = torch.arange(T, device=g.device)
        n = torch.full((B,), T, device=g.device) if s["lengths"] is None else s["lengths"].long()
        live = (t[None] < n[:, None])[:, None, :, None]                        # [B, 1, T, 1]
        q, k, v = (torch.where(live, s[x].float(), 0.0) for x in "qkv")
        left = (n[:, None] - 1 - t[None]).clamp(min=0)                         # tokens after t, [B, T]
        tail = _pow(g, left).transpose(0, 1).unsqueeze(-1)                     # [B, H, T, 1]
        whole = _pow(g, n).transpose(0, 1)[..., None, None]                    # [B, H, 1, 1]
        head = _pow(g, t + 1)[None, :, :, None]                                # [1, H, T, 1]
        if kind == "prompt":
            o, S = _causal(q, k, v, g), (v * tail).transpose(-1, -2) @ k
            if s["state"] is not None:
                o = o + (q @ s["state"].transpose(-1, -2)) * head
                S = S + s["state"] * whole
            return {"o": (o * scale).to(dt), "S": S}
        do = torch.where(live, s["grad_o"].float(), 0.0)
        back = lambda a, b, c: _causal(a.flip(2), b.flip(2), c.flip(2), g).flip(2)  # noqa: E731
        dq, dk, dv = _causal(do, v, k, g) * scale, back(v, do, q) * scale, back(k, q, do) * scale
        dS0 = (do * head).transpose(-1, -2) @ q * scale
        if s["state"] is not None:
            dq = dq + (do @ s["state"]) * head * scale
        if s["grad_state"] is not None:
            dk = dk + (v @ s["grad_state"]) * tail
            dv = dv + (k @ s["grad_state"].transpose(-1, -2)) * tail
            dS0 = dS0 + s["grad_state"] * whole
        return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dS0": dS0}
    if kind == "step":
        at, q, k, v = s["slots"].long(), s["q"].float(), s["k"].float(), s["v"].float()
        S = s["pool"][at] * torch.exp(s["log_decay"])[:, None, None] + v[..., :, None] * k[..., None, :]
        s["pool"][at] = S
        return {"o": ((S @ q[..., None])[..., 0] * s["scale"]).to(s["q"].dtype), "pool": s["pool"]}
    if kind == "norm":
        x, w = s["x"].float(), s["weight"][None, :, None]
        mean = x.mean(-1)
        xc = x - mean[..., None]
        rstd = torch.rsqrt((xc * xc).mean(-1) + EPS)
        xn = xc * rstd[..., None]
        y = xn * w
        if s["bias"] is not None:
            y = y + s["bias"][None, :, None]
        s["y"].copy_(y)
        got = {"y": s["y"], "mean": mean, "rstd": rstd}
        if s["train"]:
            dy = s["grad_y"].float()
            gw = dy * w
            dx = (gw - gw.mean(-1, keepdim=True) - xn * (gw * xn).mean(-1, keepdim=True)) * rstd[..., None]
            got.update(dx=dx.to(s["x"].dtype), dw=(dy * xn).sum((0, 2)), db=dy.sum((0, 2)))
        return got
    if kind == "park":
        _plain_store(s["x"], s["codes"], s["scales"], s["slots"].long())
        return {"x": _plain_load(s["codes"], s["scales"], s["back"].long()), "scales": s["scales"]}
    return {"x": _plain_load(s["codes"], s["scales"], s["slots"].long())}


def _plain_store(x, codes, scales, at):
    """Groups of 32 values to whole numbers of at most 127 (8 bits) or 7 (4 bits) in size, times the group's scale."""
    top = 127 if codes.dtype == torch.int8 else 7
    x = x.view(*x.shape[:-1], -1, GROUP)
    scale = (x.abs().amax(-1).double() / top).float()
    scale = torch.where(scale < 2.0 ** -126, 0.0, scale)
    # the quotient in 64 bits: a value between two codes goes to the nearer one, ties to the even one
    c = torch.round(x.double() / torch.where(scale == 0, 1.0, scale).double()[..., None]) * (scale != 0)[..., None]
    c = c.clamp(-top, top).to(torch.int8).flatten(-2)
    if top == 7:
        c = ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).view(torch.uint8)
    codes[at] = c
    scales[at] = scale


def _plain_load(codes, scales, at):
    c = codes[at]
    if codes.dtype != torch.int8:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2).to(torch.int8)
        c = c - 16 * (c > 7).to(torch.int8)
    return (c.float().view(*c.shape[:-1], -1, GROUP) * scales[at][..., None]).flatten(-2)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    kind, B, H, d = case["kind"], case["B"], case["H"], case["d"]
    es = 4 if case.get("dtype") == "f32" else 2
    if kind in ("prompt", "train"):
        rows, states = B * H * case["T"], B * H * d * d * 4
        if kind == "prompt":
            return {"bytes": rows * d * es * 4 + states * (2 if case["state"] else 1), "flops": rows * 4 * d * d}
        return {"bytes": rows * d * es * 7 + states * (3 if case["state"] else 1), "flops": rows * 10 * d * d}
    if kind == "step":
        return {"bytes": B * H * d * (8 * d + 4 * es), "flops": B * H * 5 * d * d}
    if kind == "norm":
        rows = B * H * case["T"]
        tensors = 4 if case["train"] else 2  # x once, y; grad_y and dx
        return {"bytes": rows * (tensors * d * es + 8) + H * d * 16, "flops": rows * d * (20 if case["train"] else 8)}
    values = B * H * d * d
    code = case["bits"] / 8 + 4 / GROUP
    if kind == "park":
        return {"bytes": values * (4 + code + code + 4), "flops": values * 4}
    return {"bytes": values * 4 + min(B, case["slots"]) * H * d * d * code, "flops": values}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("prompt", "train"):
        return _exact_sequences(s)
    if kind == "step":
        S, q, k, v = s["pool"].double(), s["q"].double(), s["k"].double(), s["v"].double()
        lam, o = torch.exp(s["log_decay"].double()), torch.zeros_like(q)
        for b, n in enumerate(s["slots"].tolist()):
            state = S[n]
            state.mul_(lam[:, None, None]).add_(torch.einsum("hi,hj->hij", v[b], k[b]))
            o[b] = torch.einsum("hij,hj->hi", state, q[b]) * s["scale"]
        return {"o": o, "pool": S}
    if kind == "norm":
        x, w = s["x"].double(), s["weight"].double().view(1, s["H"], 1, -1)
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        hat = (x - mean[..., None]) * rstd[..., None]
        got = {"y": hat * w + (0 if s["bias"] is None else s["bias"].double().view(1, s["H"], 1, -1)), "mean": mean, "rstd": rstd}
        if s["train"]:
            dy = s["grad_y"].double()
            p, d = dy * w, s["d"]
            got["dx"] = rstd[..., None] / d * (d * p - p.sum(-1, keepdim=True) - hat * (p * hat).sum(-1, keepdim=True))
            got["dw"], got["db"] = torch.einsum("bhtd,bhtd->hd", dy, hat), torch.einsum("bhtd->hd", dy)
        return got
    if kind == "park":
        # each value to the nearest multiple of its group's 32-bit scale
        top, x = (127.0 if s["bits"] == 8 else 7.0), s["x"].double()
        groups = x.unflatten(-1, (-1, GROUP))
        scale = (groups.abs().max(-1).values / top).float().double()
        near = (torch.round(groups / scale[..., None]) * scale[..., None]).flatten(-2)
        scales = torch.zeros_like(s["scales"], dtype=torch.float64)
        scales[s["slots"].long()] = scale
        return {"x": near.flip(0), "scales": scales}
    # codes and scales are whole numbers and 32-bit values: their products in 64 bits
    c = s["codes"].index_select(0, s["slots"].long())
    if s["bits"] == 4:
        low, high = (c.long() & 15), (c.long() >> 4)
        c = torch.stack(((low + 8) % 16 - 8, (high + 8) % 16 - 8), -1).flatten(-2)
    return {"x": c.double() * s["scales"].index_select(0, s["slots"].long()).double().repeat_interleave(GROUP, -1)}


def _exact_sequences(s):
    """The recurrence, a block of tokens at a time, sequence by sequence."""
    B, H, T, d = s["q"].shape
    g, scale, dev = s["log_decay"].double(), s["scale"], s["q"].device
    out = {n: torch.zeros(B, H, T, d, dtype=torch.float64, device=dev) for n in (("o",) if s["kind"] == "prompt" else ("dq", "dk", "dv"))}
    ends = torch.zeros(B, H, d, d, dtype=torch.float64, device=dev)
    W = 256
    i = torch.arange(W, device=dev, dtype=torch.float64)
    D = torch.exp(g[:, None, None] * (i[:, None] - i).clamp(min=0)).tril()
    up = torch.exp(g[:, None] * (i + 1))[..., None]
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        x = {m: s[m][b, :, :n].double() for m in ("q", "k", "v", "grad_o") if m in s}
        S = torch.zeros(H, d, d, dtype=torch.float64, device=dev) if s["state"] is None else s["state"][b].double()
        for t in range(0, n, W):
            e = min(n, t + W)
            m = e - t
            k, v = x["k"][:, t:e], x["v"][:, t:e]
            if s["kind"] == "prompt":
                q = x["q"][:, t:e]
                out["o"][b, :, t:e] = scale * (torch.einsum("hij,hjd->hid", torch.einsum("hid,hjd->hij", q, k) * D[:, :m, :m], v)
                                               + up[:, :m] * torch.einsum("hid,hcd->hic", q, S))
            else:
                y = x["grad_o"][:, t:e]
                out["dq"][b, :, t:e] = scale * (torch.einsum("hij,hjd->hid", torch.einsum("hid,hjd->hij", y, v) * D[:, :m, :m], k)
                                                + up[:, :m] * torch.einsum("hic,hcd->hid", y, S))
            S = torch.exp(g * m)[:, None, None] * S + torch.einsum("hjc,hjd->hcd", v * D[:, m - 1, :m, None], k)
        ends[b] = S
        if s["kind"] == "train":
            R = torch.zeros(H, d, d, dtype=torch.float64, device=dev) if s["grad_state"] is None else s["grad_state"][b].double()
            for t in reversed(range(0, n, W)):  # R: the state's gradient behind token e - 1
                e = min(n, t + W)
                m = e - t
                q, k, v, y = (x[a][:, t:e] for a in ("q", "k", "v", "grad_o"))
                U = D[:, :m, :m].transpose(1, 2)
                last = D[:, m - 1, :m, None]
                out["dk"][b, :, t:e] = (scale * torch.einsum("hji,hid->hjd", torch.einsum("hjc,hic->hji", v, y) * U, q)
                                        + last * torch.einsum("hjc,hcd->hjd", v, R))
                out["dv"][b, :, t:e] = (scale * torch.einsum("hji,hic->hjc", torch.einsum("hjd,hid->hji", k, q) * U, y)
                                        + last * torch.einsum("hjd,hcd->hjc", k, R))
                R = torch.exp(g * m)[:, None, None] * R + scale * torch.einsum("hic,hid->hcd", y * up[:, :m], q)
            ends[b] = R
    return out | ({"S": ends} if s["kind"] == "prompt" else {"dS0": ends})
