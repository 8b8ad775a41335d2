"""Normwise accuracy of the decayed linear attention: tighter than the elementwise bounds of layer_ref.py, which
are worst cases over every term, and an emulation of the bf16 kernel's arithmetic to show what each limit catches.

Limits, by arithmetic:

ROWS, bf16 outputs (o, dq, dk, dv), relative 2-norm over blocks of 128 rows of a head. A rounding to bf16 of values
that are spread evenly over their logarithm is off by 2^-7 / sqrt(12) times sqrt(E[1 / m^2]) = sqrt(3 / (8 ln 2)), that
is 1.66e-3, rms. A result meets two, of its terms (errors of random signs, like the terms) and of itself: 2.35e-3. Where a
row has one term its error is that of one number, with E[e^4] < 2 E[e^2]^2; rows weigh by their squared size, which is at
worst that of one normal product (a kurtosis of 3): of 128 rows the mean square is 2 sqrt(3 / 128) of 2.76e-6 off at most,
at six standard deviations: sqrt(2 * 2.76e-6 + 6 * sqrt(3 / 128) * 2.76e-6) = 2.84e-3 < 3e-3.

STATES, relative 2-norm of a head. bf16: a chunk's sums take 12 steps in fp32 (three parts of the decayed values, four times
16 tokens), each cut off by at most 2^-23 of the sum so far, half of that on average, whose size grows with the root
of the steps: 12 * 2 / 3 * 2^-24 = 4.8e-7 of the chunk's share, in its own direction. Adding n chunks up rounds n times,
2^-24 / sqrt(3) each of random signs: 1.6e-7 for 20. Powers of the decay are within 2 ulp, 1.2e-7 each, of one
sign for a chunk at worst. Below 1e-6 together. fp32: T additions in turn, each off by 2^-24 / sqrt(3) of a sum whose size
grows with the root of the tokens: sqrt(T / 2) * 3.4e-8, 7.7e-7 for 1,000.

ROWS32, fp32 outputs: a state's error, a dot product over its d columns (sqrt(d / 2) * 3.4e-8 = 2.8e-7 for 128) and
those of the pairs and their weights (5e-7): below 2e-6.
"""
import torch

ROWS, ROWS32, STATES, BLOCK = 3e-3, 2e-6, 1e-6, 128


def block_errors(x, ref):
    """Relative 2-norms of x - ref over blocks of 128 rows of each head (the rest of a head's rows with the last block)."""
    x, ref = x.detach().double().cpu(), ref.double().cpu()
    B, H, T, d = ref.shape
    out = []
    n = max(1, T // BLOCK)
    for i in range(n):
        rows = slice(i * BLOCK, T if i == n - 1 else (i + 1) * BLOCK)
        a, r = (x[:, :, rows] - ref[:, :, rows]).flatten(2).norm(dim=-1), ref[:, :, rows].flatten(2).norm(dim=-1)
        out.append(torch.where(r > 0, a / torch.where(r > 0, r, 1.0), a))
    return torch.stack(out)


def state_errors(x, ref):
    x, ref = x.detach().double().cpu(), ref.double().cpu()
    return (x - ref).flatten(2).norm(dim=-1) / ref.flatten(2).norm(dim=-1).clamp(min=1e-300)


def to_bits(x, bits):
    """x (fp32) to `bits` significant bits, to nearest."""
    m, e = torch.frexp(x.double())
    return torch.ldexp(torch.round(m * 2 ** bits), e - bits).float()


def cut(x):
    """The leading eight bits of x, the rest cut off."""
    return (x.view(torch.int32) & -65536).view(torch.float32)


def emulate(q, k, v, g, scale, state=None, parts=3, pair_bits=8, state_bits=8, older=1.0):
    """The bf16 kernel's arithmetic: chunks of 64 tokens, pairs and the state that they find in `pair_bits` and
    `state_bits` bits, the decayed values in `parts` parts; `older`: a factor on what older chunks give."""
    B, H, T, d = q.shape
    q, k, v = (x.float() for x in (q, k, v))
    S = torch.zeros(B, H, d, d) if state is None else state.clone()
    o = torch.empty(B, H, T, d)
    for t in range(0, T, 64):
        n = min(64, T - t)
        a, b, c = (x[:, :, t:t + n] for x in (q, k, v))
        i = torch.arange(n)
        power = lambda m: torch.exp(g.double()[:, None] * m).float()  # noqa: E731
        W = torch.where(i[:, None] >= i, power((i[:, None] - i).clamp(min=0).flatten()).view(H, n, n), 0.0)
        P = to_bits((a @ b.transpose(-1, -2)) * (scale * W), pair_bits)
        OE = a @ to_bits(S, state_bits).transpose(-1, -2)
        o[:, :, t:t + n] = P @ c + older * scale * power(i + 1)[..., None] * OE
        z = c * power(n - 1 - i)[..., None]
        S = S * power(torch.tensor([n]))[..., None]
        for _ in range(parts):
            S = S + cut(z).transpose(-1, -2) @ b
            z = z - cut(z)
    return o.bfloat16(), S
