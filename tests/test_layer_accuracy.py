"""What the normwise limits of layer_accuracy.py let pass and what they catch, on an emulation of the bf16 kernel."""
import pytest
import torch

import layer_accuracy as A
import layer_ref as R

SIZES = [(2, 3, 129, 96), (1, 4, 200, 128), (2, 4, 256, 32), (1, 2, 1024, 64)]


def inputs(B, H, T, d):
    gen = torch.Generator().manual_seed(T + d)
    q, k, v = (torch.randn(B, H, T, d, generator=gen).bfloat16() for _ in range(3))
    g = -torch.exp2(torch.linspace(-9, 1, H))
    return q, k, v, g, torch.randn(B, H, d, d, generator=gen)


@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_limits_of_rows_and_states(B, H, T, d):
    q, k, v, g, S0 = inputs(B, H, T, d)
    ro, rS = R.decay(q, k, v, g, 0.3, S0)
    run = lambda **kw: (lambda o, S: (float(A.block_errors(o, ro).max()), float(A.state_errors(S, rS).max())))(  # noqa: E731
        *A.emulate(q, k, v, g, 0.3, S0, **kw))
    rows, states = run()
    assert rows <= A.ROWS and states <= A.STATES
    assert run(pair_bits=6)[0] > A.ROWS
    assert run(state_bits=6)[0] > A.ROWS
    assert run(older=1.02)[0] > A.ROWS
    assert run(parts=2)[1] > A.STATES


def test_to_bits_and_cut():
    x = torch.randn(1000, generator=torch.Generator().manual_seed(0))
    assert torch.equal(A.to_bits(x, 8), x.bfloat16().float())
    assert torch.equal(A.cut(x) + A.cut(x - A.cut(x)) + A.cut(x - A.cut(x) - A.cut(x - A.cut(x))), x)
