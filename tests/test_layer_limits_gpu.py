"""The operators of include/vla_layer.h at the edges of their contract."""
import pytest
import torch

import layer_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import check_backward, check_forward, seqs, state_like

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---- values that are not finite -----------------------------------------------------------------------------------

def clean_of(x, *at):
    """x with the planted values taken out."""
    y = x.clone()
    y[at] = 0
    return y


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,t,d", [(1, 0, 32), (8, 5, 64), (64, 63, 96), (50, 20, 64), (200, 150, 128), (77, 70, 32),
                                   (1500, 1111, 64), (130, 0, 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_earlier_tokens_do_not_see_later_values(T, t, d, dtype, bad):
    """o_i depends on tokens j <= i alone, and the gradients at i of dk and dv on j >= i, whatever the others hold."""
    B, H, h = 1, 2, 1
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=T + d)
    g = torch.tensor([-0.3, -0.01], device="cuda")
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    x = 3

    def same_rows(got, ref, mag, rows, name):
        R.assert_within(got[:, h:, rows], ref[:, h:, rows], R.seq_bound(ref, mag, dtype, T, d, g)[:, h:, rows], name)

    # v: o's rows before t, and all of the other head
    v2 = v.clone()
    v2[0, h, t, x] = bad
    v0 = clean_of(v, 0, h, t, x)
    ro, mo = (R.decay(*a, g, s, S, None)[0] for a, s, S in (((q, k, v0), 0.5, S0),
                                                            ((q.abs(), k.abs(), v0.abs()), 0.5, S0.abs())))
    S = S0.clone()
    o, _ = vla.vla_decay_forward(q, k, v2, g, 0.5, S, out=(torch.empty_like(q), S))
    same_rows(o, ro, mo, slice(0, t), "o")
    # in row t every coordinate but x is finite, and x is not
    assert torch.isfinite(o[0, h, t, :x]).all() and not torch.isfinite(o[0, h, t, x]).any()
    assert not torch.isfinite(S[0, h, x]).all() and torch.isfinite(S[0, h, x + 1:]).all()
    assert torch.isfinite(o[0, 0]).all() and torch.isfinite(S[0, 0]).all()
    assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_NONFINITE

    # k in dq: rows before t. q in dk and dO in dv: rows behind t
    for i, name, rows in ((1, "dq", slice(0, t)), (0, "dk", slice(t + 1, T)), (2, "dv", slice(t + 1, T))):
        ins = [q, k, do]
        planted = [y.clone() for y in ins]
        planted[i][0, h, t, x] = bad
        got = vla.vla_decay_backward(planted[0], planted[1], v, g, 0.5, S0, planted[2], dS)[0]
        ins[i] = clean_of(ins[i], 0, h, t, x)
        ref = R.decay_grads(ins[0], ins[1], v, g, 0.5, S0, ins[2], dS)
        mag = R.decay_grads(ins[0].abs(), ins[1].abs(), v.abs(), g, 0.5, S0.abs(), ins[2].abs(), dS.abs())
        at = ("dq", "dk", "dv").index(name)
        same_rows(got[at], ref[at], mag[at], rows, name)
        assert torch.isfinite(got[at][0, 0]).all()
        assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_NONFINITE


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths", [None, [150, 64, 133]])
def test_every_place_of_a_value_that_is_not_finite(lengths, dtype):
    """Another token in each head, around every edge of a chunk: exactly the rows from it on are not finite, in its
    column alone; for gradients that run against time the rows up to it."""
    B, T, d, x = 3, 150, 64, 11
    places = [0, 1, 31, 32, 33, 62, 63, 64, 65, 95, 96, 127, 128, 149]
    H = len(places)
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=1)
    g = torch.full((H,), -0.05, device="cuda")
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for h, t in enumerate(places):
        v[:, h, t, x] = do[:, h, t, x] = float("nan")
    o, _ = vla.vla_decay_forward(q, k, v, g, lengths=n)
    (_, _, dv), _ = vla.vla_decay_backward(q, k, k, g, grad_o=do, lengths=n)
    t = torch.arange(T, device="cuda")
    at = torch.tensor(places, device="cuda")[None, :, None]
    live = torch.full((B, 1, 1), T, device="cuda") if n is None else n.view(B, 1, 1)
    for got, after in ((o, t >= at), (dv, t <= at)):
        want = torch.zeros(B, H, T, d, dtype=torch.bool, device="cuda")
        want[..., x] = after & (t < live) & (at < live)
        assert torch.equal(torch.isnan(got), want) and torch.isfinite(got[~want]).all()
    assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_NONFINITE  # read and cleared


# ---- heads that grow ----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("T", [90, 300, 1300])
def test_growth_beyond_the_range_of_a_factor(T, d, dtype):
    """A chunk's factor overflows, the sequence's results do not: nothing but zeros are multiplied by it."""
    B, H, live = 2, 4, 20
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=d + T)
    g = torch.tensor([2.5, 1.4, 0.2, -0.1], device="cuda")
    for x in (k, v):
        x[:, :, :T - live] = 0
    check_forward(q, k, v, g, 0.3, None, None)
    check_forward(q, k, v, g, 0.3, torch.zeros(B, H, d, d, device="cuda"), None)
    do[:, :, live:] = 0
    check_backward(q, k, v, g, 0.3, None, do, None, None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,d,g", [(63, 64, 1.3), (78, 128, 1.0), (78, 32, 1.0), (110, 96, 0.72), (700, 64, 0.1)])
def test_growth_with_every_token(T, d, g, dtype):
    q, k, v, do = seqs(4, 1, 3, T, d, dtype, seed=d)
    g = torch.tensor([g, -0.2, g], device="cuda")
    n = torch.tensor([T - 2], dtype=torch.int32, device="cuda")
    S0, dS = state_like(1, 3, d, 1), state_like(1, 3, d, 2)
    check_forward(q, k, v, g, 0.3, S0, n)
    check_backward(q, k, v, g, 0.3, S0, do, dS, n)


def test_growth_as_in_single_tokens():
    """A prompt of a head that grows a hundredfold a token, and the same tokens one at a time."""
    B, H, T, d = 2, 2, 12, 64
    q, k, v = seqs(3, B, H, T, d, F32, seed=7)
    g = torch.tensor([4.6, 0.8], device="cuda")
    S0 = state_like(B, H, d, 1)
    o, S = check_forward(q, k, v, g, 0.1, S0, None)
    pool = S0.clone()
    rows = [vla.vla_decay_step(q[:, :, t], k[:, :, t], v[:, :, t], g, pool, 0.1, check=True) for t in range(T)]
    check_forward(q, k, v, g, 0.1, S0, None, (torch.stack(rows, 2), pool))
