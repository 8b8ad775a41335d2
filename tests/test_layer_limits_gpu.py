"""The operators of include/vla_layer.h at the edges of their contract."""
import pytest
import torch

import layer_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import check_backward, check_forward, decays, seqs, state_like

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


# ---- outputs on top of inputs -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF])
def test_outputs_on_top_of_inputs_are_refused(dtype):
    """Blocks of one call read what others write: refused, and nothing is written."""
    B, H, T, d = 2, 2, 90, 64
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=3)
    g = decays(H)
    S, dS, dS0 = (state_like(B, H, d, i) for i in range(3))
    pool = state_like(3 * B, H, d, 4)
    w = torch.ones(H, d, device="cuda")
    one = [x[:, :, 0].contiguous() for x in (q, k, v)]
    longer = torch.zeros(B, H, T + 1, d, dtype=dtype, device="cuda")
    x = longer[:, :, :T]
    everything = [q, k, v, do, S, dS, dS0, pool, *one, longer]
    before = [t.clone() for t in everything]
    fresh = lambda: torch.empty_like(q)  # noqa: E731
    stats = vla.vla_head_norm(q)[1]
    calls = [lambda y=y: vla.vla_decay_forward(q, k, v, g, 1.0, S, out=(y, torch.empty_like(S))) for y in (q, k, v)]
    calls += [lambda y=y: vla.vla_decay_backward(q, k, v, g, 1.0, S, do, dS, out=(*y, dS0))
              for y in ((q, k, v), (fresh(), fresh(), do), (q, fresh(), fresh()), (x, x, fresh()))]
    calls += [lambda y=y: vla.vla_decay_backward(q, k, v, g, 1.0, pool[:B], do, pool[2 * B:], out=(fresh(), fresh(), fresh(), y))
              for y in (pool[1:B + 1], pool[2 * B - 1:3 * B - 1], pool[:B])]
    calls += [lambda: vla.vla_decay_forward(q, k, v, g, 1.0, pool[:B], out=(fresh(), pool[1:B + 1]))]
    calls += [lambda y=y: vla.vla_decay_step(*one, g, S, out=y) for y in one]
    calls += [lambda: vla.vla_head_norm(x, w, out=longer[:, :, 1:]),
              lambda: vla.vla_head_norm_backward(x, q, stats, w, out=longer[:, :, 1:])]
    for call in calls:
        with pytest.raises(vla.VLAError) as e:
            call()
        assert e.value.status == vla._binding.VLA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(everything, before))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [32, 96])
def test_outputs_between_each_others_rows(d, dtype):
    """dq, dk and dv as slices of one projection's gradient [B, T, 3, H, d], whose input's slices are q, k and v."""
    B, H, T = 2, 3, 70
    qkv = torch.randn(B, T, 3, H, d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    do, = seqs(1, B, H, T, d, dtype, seed=2)
    g = torch.tensor([-0.01, -0.1, -1.0], device="cuda")
    dqkv = torch.empty_like(qkv)
    out = [dqkv[:, :, i].transpose(1, 2) for i in range(3)]
    dS0 = torch.empty(B, H, d, d, device="cuda")
    got = vla.vla_decay_backward(q, k, v, g, 0.3, None, do, out=(*out, dS0), check=True)
    check_backward(q, k, v, g, 0.3, None, do, None, None, got)
    # o beside q in the rows of a wider buffer
    wide = torch.randn(B, H, T, 2 * d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dtype)
    left = wide[..., :d].clone()
    got = vla.vla_decay_forward(wide[..., :d], k, v, g, 0.3, out=(wide[..., d:], dS0), check=True)
    assert torch.equal(wide[..., :d], left)
    check_forward(left, k, v, g, 0.3, None, None, got)


# ---- offsets behind 2^31 ------------------------------------------------------------------------------------------

def test_head_norm_weights_behind_two_to_the_31():
    """More than 2^24 heads of 128 values: a head's weight, bias and their gradients lie 2^31 values and more in."""
    H, d = (1 << 24) + 3, 128
    heads = [0, 1, H - 4, H - 3, H - 2, H - 1]
    gen = torch.Generator(device="cuda").manual_seed(0)
    some = lambda *s: torch.randn(*s, len(heads), d, generator=gen, device="cuda")  # noqa: E731
    x, dy = (torch.zeros(1, H, 1, d, dtype=BF, device="cuda") for _ in range(2))
    w, b = (torch.zeros(H, d, device="cuda") for _ in range(2))
    x[0, heads, 0], dy[0, heads, 0] = some().to(BF), some().to(BF)
    w[heads], b[heads] = some(), some()
    part = lambda y: y[:, heads].contiguous()  # noqa: E731
    want_y, stats = vla.vla_head_norm(part(x), w[heads], b[heads])
    want = vla.vla_head_norm_backward(part(dy), part(x), stats, w[heads])
    y, stats = vla.vla_head_norm(x, w, b)
    assert torch.equal(part(y), want_y) and not y[:, 2:H - 4].any()
    del y, b
    dx, dw, db = vla.vla_head_norm_backward(dy, x, stats, w)
    assert torch.equal(part(dx), want[0]) and torch.equal(dw[heads], want[1]) and torch.equal(db[heads], want[2])
    assert not dw[2:H - 4].any() and not db[2:H - 4].any() and not dx[:, 2:H - 4].any()
    # the few heads against the definition
    n = R.norm_grads(part(dy), part(x), w[heads], 1e-5)
    assert float((dw[heads].double().cpu() - n[1]).abs().max()) <= 64 * d * R.U * float(n[3].max())


# ---- waits that run out -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,d", [(9, 32), (64, 96), (70, 128), (700, 64), (1000, 128), (640, 96)])
def test_a_wait_that_runs_out_is_reported(T, d):
    """The last chunk's loads kept back: every block of the call returns within its limit, the call reports it, and the
    next one on the stream is right. In one piece (many heads) and in segments (few)."""
    for B, H in ((1, 2), (2, 160)):
        q, k, v, do = seqs(4, B, H, T, d, BF, seed=T)
        g = -torch.linspace(0.01, 0.5, H).cuda()
        S0 = state_like(B, H, d, 1)
        n = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")
        stall = dict(wait_limit_us=500, test_stall_producer=True, check=True, lengths=n)
        vla.vla_get_last_device_status()
        for _ in range(2):
            with pytest.raises(vla.VLAError) as e:
                vla.vla_decay_forward(q, k, v, g, 0.3, S0, **stall)
            assert e.value.status == vla._binding.VLA_ERR_TIMEOUT and 0 <= e.value.detail[1] < B * H
            with pytest.raises(vla.VLAError) as e:
                vla.vla_decay_backward(q, k, v, g, 0.3, S0, do, S0, **stall)
            assert e.value.status == vla._binding.VLA_ERR_TIMEOUT
        # a limit that nothing reaches, and none given
        fwd = vla.vla_decay_forward(q, k, v, g, 0.3, S0, lengths=n, wait_limit_us=1000000, check=True)
        bwd = vla.vla_decay_backward(q, k, v, g, 0.3, S0, do, S0, lengths=n, check=True)
        pick = [0, H - 1]
        part = lambda x: x[:, pick]  # noqa: E731
        check_forward(part(q), part(k), part(v), g[pick], 0.3, part(S0), n, tuple(part(x) for x in fwd))
        check_backward(part(q), part(k), part(v), g[pick], 0.3, part(S0), part(do), part(S0), n,
                       (tuple(part(x) for x in bwd[0]), part(bwd[1])))


def test_calls_without_waits_do_not_stall():
    for dtype, T in ((F32, 100), (BF, 8)):
        q, k, v = seqs(3, 1, 2, T, 64, dtype)
        g = decays(2)
        got = vla.vla_decay_forward(q, k, v, g, wait_limit_us=500, test_stall_producer=True, check=True)
        check_forward(q, k, v, g, 1.0, None, None, got)


# ---- caches of no slots and of many -------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
def test_cache_without_slots(bits):
    """A server that parks nothing yet: idle rows are skipped and read as fresh states, any slot is out of range."""
    codes, scales = vla.vla_state_cache(0, (2, 32, 32), bits)
    idle = torch.tensor([-1, -1], dtype=torch.int32, device="cuda")
    x = state_like(2, 2, 32, 1)
    vla.vla_state_store(x, codes, scales, idle, check=True)
    assert not vla.vla_state_load(codes, scales, idle, check=True).any()
    assert vla.vla_state_load(codes, scales).shape == (0, 2, 32, 32)
    assert not vla.vla_state_load(codes, scales, idle + 1).any()
    assert vla.vla_get_last_device_status()[0] == vla._binding.VLA_ERR_BAD_SLOT


def test_cache_of_many_slots():
    """More slots than states a call may have: any of them, at most 65,535 at a time."""
    N = 65540
    codes, scales = vla.vla_state_cache(N, (32,), 8)
    x = torch.randn(N, 32, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    for call in (lambda: vla.vla_state_store(x, codes, scales), lambda: vla.vla_state_load(codes, scales),
                 lambda: vla.vla_state_load(codes, scales, slots)):
        with pytest.raises(ValueError, match="65,535"):
            call()
    assert not codes.any()
    vla.vla_state_store(x[:65535], codes, scales, check=True)
    vla.vla_state_store(x[65535:], codes, scales, slots[65535:], check=True)
    got = torch.cat([vla.vla_state_load(codes, scales, s.contiguous(), check=True) for s in (slots[:65535], slots[65535:])])
    assert torch.equal(got.cpu(), R.store(x, 8)[0])
