"""Normwise accuracy of the decayed linear attention on the GPU (limits derived in layer_accuracy.py): every output in
blocks of 128 rows, every final state, forward and gradients, in one piece, in segments and padded."""
import pytest
import torch

import layer_accuracy as A
import layer_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import decays, seqs, state_like

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,T,d,lengths", [
    (2, 4, 200, 128, None), (1, 4, 1000, 128, None), (1, 4, 1000, 96, None), (2, 4, 700, 64, None), (3, 5, 333, 32, None),
    (2, 4, 900, 32, [900, 641]), (3, 3, 515, 96, [515, 130, 400]), (2, 80, 256, 64, None)])
def test_norms_of_errors(B, H, T, d, lengths, dtype):
    q, k, v, do = seqs(4, B, H, T, d, dtype, seed=T + d)
    S0, dS = state_like(B, H, d, 1), state_like(B, H, d, 2)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    rows = A.ROWS if dtype == BF else A.ROWS32
    for g in (decays(H), torch.full((H,), -1e-4, device="cuda")):
        o, S = vla.vla_decay_forward(q, k, v, g, 0.3, S0, lengths=n, check=True)
        grads, dS0 = vla.vla_decay_backward(q, k, v, g, 0.3, S0, do, dS, lengths=n, check=True)
        ro, rS = R.decay(q, k, v, g, 0.3, S0, n)
        ref = R.decay_grads(q, k, v, g, 0.3, S0, do, dS, n)
        for b in range(B):  # blocks of each sequence's own rows
            m = T if lengths is None else lengths[b]
            for name, x, r in zip(("o", "dq", "dk", "dv"), (o, *grads), (ro, *ref[:3])):
                worst = float(A.block_errors(x[b:b + 1, :, :m], r[b:b + 1, :, :m]).max())
                assert worst <= rows, (name, b, worst)
        for name, x, r in (("S", S, rS), ("dS0", dS0, ref[3])):
            finite = r.flatten(2).norm(dim=-1) > 0  # a head that forgets everything has no dS0
            worst = float(A.state_errors(x, r)[finite].max())
            assert worst <= A.STATES, (name, worst)
            assert not x.cpu()[~finite].any()
