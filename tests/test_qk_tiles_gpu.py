"""Norm and rotation of queries and keys on the GPU where a block takes several tiles of tokens, as long training
batches have it: against the fp64 form."""
import pytest
import torch

import delta_ref as R
import sherman_morrison_memory_gb300 as vla
from test_layer_gpu import seqs
from test_qk_gpu import BF, F32, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kind", [(BF, "shared"), (BF, "heads"), (F32, "shared"), (F32, "heads")])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("tiles", [2, 4, 8])
def test_several_tiles_a_block(tiles, d, dtype, kind):
    """Gradients by blocks of 2, 4 and 8 tiles, the last of fewer, its last tile cut off; each sequence at its own
    positions, so that a tile's angles are its own."""
    B, H = 3, 8
    tile = {32: 128, 64: 64, 96: 40, 128: 32}[d]  # tokens of a tile
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count  # as many at least, before a block takes more
    spans = -(-blocks // (B * H // 4))
    count = (spans - 1) * tiles + tiles // 2
    T = (count - 1) * tile + tile // 2 + 1
    assert vla.load_library().vla_qk_norm_scratch_bytes(B, H, T, d) == B * spans * 2 * H * d * 4  # a block's tiles are `tiles`
    q, k, gq, gk = seqs(4, B, H, T, d, dtype, seed=T)
    w = weights(kind, H, d)
    freqs = vla.vla_rotation_frequencies(d // 2 // 16 * 16)
    first = torch.tensor([[0], [70001], [-5]], dtype=torch.int32, device="cuda")
    pos = first + torch.arange(T, dtype=torch.int32, device="cuda")
    y, stats = vla.vla_qk_norm(q, k, *w, 1e-6, freqs=freqs, positions=pos)
    dx, dw = vla.vla_qk_norm_backward(gq, gk, q, k, stats, *w, freqs=freqs, positions=pos)
    half = R.HALF[dtype] if dtype == BF else 0.0
    u = (d // 16 + 4 + 2 + 8) * R.U + 4 * 2.0 ** -53 * float(pos.abs().max()) * float(freqs.max())
    row = lambda a: a.norm(dim=-1, keepdim=True)  # noqa: E731
    for x, g, wt, yi, s, dxi, dwi in zip((q, k), (gq, gk), w, y, stats, dx, dw):
        x6, w6, g6 = x.double().requires_grad_(), wt.double().requires_grad_(), g.double()
        y6, r6 = R.qk(x6, w6, False, 1e-6, freqs, pos)
        (y6 * g6).sum().backward()
        with torch.no_grad():
            assert bool(((yi.double() - y6).abs() <= half * y6.abs() + u * row(y6) + 1e-30).all())
            assert bool(((s.double() - r6).abs() <= u * r6).all())
            size = r6[..., None] * row(g6) * float(wt.abs().max())
            assert bool(((dxi.double() - x6.grad).abs() <= half * x6.grad.abs() + 4 * u * size + 1e-30).all())
            # a lane adds a row of eight to its sum, in every tile of the block, before the sums of blocks are added
            terms = (row(g6) * (row(y6) + (x6 * r6[..., None]).abs())).sum((0, 1, 2) if wt.dim() == 1 else (0, 2))
            assert bool(((dwi.double() - w6.grad).abs() <= (2 * u + (16 + T // 16) * R.U) * terms).all())
