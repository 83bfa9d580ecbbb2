"""GPU tests of the plain-operand products, the int8 quantisers and the AdamW step at the ends of what their
contract allows: offsets out of order, values near the ends of fp32, long sums and long tensors."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,M", [(6, 6144), (7, 6272), (49, 768)])
def test_offsets_out_of_order_list_more_tiles_than_a_small_launch_counts(G, M):
    """Every other expert claims all rows, so the list is longer than any valid offsets' and a workgroup of a small
    launch takes several of its tiles.  All experts have the same weights, so every tile computed writes the same
    values: the outputs are the product, and nothing around them is written."""
    m = require_gpu()
    N, K = 128, 64
    gen = torch.Generator(device="cuda").manual_seed(G)
    offs = torch.tensor([(g % 2) * M for g in range(G + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(N, K, device="cuda", generator=gen).bfloat16()
    y, dx, y8 = (torch.full((M * c + 4096,), 3.0, device="cuda") for c in (N, K, N))
    m.bf16_grouped_gemm_fwd(x, w.repeat(G, 1), offs, N, y=y[:M * N].view(M, N))
    dy = torch.randn(M, N, device="cuda", generator=gen).bfloat16()
    m.bf16_grouped_gemm_dgrad(dy, w.repeat(G, 1), offs, K, dx=dx[:M * K].view(M, K))
    qx, sx = m.int8_quantize_rowwise(x)
    qw, sw = m.int8_quantize_rowwise(w)
    m.int8_grouped_gemm_fwd(qx, sx, qw.repeat(G, 1), sw.repeat(G), offs, N, y=y8[:M * N].view(M, N))
    for t in (y, dx, y8):
        assert (t[-4096:] == 3.0).all()
    for got, a, b in ((y, x, w.t().contiguous()), (dx, dy, w)):
        a, b = a.double(), b.double()
        assert bool(((got[:-4096].view(M, -1).double() - a @ b).abs() <= 1e-5 * (a.abs() @ b.abs())).all())
    ref = (qx.double() @ qw.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    assert bool(((y8[:-4096].view(M, N).double() - ref).abs() <= 2.0 ** -22 * ref.abs()).all())
