"""The embedding's gradient into tables of any row stride and address (GPU): what a contiguous
table gets, bit for bit, the join of the runs that cross segments among it."""
import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("t,v,d", [(4000, 40, 512), (3001, 7, 516), (5000, 300, 36), (2000, 3, 515),
                                   (40000, 90, 64)])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 2), (4, 0), (4, 1), (8, 4)])
def test_strided_and_shifted_tables(t, v, d, pad, shift, accumulate):
    g = torch.Generator().manual_seed(t)
    ids = torch.randint(-1, v, (t,), generator=g).cuda()
    dout = torch.randn(t, d, generator=g).bfloat16().cuda()
    start = torch.randn(v, d, generator=g).cuda()
    want = start.clone()
    dion.EmbedGradPlan(ids, dout, want, scale=1.5).backward(accumulate=accumulate)
    buf = torch.full((v * (d + pad) + shift + 8,), 77.0, device="cuda")
    table = buf[shift:shift + v * (d + pad)].view(v, d + pad)[:, :d]
    table.copy_(start)
    dion.EmbedGradPlan(ids, dout, table, scale=1.5).backward(accumulate=accumulate)
    assert torch.equal(table, want)
    table.fill_(77.0)
    assert bool((buf == 77.0).all())
