"""Weight gradients whose device waits run out (GPU): the limit of the plan's options reaches
them through the step from kept activations, the kernels give up and free what they hold, say so,
and the calls after are what they are without it.  The step itself runs on the CUDA-core kernels
here, which wait for nothing."""
import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion

pytestmark = pytest.mark.gpu

TIMEOUT = 8      # DION_MAT_TIMEOUT

# (tokens, m, n): converted in the kernel over 128 and 256 columns, whole and split over the
# tokens, one tile a pair and several; converted beforehand (from 1536 columns and 512 tokens on)
SHAPES = [(1, 64, 64), (700, 256, 128), (4099, 256, 128), (130, 304, 704), (3000, 264, 200),
          (300, 2504, 3000), (640, 520, 2048), (8192, 304, 1600), (2000, 2504, 3000)]


def _inputs(t, m, n, count=1):
    g = torch.Generator().manual_seed(t + m + n)
    kept, dys = [], []
    for _ in range(count):
        k = dion.ActCheckpoint(t, m)
        k.save(torch.randn(t, m, generator=g).cuda())
        kept.append(k)
        dys.append(torch.randn(t, n, generator=g).bfloat16().cuda())
    X, M = (torch.randn(count, m, n, generator=g).cuda() for _ in range(2))
    Q = torch.nn.functional.normalize(torch.randn(count, n, 16, generator=g), dim=1).cuda()
    return kept, dys, X, M, Q


@pytest.mark.parametrize("limit", [1, 3, 20, 200])
@pytest.mark.parametrize("t,m,n", SHAPES)
def test_waits_run_out_cleanly(t, m, n, limit):
    """A gradient that is not marked is right, whatever the limit; one poll is less than one load
    takes.  The call after it is right in any case."""
    kept, dys, X, M, Q = _inputs(t, m, n)
    G = torch.zeros(1, m, n, device="cuda")
    plan = dion.WeightGradPlan(kept, dys, [G[0]])
    plan.backward()
    want = G.clone()
    short = dion.DionB200([(1, m, n, 16)], kernel_path="simt", max_wait_spins=limit)
    for _ in range(3):
        saved = dion.SavedStep(short, kept, dys)
        G.fill_(7.0)
        saved.step([X.clone()], [M.clone()], [G], [Q.clone()], 0.01)
        torch.cuda.synchronize()
        marked = int(saved.grad_status[0])
        assert marked == TIMEOUT or (marked == 0 and torch.equal(G, want))
        assert marked or limit > 1 or t == 1
        G.fill_(7.0)
        plan.backward()
        torch.cuda.synchronize()
        assert torch.equal(G, want) and not plan.status.any()
