"""Weight gradients whose device waits run out (GPU): the limit of the plan's options reaches
them through the step from kept activations, the kernels give up and free what they hold, say so,
and the calls after are what they are without it.  The step leaves the matrices of such gradients
alone.  It runs on the CUDA-core kernels where nothing is said, which wait for nothing."""
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
    """A gradient that is not marked is right, whatever the limit, and every entry of a marked one is
    right or as it was; one poll is less than one load takes.  The call after it is right."""
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
        assert bool(((G == 7.0) | (G == want)).all())
        assert marked or limit > 1 or t == 1
        # accumulating: nothing but the gradient itself is added to an earlier micro-batch
        G.copy_(want)
        saved.grad_status.zero_()
        saved.step([X.clone()], [M.clone()], [G], [Q.clone()], 0.01, accumulate=True)
        torch.cuda.synchronize()
        assert bool(((G == want) | (G == want + want)).all())
        assert int(saved.grad_status[0]) or torch.equal(G, want + want)
        plan.backward()
        torch.cuda.synchronize()
        assert torch.equal(G, want) and not plan.status.any()


@pytest.mark.parametrize("limit", [1, 8, 32, 128, 512])
@pytest.mark.parametrize("path,precision", [("simt", "bf16"), ("simt", "fp32"), ("tensor", "bf16"),
                                            ("tensor", "fp32")])
def test_the_step_leaves_a_marked_matrix_alone(path, precision, limit):
    """Of a bucket's four matrices two have no tokens, so that their gradients wait for nothing."""
    m, n, count = 264, 200, 4
    kept, dys, X, M, Q = _inputs(3000, m, n, count)
    for i in (1, 3):
        kept[i] = dion.ActCheckpoint(0, m)
        dys[i] = torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    G = torch.zeros(count, m, n, device="cuda")
    opt = dion.DionB200([(count, m, n, 16)], kernel_path=path, precision=precision)
    want = [v.clone() for v in (X, M, Q)]
    dion.SavedStep(opt, kept, dys).step([want[0]], [want[1]], [G], [want[2]], 0.01)
    short = dion.DionB200([(count, m, n, 16)], kernel_path=path, precision=precision,
                          max_wait_spins=limit)
    for _ in range(3):
        saved, status = dion.SavedStep(short, kept, dys), opt.alloc_status()
        got = [v.clone() for v in (X, M, Q)]
        saved.step([got[0]], [got[1]], [G], [got[2]], 0.01, status=status)
        torch.cuda.synchronize()
        marked, stepped = saved.grad_status.tolist(), status.tolist()
        assert marked[1] == marked[3] == 0 and (limit > 1 or marked[0] == marked[2] == TIMEOUT)
        for i in range(count):
            if marked[i]:
                assert stepped[i] & TIMEOUT
                for a, b in zip(got, (X, M, Q)):
                    assert torch.equal(a[i], b[i])
            elif not stepped[i] & TIMEOUT:
                for a, b in zip(got, want):
                    assert torch.equal(a[i], b[i])
            else:
                assert path == "tensor"          # its own waits ran out


def test_marks_are_of_the_call():
    """A mark in grad_status stays until it is cleared; what the step does goes by its own call."""
    m, n = 264, 200
    kept, dys, X, M, Q = _inputs(3000, m, n)
    G = torch.zeros(1, m, n, device="cuda")
    opt = dion.DionB200([(1, m, n, 16)])
    saved, status = dion.SavedStep(opt, kept, dys), opt.alloc_status()
    saved.grad_status.fill_(TIMEOUT)
    before = X.clone()
    saved.step([X], [M], [G], [Q], 0.01, status=status)
    torch.cuda.synchronize()
    assert int(saved.grad_status[0]) == TIMEOUT and not int(status[0]) & TIMEOUT
    assert not torch.equal(X, before) and bool(torch.isfinite(X).all())


@pytest.mark.parametrize("r", [16, 272])
def test_the_step_captured_and_replayed(r):
    """The words of the call are cleared in each replay, too."""
    m, n, count = 512, 288, 2
    kept, dys, X, M, Q = _inputs(900, m, n, count)
    Q = torch.nn.functional.normalize(torch.randn(count, n, r, generator=torch.Generator().manual_seed(2)),
                                      dim=1).cuda()
    G = torch.zeros(count, m, n, device="cuda")
    opt = dion.DionB200([(count, m, n, r)])
    saved, status = dion.SavedStep(opt, kept, dys), opt.alloc_status()
    want, state = [[v.clone() for v in (X, M, Q)] for _ in range(2)]
    for _ in range(3):
        saved.step([want[0]], [want[1]], [G], [want[2]], 0.01, status=status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saved.step([state[0]], [state[1]], [G], [state[2]], 0.01, status=status)
    for _ in range(3):
        status.fill_(-1)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(state, want):
        assert torch.equal(a, b)
    assert not (status & TIMEOUT).any() and not saved.grad_status.any()
