"""The step from kept activations, on the host: its workspace holds a word per matrix beside what
the gradients and the step need, and is checked for it; the wait limit is the handle's (no GPU)."""
import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion
from rank_orthonormalized_optimizer_b200 import gradients as gr
from test_gradients_memory import FakeCuda, _rows, fake  # noqa: F401

FAKE = 1 << 20          # an aligned address that is never dereferenced
REACHED = (dion.OK, dion.ERR_CUDA, dion.ERR_DEVICE)


pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would launch on fake pointers")


def _sources(count, tokens):
    return (gr.GradSource * count)(*[
        gr.GradSource(kept=gr.ActKept(FAKE, FAKE, tokens, 64), d=FAKE, ldd=32, n=32, G=None, ldg=0,
                      transposed=0) for _ in range(count)])


@pytest.mark.parametrize("count,tokens", [(1, 8), (3, 8), (7, 1 << 14)])
def test_the_workspace_holds_a_word_per_matrix(count, tokens):
    opt = dion.DionB200([(count, 64, 32, 16)])
    src = _sources(count, tokens)
    ptrs = (dion.BucketPtrs * 1)(dion.BucketPtrs(FAKE, FAKE, FAKE, FAKE))
    need = gr.dion_step_from_saved_workspace(opt._h, src, count)
    grads = gr.dion_weight_grad_workspace(src, count)
    assert need >= max(opt.workspace_bytes, grads) + 4 * count
    call = lambda b, grad_status=None: gr.dion_step_batched_from_saved(  # noqa: E731
        opt._h, ptrs, src, 1, 0, 0.1, FAKE, b, None, grad_status, None)
    assert call(need) in REACHED
    assert call(need, FAKE) in REACHED
    assert call(need - 1) == dion.ERR_WORKSPACE_TOO_SMALL
    assert call(need, FAKE + 2) == dion.ERR_MISALIGNED
    opt.close()


class Elsewhere(FakeCuda):
    device = property(lambda self: torch.device("cuda", 1))


def test_a_step_refuses_tensors_of_another_device_and_a_status_that_does_not_fit(fake):
    """Such pointers would reach the kernels (the plan's own tensors are on cuda:0)."""
    kept = dion.ActCheckpoint(64, 32)
    opt = dion.DionB200([(1, 32, 32, 16)])
    step = dion.SavedStep(opt, [kept], [_rows(64, 32, torch.bfloat16)])
    good = [[torch.ones(1, 32, n).as_subclass(FakeCuda)] for n in (32, 32, 32, 16)]
    step.step(*good, 0.1)
    for i, name in enumerate("XMGQ"):
        bad = list(good)
        bad[i] = [good[i][0].as_subclass(Elsewhere)]
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            step.step(*bad, 0.1)
    words = torch.ones(1, dtype=torch.int32)
    step.step(*good, 0.1, status=words.as_subclass(FakeCuda))
    for bad in (words, words.as_subclass(Elsewhere), torch.ones(1).as_subclass(FakeCuda),
                torch.ones(0, dtype=torch.int32).as_subclass(FakeCuda), [0]):
        with pytest.raises(ValueError, match="status must be 1 contiguous int32"):
            step.step(*good, 0.1, status=bad)
    opt.close()
