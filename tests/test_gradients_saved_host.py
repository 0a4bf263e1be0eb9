"""The step from kept activations, on the host: its workspace holds a word per matrix beside what
the gradients and the step need, and is checked for it; the wait limit is the handle's (no GPU)."""
import pytest

import rank_orthonormalized_optimizer_b200 as dion
from rank_orthonormalized_optimizer_b200 import gradients as gr

FAKE = 1 << 20          # an aligned address that is never dereferenced
REACHED = (dion.OK, dion.ERR_CUDA, dion.ERR_DEVICE)


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


pytestmark = pytest.mark.skipif(not _no_gpu(), reason="valid calls would launch on fake pointers")


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
