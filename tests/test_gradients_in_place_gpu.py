"""The norm over rows in place (GPU): every pair of arrays that include/dion.h lets coincide, in
every form of the kernels, with several rows to a CTA, so that rows are fetched ahead while others
are written.  In place equals out of place bit for bit."""
import itertools

import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# (tokens, features, type): rings of aligned rows and of rows off 16 bytes (whose neighbourhoods
# overlap the rows of other CTAs), a warp and a CTA to a row; the forms without a ring
CASES = [(5000, 264, "bf16"), (5000, 260, "bf16"), (4801, 99, "fp16"), (2500, 1015, "bf16"),
         (2500, 1016, "fp16"), (1300, 4096, "bf16"), (1300, 4095, "bf16"), (700, 8192, "bf16"),
         (5000, 264, "fp32"), (2500, 1023, "fp32"), (2500, 1024, "fp32"), (1300, 4096, "fp32"),
         (500, 8200, "bf16"), (500, 12345, "fp16"), (400, 16384, "fp32"), (400, 9001, "fp32")]


def _rows(t, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(t, d, generator=g).to(DT[dtype]).cuda()


def _gains(d):
    g = torch.Generator().manual_seed(9)
    return {k: (1 + 0.2 * torch.randn(d, generator=g)).cuda() for k in ("pre_gain", "post_gain", "gate")}


@pytest.mark.parametrize("t,d,dtype", CASES)
def test_forward(t, d, dtype):
    gains = _gains(d)
    x0, y0 = _rows(t, d, dtype, 1), _rows(t, d, dtype, 2)
    h, u = torch.empty_like(x0), torch.empty_like(x0)
    kept = dion.ActCheckpoint(t, d)
    dion.NormPlan(x0, y0, h=h, u=u, checkpoint=kept, residual_scale=0.5, **gains).forward()
    for h_in, u_in in itertools.product((None, "x"), (None, "x", "y")):
        if h_in == u_in:                    # out of place, or both into x
            continue
        x, y = x0.clone(), y0.clone()
        place = {None: None, "x": x, "y": y}
        ha = torch.empty_like(x) if h_in is None else place[h_in]
        ua = torch.empty_like(x) if u_in is None else place[u_in]
        k = dion.ActCheckpoint(t, d)
        dion.NormPlan(x, y, h=ha, u=ua, checkpoint=k, residual_scale=0.5, **gains).forward()
        assert torch.equal(ha, h) and torch.equal(ua, u), (h_in, u_in)
        assert torch.equal(k.q, kept.q) and torch.equal(k.scale, kept.scale)
    # without y, and without the norm of y
    u2, x = torch.empty_like(x0), x0.clone()
    dion.NormPlan(x0, u=u2, pre_gain=gains["pre_gain"]).forward()
    dion.NormPlan(x, u=x, pre_gain=gains["pre_gain"]).forward()
    assert torch.equal(x, u2)


@pytest.mark.parametrize("t,d,dtype", CASES)
def test_backward(t, d, dtype):
    gains = _gains(d)
    src = {k: _rows(t, d, dtype, i) for i, k in enumerate(("h", "y", "du", "dh"))}
    new = lambda: {k: torch.empty(d, device="cuda") for k in ("dpre_gain", "dpost_gain", "dgate")}  # noqa: E731
    dx, dy, want = torch.empty_like(src["h"]), torch.empty_like(src["h"]), new()

    def run(a, dx, dy, grads):
        dion.NormGradPlan(a["h"], a["y"], du=a["du"], dh=a["dh"], dx=dx, dy=dy, residual_scale=0.5,
                          **gains, **grads).backward()

    run(src, dx, dy, want)
    for dx_in, dy_in in itertools.product((None, "dh", "du", "h"), (None, "y", "du")):
        if dx_in == dy_in:                  # out of place, or both into du
            continue
        a, got = {k: v.clone() for k, v in src.items()}, new()
        dxa = torch.empty_like(dx) if dx_in is None else a[dx_in]
        dya = torch.empty_like(dy) if dy_in is None else a[dy_in]
        run(a, dxa, dya, got)
        assert torch.equal(dxa, dx) and torch.equal(dya, dy), (dx_in, dy_in)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, dx_in, dy_in)
