"""Weight gradients of 8-bit rows over the whole range of their block exponents, and with the
exponent bytes at any address (GPU), against fp64.

The bound is the one of the weight gradients near 1 (the values scale by powers of two, exactly):
a chunk of 1024 tokens takes 64 additions in the tensor cores, each cut off by at most 2^-23 of a
running absolute sum that grows from nothing, 2^-18 of the chunk's; chunks, splits and the join
are fp32 additions: (2^-18 + (T / 256 + 8) 2^-24) sum |a| |d|.  Every product and sum here lies
within fp32's normal numbers or is exactly zero."""
import numpy as np
import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion
from oracle import gradient_oracle as go

pytestmark = pytest.mark.gpu

# (tokens, m, n): converted in the kernel (two widths of tile), and beforehand
SHAPES = [(300, 200, 96), (1000, 256, 128), (700, 333, 700), (640, 264, 1600)]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _kept(t, m, exponents, seed, skew=0):
    """8-bit rows whose block exponents are drawn from `exponents` (bytes), every e4m3 value among
    them, the scale bytes `skew` past an aligned address."""
    ld = -(-m // 32) * 32
    q = torch.randint(0, 256, (t, ld), generator=_gen(seed), dtype=torch.int64)
    q = torch.where(q % 128 == 127, q - 1, q).to(torch.uint8)     # no NaN bytes
    q[:, m:] = 0
    pick = torch.randint(0, len(exponents), (t, ld // 32), generator=_gen(seed + 1))
    scale = torch.tensor(exponents, dtype=torch.uint8)[pick]
    buf = torch.full((t * ld // 32 + 16,), 255, dtype=torch.uint8, device="cuda")
    place = buf[skew:skew + t * ld // 32].view(t, ld // 32)
    place.copy_(scale.cuda())
    kept = dion.ActCheckpoint(t, m, q=q.cuda(), scale=place)
    return kept, go.act_value(q.numpy(), scale.numpy(), m)


def _check(kept, a, d, t, m, n):
    for transposed in (False, True):
        G = torch.empty((n, m) if transposed else (m, n), device="cuda")
        dion.WeightGradPlan([kept], [d], [G], transposed=transposed).backward()
        dn = d.cpu().double().numpy()
        ref = go.weight_grad(a, dn, transposed)
        bound = (2.0 ** -18 + (t / 256 + 8) * 2.0 ** -24) * go.weight_grad(np.abs(a), np.abs(dn), transposed)
        assert np.all(np.abs(G.cpu().double().numpy() - ref) <= bound)


# exponent bytes of a case and the size of D that keeps the sums within fp32: the border of the
# converter's one and two products (134), the largest, the smallest, all of them about 1
@pytest.mark.parametrize("exponents,size", [
    ([133, 134, 135, 136], 1e-3), ([134], 1.0), ([135], 1.0), ([120, 125, 130, 140, 150], 1e-6),
    ([240, 243, 246], 1e-12), ([10, 11, 13, 20], 1e20), ([100, 127, 160], 1e-8)])
@pytest.mark.parametrize("t,m,n", SHAPES)
def test_exponents(t, m, n, exponents, size):
    kept, a = _kept(t, m, exponents, 5)
    d = (size * torch.randn(t, n, generator=_gen(7))).bfloat16().cuda()
    _check(kept, a, d, t, m, n)


@pytest.mark.parametrize("t,m,n", SHAPES)
def test_large_activations_kept_and_used(t, m, n):
    """Rows of 1e5 to 1e6 (exponents above 134), kept by save."""
    x = 10.0 ** torch.empty(t, m).uniform_(5, 6, generator=_gen(1)) * torch.randn(t, m, generator=_gen(2)).sign()
    kept = dion.ActCheckpoint(t, m)
    kept.save(x.cuda())
    assert int(kept.scale.min()) > 134
    a = go.act_value(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), m)
    assert np.all(np.abs(a - x.double().numpy()) <= 2.0 ** -4 * np.abs(x.double().numpy()))
    _check(kept, a, torch.randn(t, n, generator=_gen(3)).bfloat16().cuda(), t, m, n)


@pytest.mark.parametrize("skew", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("t,m,n", SHAPES + [(1, 40, 16), (65, 128, 64), (130, 1024, 64), (64, 31, 8)])
def test_scale_bytes_at_any_address(t, m, n, skew):
    """Their neighbours in memory are 255, which would make NaN of what they scale."""
    kept, a = _kept(t, m, [126, 127, 129, 131], 11, skew)
    _check(kept, a, torch.randn(t, n, generator=_gen(4)).bfloat16().cuda(), t, m, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 65])
def test_magnitudes_past_the_form_are_cut(dtype, d):
    """Above 448 * 2^119 a value reads as that, up to it within half a step; an infinity is NaN."""
    top = 448.0 * 2.0 ** 119
    x = torch.zeros(4, d, dtype=dtype, device="cuda")
    x[0, 3], x[0, 5], x[0, 6] = torch.finfo(dtype).max, -torch.finfo(dtype).max, 1e38
    x[1, 40], x[1, 41] = top, 3.2e38
    x[2, 0] = float("inf")
    kept = dion.ActCheckpoint(4, d)
    kept.save(x)
    out = kept.load(torch.empty(4, d, device="cuda")).cpu().double()
    assert out[0, 3] == top and out[0, 5] == -top and out[1, 40] == top and out[1, 41] == top
    ref, scale = go.act_round(x.cpu().double().numpy())
    assert np.array_equal(out.numpy(), ref, equal_nan=True)
    assert np.array_equal(kept.scale.cpu().numpy(), scale)
    assert bool(torch.isnan(out[2, :32]).all()) and not out[3].any()
