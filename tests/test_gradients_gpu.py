"""Parity of the gradient operators with their fp64 oracle (GPU).

Tolerances, each from counting roundings (u = 2^-24, fp32's half step; half = half a step of
the stored type: bf16 2^-8, fp16 2^-11, fp32 2^-24).

norm: a row sum runs over at most 32 terms in a thread, 5 shuffles and 16 warps, so its
  error is below 2^-18 of the sum of absolute terms; everything else is a handful of
  roundings.  h: half |h| + 2^-21 (|x| + |s gate z|) + 2^-18 |s gate z|; u: half |u| + 2^-17 of
  |pre_gain| rms(h) (|x| + |s gate z|).  Backward, with A = |dh| + r (|w| + |hn| mean|w hn|)
  the sum of absolute terms of dx: half |dx| + 2^-17 A; dy likewise from |c| A; a column sum
  over T rows adds T / 148 + 60 terms one after the other: below 2^-16 of the absolute sum for
  T <= 10^4 (the gradient A itself is off by 2^-17).
act: exact (the same rounding rule): values must be equal.
weight_grad: products are exact; a chunk of 1024 tokens takes 64 tensor-core additions, each
  cut off by at most 2^-23 of the running absolute sum, which grows from nothing to the
  chunk's: 64 * 2^-23 / 2 = 2^-18 of it; the chunks and splits are added in fp32:
  2^-18 + (T / 256 + 8) u of sum |a| |d|.
embedding: lookup half |out| + u |out|; the gradient of a token met k times
  (k + 2) u of scale * sum |dout|.
A stored fp16 value below its smallest normal is off by up to 2^-25.
"""
import numpy as np
import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion
from oracle import gradient_oracle as go

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
U = 2.0 ** -24


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


class Rows:
    """A [t, d] tensor inside a wider buffer of sentinels, so that writes outside show.
    pad: extra columns; shift: elements before the first row (breaks the alignment)."""

    def __init__(self, t, d, dtype, pad=0, shift=0, fill=None, seed=0, size=1.0):
        self.buf = torch.full(((t + 1) * (d + pad) + shift + 8,), 77.0, dtype=dtype, device="cuda")
        self.t = self.buf[shift:shift + t * (d + pad)].view(t, d + pad)[:, :d]
        mask = torch.zeros_like(self.buf, dtype=torch.bool)
        mask[shift:shift + t * (d + pad)].view(t, d + pad)[:, :d] = True
        self.outside = ~mask
        if fill is not None:
            self.t.copy_((size * torch.randn(t, d, generator=_gen(seed))).to(dtype).cuda())

    def clean(self):
        return bool((self.buf[self.outside] == 77.0).all())


# (tokens, features, pad, shift): a row of one, odd widths, widths at the borders of the
# kernel's forms (256, 512, 1024, 2048, 4096, 8192), strided and unaligned rows
NORM_SHAPES = [(1, 1, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0), (4, 256, 0, 0), (9, 264, 0, 0),
               (2, 512, 8, 0), (7, 1000, 0, 0), (6, 1024, 0, 0), (3, 1023, 1, 0), (5, 1032, 0, 0),
               (4, 2048, 0, 0), (3, 2056, 24, 0), (2, 4096, 0, 0), (600, 4096, 0, 0),
               (2, 4097, 0, 0), (3, 8192, 0, 0), (2, 8200, 0, 0), (2, 16384, 0, 0),
               (2, 12345, 0, 0), (4, 512, 0, 1), (3, 4096, 3, 5), (1300, 96, 0, 0),
               # batches that are streamed, ragged in rows and columns
               (4801, 104, 0, 0), (5000, 264, 8, 0), (2500, 1016, 0, 0), (1201, 2048, 0, 0),
               (607, 4088, 8, 0), (301, 8192, 0, 0), (301, 8200, 0, 0),
               (700, 5120, 0, 0), (450, 4104, 8, 0), (450, 6144, 0, 0), (301, 6001, 0, 0), (301, 5122, 0, 1),
               (2000, 1280, 0, 0), (1500, 1531, 0, 0), (1000, 2552, 0, 0), (900, 2301, 0, 0),
               (607, 4095, 0, 0), (1203, 2041, 3, 5), (2500, 1015, 0, 1), (5000, 261, 0, 0),
               (4801, 99, 2, 3), (301, 8191, 1, 7)]


def _norm_inputs(t, d, pad, shift, dtype, seed):
    r = {n: Rows(t, d, DT[dtype], pad, shift, fill=True, seed=seed + i, size=z)
         for i, (n, z) in enumerate((("x", 2.0), ("y", 0.5), ("du", 0.1), ("dh", 0.1)))}
    g = [1 + 0.2 * torch.randn(d, generator=_gen(seed + 9 + i)) for i in range(3)]
    return r, {n: v.cuda() for n, v in zip(("pre_gain", "post_gain", "gate"), g)}


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,d,pad,shift", NORM_SHAPES)
def test_norm_forward(t, d, pad, shift, dtype):
    r, g = _norm_inputs(t, d, pad, shift, dtype, 100)
    h, u = Rows(t, d, DT[dtype], pad, shift), Rows(t, d, DT[dtype], pad, shift)
    kept = dion.ActCheckpoint(t, d)
    dion.NormPlan(r["x"].t, r["y"].t, h=h.t, u=u.t, **g, residual_scale=0.5, eps=1e-5,
                  checkpoint=kept).forward()
    torch.cuda.synchronize()
    n = {k: _np(v) for k, v in g.items()}
    x, y = _np(r["x"].t), _np(r["y"].t)
    rh, ru = go.norm_forward(x, y, **n, residual_scale=0.5, eps=1e-5)
    z = np.abs(rh - x)
    terms = np.abs(x) + z
    assert np.all(np.abs(_np(h.t) - rh) <= HALF[dtype] * np.abs(rh) + 2.0 ** -21 * terms
                  + 2.0 ** -18 * z + TINY[dtype])
    rms = 1 / np.sqrt(np.mean(rh * rh, 1, keepdims=True) + 1e-5)
    ub = 2.0 ** -17 * np.abs(n["pre_gain"]) * rms * terms
    assert np.all(np.abs(_np(u.t) - ru) <= HALF[dtype] * np.abs(ru) + ub + TINY[dtype])
    assert h.clean() and u.clean()
    # the 8-bit form holds u within half a step of 3 fraction bits of the fp32 u
    v = go.act_value(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), d)
    top = np.repeat(np.stack([np.abs(ru[:, i:i + 32]).max(1) for i in range(0, d, 32)], 1), 32, 1)[:, :d]
    assert np.all(np.abs(v - ru) <= 2.0 ** -4 * np.abs(ru) + 2.0 ** -16 * top + 2 * ub)
    assert not kept.q[:, d:].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,d,pad,shift", NORM_SHAPES)
def test_norm_backward(t, d, pad, shift, dtype):
    r, g = _norm_inputs(t, d, pad, shift, dtype, 200)
    dx, dy = Rows(t, d, DT[dtype], pad, shift), Rows(t, d, DT[dtype], pad, shift)
    grads = {n: torch.full((d,), 5.0, device="cuda") for n in ("dpre_gain", "dpost_gain", "dgate")}
    plan = dion.NormGradPlan(r["x"].t, r["y"].t, du=r["du"].t, dh=r["dh"].t, dx=dx.t, dy=dy.t, **g,
                             **grads, residual_scale=0.5, eps=1e-5)
    plan.backward()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in grads.items()}
    _check_norm_backward(r, g, dtype, dx, dy, grads, 0.5)
    assert dx.clean() and dy.clean()
    plan.backward(accumulate=True)           # adds the same again, bit for bit twice
    torch.cuda.synchronize()
    for k, v in grads.items():
        assert torch.equal(v, first[k] + first[k]), k


def _check_norm_backward(r, g, dtype, dx, dy, grads, s):
    n = {k: _np(v) for k, v in g.items()}
    h, y, du, dh = (_np(r[k].t) for k in ("x", "y", "du", "dh"))
    ref = go.norm_backward(h, y, du=du, dh=dh, **n, residual_scale=s, eps=1e-5)
    rh = 1 / np.sqrt(np.mean(h * h, 1, keepdims=True) + 1e-5)
    ry = 1 / np.sqrt(np.mean(y * y, 1, keepdims=True) + 1e-5)
    w, hn, yn = np.abs(n["pre_gain"] * du), np.abs(h * rh), np.abs(y * ry)
    A = np.abs(dh) + rh * (w + hn * np.mean(w * hn, 1, keepdims=True))
    c = np.abs(s * n["gate"] * n["post_gain"])
    B = ry * (c * A + yn * np.mean(c * A * yn, 1, keepdims=True))
    assert np.all(np.abs(_np(dx.t) - ref["dx"]) <= HALF[dtype] * np.abs(ref["dx"]) + 2.0 ** -17 * A
                  + TINY[dtype])
    assert np.all(np.abs(_np(dy.t) - ref["dy"]) <= HALF[dtype] * np.abs(ref["dy"]) + 2.0 ** -15 * B
                  + TINY[dtype])
    S = np.sum(A * yn, 0)
    bounds = {"dpre_gain": np.sum(np.abs(du) * hn, 0), "dpost_gain": np.abs(s * n["gate"]) * S,
              "dgate": np.abs(s * n["post_gain"]) * S}
    for k, b in bounds.items():
        assert np.all(np.abs(_np(grads[k]) - ref[k]) <= 2.0 ** -15 * b + 1e-30), k


@pytest.mark.parametrize("case", ["pre", "pre_no_gain", "residual", "gate_only", "post_no_u",
                                  "du_only", "dh_only"])
def test_norm_forms(case):
    """The forms with parts left out, against the same oracle (bf16, 33 x 1536)."""
    t, d = 33, 1536
    r, g = _norm_inputs(t, d, 0, 0, "bf16", 300)
    x, y = r["x"].t, r["y"].t
    has_y = case not in ("pre", "pre_no_gain")
    fw = {"pre": dict(pre_gain=g["pre_gain"]), "pre_no_gain": {}, "residual": {},
          "gate_only": dict(gate=g["gate"], pre_gain=g["pre_gain"]),
          "post_no_u": dict(post_gain=g["post_gain"])}.get(case, dict(g))
    h = torch.empty_like(x) if has_y else None
    u = None if case == "post_no_u" else torch.empty_like(x)
    dion.NormPlan(x, y if has_y else None, h=h, u=u, residual_scale=0.7, eps=1e-4, **fw).forward()
    rh, ru = go.norm_forward(_np(x), _np(y) if has_y else None, residual_scale=0.7, eps=1e-4,
                             **{k: _np(v) for k, v in fw.items()})
    torch.cuda.synchronize()
    if has_y:
        assert np.all(np.abs(_np(h) - rh) <= 2.0 ** -8 * np.abs(rh) + 2.0 ** -18 * 8)
    if u is not None:
        assert np.all(np.abs(_np(u) - ru) <= 2.0 ** -8 * np.abs(ru) + 2.0 ** -16 * 8)
    # and back, at the stored h
    at = h if has_y else x
    du = None if u is None or case == "dh_only" else r["du"].t
    dh = None if case in ("pre", "pre_no_gain", "du_only") else r["dh"].t
    bw = {k: v for k, v in fw.items() if k != "pre_gain" or du is not None}
    out = {"dx": torch.empty_like(x)}
    if has_y:
        out |= {"dy": torch.empty_like(x), "dgate": torch.empty(d, device="cuda")}
    if du is not None:
        out["dpre_gain"] = torch.empty(d, device="cuda")
    dion.NormGradPlan(at, y if has_y else None, du=du, dh=dh, residual_scale=0.7, eps=1e-4, **bw,
                      **out).backward()
    torch.cuda.synchronize()
    ref = go.norm_backward(_np(at), _np(y) if has_y else None, du=_np(du), dh=_np(dh),
                           residual_scale=0.7, eps=1e-4, **{k: _np(v) for k, v in bw.items()})
    for k, v in out.items():
        scale = np.abs(ref[k]).max()
        tol = (2.0 ** -8 * np.abs(ref[k]) + 2.0 ** -15 * scale) if k in ("dx", "dy") \
            else 2.0 ** -15 * t ** 0.5 * scale
        assert np.all(np.abs(_np(v) - ref[k]) <= tol), k


def test_norm_in_place_equals_out_of_place():
    """h may be x, u may be y; dx may be dh or du, dy may be y (same rows)."""
    for t, d in ((50, 4096), (50, 260)):
        r, g = _norm_inputs(t, d, 0, 0, "bf16", 400)
        h, u = torch.empty_like(r["x"].t), torch.empty_like(r["x"].t)
        dion.NormPlan(r["x"].t, r["y"].t, h=h, u=u, **g).forward()
        x2, y2 = r["x"].t.clone(), r["y"].t.clone()
        dion.NormPlan(x2, y2, h=x2, u=y2, **g).forward()
        assert torch.equal(h, x2) and torch.equal(u, y2)
        dx, dy = torch.empty_like(h), torch.empty_like(h)
        dion.NormGradPlan(h, r["y"].t, du=r["du"].t, dh=r["dh"].t, dx=dx, dy=dy, **g).backward()
        dh2, y3 = r["dh"].t.clone(), r["y"].t.clone()
        dion.NormGradPlan(h, y3, du=r["du"].t, dh=dh2, dx=dh2, dy=y3, **g).backward()
        assert torch.equal(dx, dh2) and torch.equal(dy, y3)


def test_norm_rows_are_apart():
    """A NaN or an infinity stays in its row; an all-zero row gives zeros; gains' gradients of
    the finite rows' columns only turn NaN through the bad row."""
    t, d = 9, 2048
    r, g = _norm_inputs(t, d, 0, 0, "bf16", 500)
    r["x"].t[2, 5], r["y"].t[4, 7] = float("nan"), float("inf")
    r["x"].t[6] = 0
    r["y"].t[6] = 0
    h, u = torch.empty_like(r["x"].t), torch.empty_like(r["x"].t)
    kept = dion.ActCheckpoint(t, d)
    dion.NormPlan(r["x"].t, r["y"].t, h=h, u=u, **g, checkpoint=kept).forward()
    back = kept.load(torch.empty_like(u))
    good = [0, 1, 3, 5, 6, 7, 8]
    assert torch.isfinite(u[good]).all() and torch.isfinite(back[good]).all()
    assert not torch.isfinite(u[2]).any() and torch.isnan(back[2]).all()
    assert not u[6].any() and not h[6].any() and not back[6].any()


def test_no_tokens():
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    dion.NormPlan(x, u=x).forward()
    grads = torch.full((96,), 3.0, device="cuda")
    plan = dion.NormGradPlan(x, du=x, dx=x, dpre_gain=grads)
    plan.backward(accumulate=True)
    assert bool((grads == 3.0).all())
    plan.backward()
    assert not grads.any()
    kept = dion.ActCheckpoint(0, 96)
    kept.save(x)
    kept.load(x)
    G = torch.full((96, 32), 3.0, device="cuda")
    plan = dion.WeightGradPlan([kept], [torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")], [G])
    plan.backward(accumulate=True)
    assert bool((G == 3.0).all())
    plan.backward()
    assert not G.any()
    ids, table = torch.empty(0, dtype=torch.int64, device="cuda"), torch.full((5, 96), 3.0, device="cuda")
    dion.EmbedPlan(table, ids, x).lookup()
    plan = dion.EmbedGradPlan(ids, x, table)
    plan.backward(accumulate=True)
    assert bool((table == 3.0).all())
    plan.backward()
    assert not table.any()


# ------------------------------------------------------------------ activations in 8 bits
ACT_SHAPES = [(1, 1, 0, 0), (3, 31, 0, 0), (2, 32, 0, 0), (5, 33, 0, 0), (17, 72, 0, 0),
              (40, 200, 8, 0), (9, 1000, 0, 0), (300, 1024, 0, 0), (7, 104, 0, 3), (2, 5000, 1, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,d,pad,shift", ACT_SHAPES)
def test_act_round_trip(t, d, pad, shift, dtype):
    x = Rows(t, d, DT[dtype], pad, shift)
    mag = 10.0 ** torch.randint(-12, 4, (t, d), generator=_gen(7)).float()
    x.t.copy_((mag * torch.randn(t, d, generator=_gen(8))).to(DT[dtype]).cuda())
    kept = dion.ActCheckpoint(t, d)
    kept.q.fill_(99)
    kept.save(x.t)
    ref, scale = go.act_round(_np(x.t))
    torch.cuda.synchronize()
    assert np.array_equal(kept.scale.cpu().numpy(), scale)
    assert np.array_equal(go.act_value(kept.q.cpu().numpy(), scale, d), ref)
    assert not kept.q[:, d:].any()                       # the last block's padding
    for out_t in ("bf16", "fp32", "fp16"):
        out = Rows(t, d, DT[out_t], pad, shift)
        kept.load(out.t)
        torch.cuda.synchronize()
        want = torch.from_numpy(ref).to(DT[out_t])       # exact but for fp16's range
        assert torch.equal(out.t.cpu(), want) and out.clean()
    assert x.clean()


def test_act_special_blocks():
    x = torch.zeros(4, 96, device="cuda")
    x[0, 3] = float("nan")
    x[0, 40] = float("inf")
    x[1, :32] = 3.4e38
    x[1, 32:64] = -1e-44
    x[1, 64] = 2.0 ** -126
    x[2, :3] = torch.tensor([448.0, 449.0, -463.0])
    kept = dion.ActCheckpoint(4, 96)
    kept.save(x)
    out = kept.load(torch.empty_like(x))
    ref, scale = go.act_round(_np(x))
    assert np.array_equal(kept.scale.cpu().numpy(), scale)
    assert np.array_equal(_np(out), ref, equal_nan=True)
    assert np.isnan(_np(out)[0, :64]).all() and np.isfinite(_np(out)[1]).all()


# ------------------------------------------------------------------ weight gradient
# (tokens, m, n): one token, ragged tokens, tiles' borders, odd n (copied rows), many splits
WGRAD_SHAPES = [(1, 8, 8), (1, 1, 1), (3, 40, 24), (63, 128, 64), (64, 128, 256), (65, 129, 65),
                (255, 256, 128), (256, 32, 512), (257, 96, 264), (1000, 200, 72), (700, 130, 300),
                (4099, 256, 128), (515, 1000, 777), (5000, 64, 8), (2048, 640, 1408), (300, 3, 1001), (517, 2000, 96), (700, 333, 257), (90, 770, 9665), (64, 500, 4099),
                (1024, 300, 2048), (2050, 520, 2501), (1500, 40, 5000), (4096, 520, 6500),
                (1100, 3400, 1400), (2050, 520, 1700)]


def _wgrad_inputs(t, m, n, seed, pad=0, shift=0):
    x = torch.randn(t, m, generator=_gen(seed)) * torch.exp(torch.randn(m, generator=_gen(seed + 1)))
    kept = dion.ActCheckpoint(t, m)
    kept.save(x.cuda())
    d = Rows(t, n, torch.bfloat16, pad, shift, fill=True, seed=seed + 2)
    a = go.act_value(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), m)
    return kept, d, a


def _wgrad_bound(a, d, t, transposed):
    return (2.0 ** -18 + (t / 256 + 8) * U) * go.weight_grad(np.abs(a), np.abs(d), transposed) + 1e-37


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("t,m,n", WGRAD_SHAPES)
def test_weight_grad(t, m, n, transposed):
    kept, d, a = _wgrad_inputs(t, m, n, 600)
    shape = (n, m) if transposed else (m, n)
    G = Rows(*shape, torch.float32, pad=4)
    plan = dion.WeightGradPlan([kept], [d.t], [G.t], transposed=transposed)
    plan.backward()
    torch.cuda.synchronize()
    ref = go.weight_grad(a, _np(d.t), transposed)
    bound = _wgrad_bound(a, _np(d.t), t, transposed)
    assert np.all(np.abs(_np(G.t) - ref) <= bound)
    first = G.t.clone()
    plan.backward(accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(G.t, first + first) and G.clean()
    assert not plan.status.any()


@pytest.mark.parametrize("pad,shift,gpad,gshift", [(8, 0, 0, 0), (3, 0, 1, 0), (0, 1, 0, 1), (5, 7, 3, 2)])
def test_weight_grad_strides(pad, shift, gpad, gshift):
    t, m, n = 333, 160, 200
    kept, d, a = _wgrad_inputs(t, m, n, 700, pad, shift)
    for transposed in (False, True):
        G = Rows(*((n, m) if transposed else (m, n)), torch.float32, gpad, gshift)
        dion.WeightGradPlan([kept], [d.t], [G.t], transposed=transposed).backward()
        torch.cuda.synchronize()
        assert np.all(np.abs(_np(G.t) - go.weight_grad(a, _np(d.t), transposed))
                      <= _wgrad_bound(a, _np(d.t), t, transposed))
        assert G.clean() and d.clean()


def test_weight_grad_nan_meets_its_entries_only():
    t, m, n = 130, 256, 72
    kept, d, a = _wgrad_inputs(t, m, n, 800)
    kept.scale[7, 2] = 255                                # features 64..95 of one token
    d.t[9, 11] = float("nan")
    G = torch.empty(m, n, device="cuda")
    dion.WeightGradPlan([kept], [d.t], [G]).backward()
    bad = torch.isnan(G).cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[64:96] = True
    want[:, 11] = True
    assert torch.equal(bad, want)


def test_weight_grad_reads_no_token_past_the_end():
    """The kept rows and D may be the front of larger buffers whose later rows hold NaN."""
    t, m, n = 100, 128, 128
    x = torch.randn(256, m, generator=_gen(1)).cuda()
    x[t:] = float("nan")
    whole = dion.ActCheckpoint(256, m)
    whole.save(x)
    kept = dion.ActCheckpoint(t, m, q=whole.q[:t], scale=whole.scale[:t])
    d = torch.randn(256, n, generator=_gen(2)).bfloat16().cuda()
    d[t:] = float("nan")
    G = torch.empty(m, n, device="cuda")
    dion.WeightGradPlan([kept], [d[:t]], [G]).backward()
    assert torch.isfinite(G).all()


def test_weight_grad_list_shares_a_workspace():
    shapes = [(4000, 64, 96), (1, 32, 16), (900, 256, 136), (4000, 96, 33)]
    parts = [_wgrad_inputs(*s, 900 + i) for i, s in enumerate(shapes)]
    Gs = [torch.empty(m, n, device="cuda") for _, m, n in shapes]
    plan = dion.WeightGradPlan([p[0] for p in parts], [p[1].t for p in parts], Gs)
    for _ in range(2):
        plan.backward()
    torch.cuda.synchronize()
    for (t, m, n), (_, d, a), G in zip(shapes, parts, Gs):
        assert np.all(np.abs(_np(G) - go.weight_grad(a, _np(d.t))) <= _wgrad_bound(a, _np(d.t), t, False))


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("table_t", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("out_t", ["bf16", "fp32", "fp16"])
@pytest.mark.parametrize("t,v,d,pad,shift", [(1, 1, 1, 0, 0), (5, 7, 24, 0, 0), (300, 50, 136, 8, 0), (90, 30, 36, 0, 0), (90, 30, 34, 0, 2), (200, 9, 52, 4, 4),
                                             (40, 9, 101, 0, 0), (33, 1000, 64, 3, 1)])
def test_lookup(t, v, d, pad, shift, table_t, out_t):
    table = Rows(v, d, DT[table_t], pad, shift, fill=True, seed=1)
    ids = torch.randint(-2, v + 2, (t,), generator=_gen(2))
    ids[0] = 0
    for id_t in (torch.int64, torch.int32):
        out = Rows(t, d, DT[out_t], pad, shift)
        dion.EmbedPlan(table.t, ids.to(id_t).cuda(), out.t, scale=3.7).lookup()
        torch.cuda.synchronize()
        ref = go.embed_lookup(_np(table.t), ids.numpy(), float(np.float32(3.7)))
        assert np.all(np.abs(_np(out.t) - ref) <= (HALF[out_t] + U) * np.abs(ref) + TINY[out_t])
        assert out.clean() and table.clean()


def test_lookup_takes_extreme_ids():
    table = torch.ones(4, 8, device="cuda")
    ids = torch.tensor([2 ** 62, -2 ** 62, 3, 4, -1, 2 ** 32, 0], device="cuda")
    out = torch.empty(7, 8, device="cuda")
    dion.EmbedPlan(table, ids, out).lookup()
    assert out[:, 0].tolist() == [0, 0, 1, 0, 0, 0, 1]
    g = torch.empty(4, 8, device="cuda")
    dion.EmbedGradPlan(ids, torch.ones(7, 8, device="cuda"), g).backward()
    assert g[:, 0].tolist() == [1, 0, 0, 1]


def _ids(kind, t, v, seed):
    if kind == "uniform":
        return torch.randint(-1, v + 1, (t,), generator=_gen(seed))
    if kind == "one":
        return torch.full((t,), v - 1)
    if kind == "none":
        return torch.full((t,), -1)
    if kind == "few":                                   # long runs of uneven lengths
        return (torch.rand(t, generator=_gen(seed)) ** 4 * min(v, 5)).long()
    return torch.arange(t) % v


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["uniform", "one", "none", "few", "cycle"])
@pytest.mark.parametrize("t,v,d,pad", [(1, 1, 8, 0), (31, 5, 24, 0), (33, 300, 40, 8), (64, 2, 7, 0),
                                       (1000, 70000, 16, 0), (5000, 257, 130, 2), (9001, 40, 2064, 0),
                                       (16384, 255, 520, 0), (16385, 3000, 24, 0), (500, 300000, 8, 0),
                                       (130, 262143, 8, 0), (70, 1030, 1032, 0), (32768, 131071, 8, 0),
                                       (32769, 90, 16, 0), (4097, 65535, 8, 0)])
def test_embed_grad(t, v, d, pad, kind, dtype):
    ids = _ids(kind, t, v, 3)
    dout = Rows(t, d, DT[dtype], pad, 0, fill=True, seed=4)
    g = Rows(v, d, torch.float32, pad)
    ref = go.embed_grad(ids.numpy(), _np(dout.t), v, 1.25)
    hits = np.bincount(np.clip(ids.numpy(), -1, v) + 1, minlength=v + 2)[1:v + 1]
    mag = go.embed_grad(ids.numpy(), np.abs(_np(dout.t)), v, 1.25)
    bound = (hits[:, None] + 2) * U * mag
    for id_t in (torch.int64, torch.int32):
        plan = dion.EmbedGradPlan(ids.to(id_t).cuda(), dout.t, g.t, scale=1.25)
        plan.backward()
        torch.cuda.synchronize()
        got = _np(g.t)
        assert np.all(np.abs(got - ref) <= bound) and not got[hits == 0].any()
        assert g.clean() and dout.clean()
    first = g.t.clone()
    plan.backward()
    assert torch.equal(first, g.t)                      # bit for bit again
    g.t[:] = 1.0
    plan.backward(accumulate=True)
    torch.cuda.synchronize()
    assert np.all(np.abs(_np(g.t) - 1 - ref) <= bound + U * (1 + mag))
    assert bool((g.t[torch.from_numpy(hits == 0).cuda()] == 1.0).all())


def test_embed_grad_does_not_read_padded_rows():
    ids = torch.tensor([2, -1, 0, 7, 2], device="cuda")
    dout = torch.ones(5, 16, device="cuda")
    dout[1] = float("nan")
    dout[3] = float("inf")
    g = torch.empty(7, 16, device="cuda")
    dion.EmbedGradPlan(ids, dout, g).backward()
    assert g[:, 3].tolist() == [1, 0, 2, 0, 0, 0, 0]


# ------------------------------------------------------------------ together, and how they are called
def _chain(seed=0):
    """One layer of a model: lookup, norm (kept in 8 bits), projection, norm after it into the
    residual, loss <w, u>.  Returns everything a step needs, from the package's calls."""
    t, v, d, n = 300, 64, 128, 128
    g = _gen(seed)
    mk = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    table, W = 0.5 * mk(v, d), 0.1 * mk(d, n)
    ids = torch.randint(-1, v, (t,), generator=g).cuda()
    gains = {k: 1 + 0.1 * mk(d) for k in ("pre", "post", "gate", "final")}
    up = 0.1 * mk(t, d)                                   # gradient of the final u
    return t, v, d, n, table, W, ids, gains, up


def test_chain_gives_the_gradients_of_its_parameters():
    """The run of operators as a training step uses them, in fp32 rows, against central
    differences of an fp64 model with the kept activations in the weight's gradient."""
    t, v, d, n, table, W, ids, gn, up = _chain()
    new = lambda: torch.empty(t, d, device="cuda")  # noqa: E731
    x, u, h, uf = new(), new(), new(), new()
    kept = dion.ActCheckpoint(t, d)
    dion.EmbedPlan(table, ids, x, scale=d ** 0.5).lookup()
    dion.NormPlan(x, u=u, pre_gain=gn["pre"], checkpoint=kept).forward()
    y = (u @ W).contiguous()
    dion.NormPlan(x, y, h=h, u=uf, pre_gain=gn["final"], post_gain=gn["post"], gate=gn["gate"],
                  residual_scale=0.5).forward()
    # backward
    dxr, dy = new(), new()
    gg = {k: torch.empty(d, device="cuda") for k in gn}
    dion.NormGradPlan(h, y, du=up, dx=dxr, dy=dy, pre_gain=gn["final"], post_gain=gn["post"],
                      gate=gn["gate"], dpre_gain=gg["final"], dpost_gain=gg["post"],
                      dgate=gg["gate"], residual_scale=0.5).backward()
    dyb = dy.bfloat16()
    G = torch.empty(d, n, device="cuda")
    dion.WeightGradPlan([kept], [dyb], [G]).backward()
    du = dy @ W.t()
    dx = new()
    dion.NormGradPlan(x, du=du, dh=dxr, dx=dx, pre_gain=gn["pre"], dpre_gain=gg["pre"]).backward()
    dtable = torch.empty_like(table)
    dion.EmbedGradPlan(ids, dx, dtable, scale=d ** 0.5).backward()
    torch.cuda.synchronize()

    par = {"table": _np(table), "W": _np(W), **{k: _np(a) for k, a in gn.items()}}
    idn, upn = ids.cpu().numpy(), _np(up)

    def loss(p):
        x0 = go.embed_lookup(p["table"], idn, d ** 0.5)
        _, u0 = go.norm_forward(x0, pre_gain=p["pre"])
        _, u1 = go.norm_forward(x0, u0 @ p["W"], pre_gain=p["final"], post_gain=p["post"],
                                gate=p["gate"], residual_scale=0.5)
        return np.sum(u1 * upn)

    rng = np.random.default_rng(1)
    got = {"table": dtable, "W": G, **gg}
    for name, grad in got.items():
        # the directional derivative along a random direction, by central differences.  The
        # kept activations are rounded by up to 2^-4 each, dY by 2^-8: W's derivative is off
        # by 2^-4 times the root sum of squares of its terms at most by chance, 3 of those here
        way = rng.standard_normal(par[name].shape)
        hi = loss({**par, name: par[name] + 1e-5 * way})
        lo = loss({**par, name: par[name] - 1e-5 * way})
        num, ours = (hi - lo) / 2e-5, float(np.sum(_np(grad) * way))
        norm = np.linalg.norm(_np(grad)) * (3 * 2.0 ** -4 if name == "W" else 1e-4)
        assert abs(num - ours) <= norm + 1e-6, (name, num, ours)


def test_step_from_saved_is_the_step_on_those_gradients():
    """dion_step_batched_from_saved against weight_grad followed by the step: bit for bit, in
    both layouts and accumulating; and the vector step takes the gains' gradients."""
    t, m, n, count = 500, 96, 64, 2
    opt = dion.DionB200([(count, m, n, 16)])
    for transposed in (False, True):
        feats, outs = (n, m) if transposed else (m, n)
        parts = [_wgrad_inputs(t, feats, outs, 50 + i) for i in range(count)]
        kept, dys = [p[0] for p in parts], [p[1].t for p in parts]
        X, M = torch.randn(count, m, n, generator=_gen(3)).cuda(), torch.randn(count, m, n, generator=_gen(4)).cuda()
        Q = torch.nn.functional.normalize(torch.randn(count, n, 16, generator=_gen(5)), dim=1).cuda()
        G = torch.full((count, m, n), 0.5, device="cuda")
        state = [v.clone() for v in (X, M, G, Q)]
        saved = dion.SavedStep(opt, kept, dys, transposed=transposed)
        saved.step([X], [M], [G], [Q], 0.01, status=opt.alloc_status(), accumulate=True)
        X2, M2, G2, Q2 = state
        dion.WeightGradPlan(kept, dys, [G2[i] for i in range(count)],
                            transposed=transposed).backward(accumulate=True)
        opt.step([X2], [M2], [G2], [Q2], 0.01, opt.alloc_workspace())
        torch.cuda.synchronize()
        for a, b in ((X, X2), (M, M2), (G, G2), (Q, Q2)):
            assert torch.equal(a, b)
        assert not saved.grad_status.any()
    opt.close()


def test_captured_and_replayed():
    """Every call captured into a graph and replayed on changed inputs gives what the eager
    call gives (workspaces need no clearing between calls)."""
    t, v, d, n = 700, 500, 256, 64
    x = torch.randn(t, d, device="cuda").bfloat16()
    y, du, dh = (torch.randn_like(x) for _ in range(3))
    ids = torch.randint(-1, v, (t,), device="cuda")
    pg = torch.randn(d, device="cuda")
    h, u, dx, dyy = (torch.empty_like(x) for _ in range(4))
    dpre, dtable, G = torch.empty(d, device="cuda"), torch.empty(v, d, device="cuda"), torch.empty(d, n, device="cuda")
    dn = torch.randn(t, n, device="cuda").bfloat16()
    kept = dion.ActCheckpoint(t, d)
    table = torch.randn(v, d, device="cuda")
    out = torch.empty_like(x)
    plans = [dion.NormPlan(x, y, h=h, u=u, pre_gain=pg, post_gain=pg, checkpoint=kept).forward,
             dion.NormGradPlan(h, y, du=du, dh=dh, dx=dx, dy=dyy, pre_gain=pg, post_gain=pg,
                               dpre_gain=dpre).backward,
             dion.WeightGradPlan([kept], [dn], [G]).backward,
             dion.EmbedPlan(table, ids, out).lookup,
             dion.EmbedGradPlan(ids, dx, dtable).backward]
    outs = [h, u, dx, dyy, dpre, G, out, dtable]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                       # warm up and capture on another stream
        for p in plans:
            p()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in plans:
            p()
    for seed in (1, 2):
        for b in (x, y, du, dh, dn, table):
            b.copy_(torch.randn(b.shape, generator=_gen(seed)).to(b.dtype).cuda())
        ids.copy_(torch.randint(-1, v, (t,), generator=_gen(seed)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        for o in outs:
            o.fill_(9)
        for p in plans:
            p()
        torch.cuda.synchronize()
        for a, b in zip(replayed, outs):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces():
    t, m, n = 4000, 128, 128
    a, b = _wgrad_inputs(t, m, n, 10), _wgrad_inputs(t, m, n, 20)
    Ga, Gb = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    pa = dion.WeightGradPlan([a[0]], [a[1].t], [Ga])
    pb = dion.WeightGradPlan([b[0]], [b[1].t], [Gb])
    pa.backward()
    pb.backward()
    torch.cuda.synchronize()
    want = Ga.clone(), Gb.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        pa.backward(stream=s1)
        pb.backward(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(Ga, want[0]) and torch.equal(Gb, want[1])


def test_offsets_past_32_bits():
    """40 rows 2^26 elements apart (5.4 GB of bf16): the last rows lie past 2^31 elements."""
    t, d, ld = 40, 64, 1 << 26
    far = torch.empty(t * ld, dtype=torch.bfloat16, device="cuda").view(t, ld)
    x = far[:, :d]
    vals = torch.randn(t, d, generator=_gen(1)).bfloat16()
    x.copy_(vals.cuda())
    kept, near = dion.ActCheckpoint(t, d), dion.ActCheckpoint(t, d)
    kept.save(x)
    near.save(vals.cuda())
    assert torch.equal(kept.q, near.q) and torch.equal(kept.scale, near.scale)
    # the norm, rows to rows of the same buffer; and backwards into it
    u, want = far[:, d:2 * d], torch.empty(t, d, dtype=torch.bfloat16, device="cuda")
    dion.NormPlan(x, u=u).forward()
    dion.NormPlan(vals.cuda(), u=want).forward()
    assert torch.equal(u, want)
    dx = far[:, 2 * d:3 * d]
    dion.NormGradPlan(x, du=u, dx=dx).backward()
    dw = torch.empty_like(want)
    dion.NormGradPlan(vals.cuda(), du=want, dx=dw).backward()
    assert torch.equal(dx, dw)
    # the far rows as a table, as dY, as the gradient of looked-up rows
    ids = torch.tensor([t - 1, 0, -1, t - 2, t - 1], device="cuda")
    out = far[:5, 3 * d:4 * d]
    dion.EmbedPlan(x, ids, out).lookup()
    assert torch.equal(out[0], x[t - 1]) and torch.equal(out[3], x[t - 2]) and not out[2].any()
    g, gw = torch.empty(t, d, device="cuda"), torch.empty(t, d, device="cuda")
    dion.EmbedGradPlan(torch.arange(t, device="cuda"), x, g).backward()
    assert torch.equal(g, x.float())
    G, Gw = torch.empty(d, d, device="cuda"), torch.empty(d, d, device="cuda")
    dion.WeightGradPlan([kept], [x], [G]).backward()
    dion.WeightGradPlan([kept], [vals.cuda()], [Gw]).backward()
    assert torch.equal(G, Gw)
    del far, x, u, dx, out
    # a table and G of far rows in fp32 (10.7 GB)
    far = torch.full((t * ld,), 7.0, device="cuda").view(t, ld)
    dion.EmbedGradPlan(torch.arange(t - 1, -1, -1, device="cuda"), vals.cuda(), far[:, :d]).backward()
    assert torch.equal(far[:, :d], vals.cuda().float().flip(0)) and bool((far[:, d] == 7.0).all())
    dion.WeightGradPlan([kept], [vals.cuda()[:, :t].contiguous()], [far[:, :d]], transposed=True).backward()
    ref = torch.empty(t, d, device="cuda")
    dion.WeightGradPlan([kept], [vals.cuda()[:, :t].contiguous()], [ref], transposed=True).backward()
    assert torch.equal(far[:, :d], ref)


def test_a_plan_of_another_device_is_refused(monkeypatch):
    x = torch.zeros(4, 64, device="cuda")
    plan, kept = dion.NormPlan(x, u=torch.empty_like(x)), dion.ActCheckpoint(4, 64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: x.device.index + 1)
    with pytest.raises(ValueError, match="current device"):
        plan.forward()
    with pytest.raises(ValueError, match="current device"):
        kept.save(x)


def test_two_lists_of_ids_in_turn_with_one_workspace():
    """Calls that follow each other on a stream may share a workspace: what one leaves there
    (sorted ids, the list of runs to join) does not reach the next."""
    v, d = 50, 264
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)
    for seed, t in ((1, 2000), (2, 3), (3, 700), (4, 2000)):
        ids = _ids("few", t, v, seed)
        dout = torch.randn(t, d, generator=_gen(seed)).cuda()
        g = torch.empty(v, d, device="cuda")
        dion.EmbedGradPlan(ids.cuda(), dout, g, workspace=ws).backward()
        mag = go.embed_grad(ids.numpy(), np.abs(_np(dout)), v)
        hits = np.bincount(ids.numpy(), minlength=v)
        assert np.all(np.abs(_np(g) - go.embed_grad(ids.numpy(), _np(dout), v)) <= (hits[:, None] + 2) * U * mag)


def test_every_operator_on_two_streams_at_once():
    """Two sets of plans, each with its own buffers, on two streams in turn: both give what they
    give alone."""
    def plans(seed):
        t, v, d, n = 3000, 700, 1032, 1600
        r = lambda *s: torch.randn(*s, generator=_gen(seed)).cuda()  # noqa: E731
        x, y, du = r(t, d).bfloat16(), r(t, d).bfloat16(), r(t, d).bfloat16()
        ids = torch.randint(-1, v, (t,), generator=_gen(seed)).cuda()
        dn, table = r(t, n).bfloat16(), r(v, d)
        h, u, dx, dy, out = (torch.empty_like(x) for _ in range(5))
        dw, dtable, G = torch.empty(d, device="cuda"), torch.empty(v, d, device="cuda"), torch.empty(d, n, device="cuda")
        kept = dion.ActCheckpoint(t, d)
        calls = [dion.NormPlan(x, y, h=h, u=u, post_norm=True, checkpoint=kept).forward,
                 dion.NormGradPlan(x, y, du=du, dx=dx, dy=dy, post_norm=True, dpre_gain=dw).backward,
                 dion.WeightGradPlan([kept], [dn], [G]).backward,
                 dion.EmbedPlan(table, ids, out).lookup,
                 dion.EmbedGradPlan(ids, du, dtable).backward]
        return calls, [h, u, dx, dy, dw, G, out, dtable]

    sets = [plans(1), plans(2)]
    for calls, _ in sets:
        for c in calls:
            c()
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for k in range(5):
            for (calls, _), s in zip(sets, streams):
                calls[k](stream=s)
    torch.cuda.synchronize()
    for (_, outs), w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_plans_refuse_tensors_that_do_not_fit():
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="must be"):
        dion.NormPlan(x, u=torch.zeros(4, 63, device="cuda"))
    with pytest.raises(ValueError, match="torch.float32"):
        dion.NormPlan(x, u=x.bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        dion.NormPlan(torch.zeros(64, 4, device="cuda").t(), u=x)
    with pytest.raises(ValueError, match="overlap"):
        dion.NormPlan(torch.zeros(1, 64, device="cuda").expand(4, 64), u=x)
    with pytest.raises(ValueError, match="vector"):
        dion.NormPlan(x, u=x, pre_gain=torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError, match="bytes"):
        dion.NormGradPlan(x, du=x, dx=x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="int32 or int64"):
        dion.EmbedPlan(x, torch.zeros(3, device="cuda"), x[:3])
    with pytest.raises(ValueError, match="must be"):
        dion.EmbedPlan(x, torch.zeros(3, dtype=torch.int64, device="cuda"), x)
    k = dion.ActCheckpoint(4, 64)
    with pytest.raises(ValueError, match="bfloat16"):
        dion.WeightGradPlan([k], [x], [torch.zeros(64, 64, device="cuda")])
    with pytest.raises(ValueError, match="must be"):
        dion.WeightGradPlan([k], [x.bfloat16()], [torch.zeros(64, 63, device="cuda")])
    with pytest.raises(ValueError, match="must be"):
        k.save(torch.zeros(5, 64, device="cuda"))
    with pytest.raises(dion.DionError):
        dion.NormPlan(x, u=x, eps=0.0).forward()
