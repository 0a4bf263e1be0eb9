"""Host-side checks of the gradient operators (dion_act_*, dion_weight_grad, dion_norm_*,
dion_embed_*): refusals come back with the documented codes before any device work, and the
Python plans refuse what the C ABI could not take (no GPU)."""
import ctypes

import pytest

import rank_orthonormalized_optimizer_b200 as dion
from rank_orthonormalized_optimizer_b200 import gradients as gr

FAKE = 1 << 20          # an aligned address that is never dereferenced
REACHED = (dion.OK, dion.ERR_CUDA, dion.ERR_DEVICE)   # past every check of the arguments


def _no_gpu():
    import torch
    return not torch.cuda.is_available()


pytestmark = pytest.mark.skipif(not _no_gpu(), reason="valid calls would launch on fake pointers")


def _kept(q=FAKE, scale=FAKE, tokens=8, features=64):
    return gr.ActKept(q, scale, tokens, features)


@pytest.mark.parametrize("kept,x,ld,dtype,code", [
    (dict(), FAKE, 64, 0, None),
    (dict(tokens=0), None, 64, 0, None),
    (dict(), FAKE, 64, 3, dion.ERR_INVALID_ARG),
    (dict(), None, 64, 0, dion.ERR_INVALID_ARG),
    (dict(), FAKE, 63, 0, dion.ERR_INVALID_ARG),
    (dict(), FAKE + 1, 64, 0, dion.ERR_MISALIGNED),
    (dict(), FAKE + 2, 64, 2, dion.ERR_MISALIGNED),
    (dict(), FAKE + 2, 64, 1, None),
    (dict(tokens=-1), FAKE, 64, 0, dion.ERR_INVALID_ARG),
    (dict(tokens=1 << 31), FAKE, 64, 0, dion.ERR_INVALID_ARG),
    (dict(features=0), FAKE, 64, 0, dion.ERR_INVALID_ARG),
    (dict(q=None), FAKE, 64, 0, dion.ERR_INVALID_ARG),
    (dict(scale=None), FAKE, 64, 0, dion.ERR_INVALID_ARG),
    (dict(q=FAKE + 8), FAKE, 64, 0, dion.ERR_MISALIGNED),
])
def test_act_refusals(kept, x, ld, dtype, code):
    k = _kept(**kept)
    for got in (gr.dion_act_save(x, ld, dtype, ctypes.byref(k), None),
                gr.dion_act_load(ctypes.byref(k), x, ld, dtype, None)):
        assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()
    assert gr.dion_act_save(x, ld, dtype, None, None) == dion.ERR_INVALID_ARG


def _norm(**kw):
    a = gr.Norm(tokens=4, features=64, dtype=0, post_norm=1, eps=1e-6, residual_scale=1.0, x=FAKE,
                ldx=64, y=FAKE, ldy=64, h=FAKE, ldh=64, u=FAKE, ldu=64, pre_gain=FAKE,
                post_gain=FAKE, gate=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(), None),
    (dict(tokens=0, x=None, y=FAKE), None),
    (dict(y=None, h=None, post_norm=0, post_gain=None, gate=None), None),
    (dict(u=None, pre_gain=None), None),
    (dict(h=None), None),
    (dict(dtype=-1), dion.ERR_INVALID_ARG),
    (dict(tokens=-1), dion.ERR_INVALID_ARG),
    (dict(features=0), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(features=16385, ldx=16385, ldy=16385, ldh=16385, ldu=16385), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(eps=0.0), dion.ERR_INVALID_ARG),
    (dict(eps=float("nan")), dion.ERR_INVALID_ARG),
    (dict(residual_scale=float("inf")), dion.ERR_INVALID_ARG),
    (dict(x=None), dion.ERR_INVALID_ARG),
    (dict(ldx=63), dion.ERR_INVALID_ARG),
    (dict(ldu=63), dion.ERR_INVALID_ARG),
    (dict(y=FAKE + 1), dion.ERR_MISALIGNED),
    (dict(gate=FAKE + 2), dion.ERR_MISALIGNED),
    (dict(y=None), dion.ERR_INVALID_ARG),                      # h without y
    (dict(y=None, h=None, post_norm=0, post_gain=None), dion.ERR_INVALID_ARG),   # gate without y
    (dict(post_norm=0), dion.ERR_INVALID_ARG),                 # a gain of no norm
    (dict(u=None), dion.ERR_INVALID_ARG),                      # pre_gain without u
    (dict(u=None, h=None, pre_gain=None), dion.ERR_INVALID_ARG),
])
def test_norm_refusals(kw, code):
    got = gr.dion_norm_forward(ctypes.byref(_norm(**kw)), None)
    assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()


def test_norm_kept_must_match():
    for k, code in ((_kept(tokens=4), None), (_kept(tokens=5), dion.ERR_INVALID_ARG),
                    (_kept(tokens=4, features=32), dion.ERR_INVALID_ARG),
                    (_kept(tokens=4, q=FAKE + 4), dion.ERR_MISALIGNED)):
        a = _norm(kept=ctypes.pointer(k))
        got = gr.dion_norm_forward(ctypes.byref(a), None)
        assert (got in REACHED) if code is None else (got == code)
    a = _norm(u=None, pre_gain=None, kept=ctypes.pointer(_kept(tokens=4)))
    assert gr.dion_norm_forward(ctypes.byref(a), None) == dion.ERR_INVALID_ARG
    assert gr.dion_norm_forward(None, None) == dion.ERR_INVALID_ARG


def _norm_grad(**kw):
    a = gr.NormGrad(tokens=4, features=64, dtype=0, post_norm=1, eps=1e-6, residual_scale=1.0)
    for k in ("h", "y", "du", "dh", "dx", "dy"):
        setattr(a, k, FAKE)
        setattr(a, "ld" + k, 64)
    for k in ("pre_gain", "post_gain", "gate", "dpre_gain", "dpost_gain", "dgate"):
        setattr(a, k, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


WS = 1 << 30


@pytest.mark.parametrize("kw,ws,bytes_,code", [
    (dict(), FAKE, WS, None),
    (dict(dh=None), FAKE, WS, None),
    (dict(du=None, pre_gain=None, dpre_gain=None, h=None), FAKE, WS, None),
    (dict(dx=None, dy=None), FAKE, WS, None),
    (dict(), None, WS, dion.ERR_INVALID_ARG),
    (dict(), FAKE, 16, dion.ERR_WORKSPACE_TOO_SMALL),
    (dict(), FAKE + 4, WS, dion.ERR_MISALIGNED),
    (dict(du=None, dh=None, pre_gain=None, dpre_gain=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(du=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(h=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(y=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(post_norm=0), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(dx=None, dy=None, dpre_gain=None, dpost_gain=None, dgate=None), FAKE, WS,
     dion.ERR_INVALID_ARG),
    (dict(lddx=10), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(dgate=FAKE + 1), FAKE, WS, dion.ERR_MISALIGNED),
    (dict(eps=-1.0), FAKE, WS, dion.ERR_INVALID_ARG),
])
def test_norm_backward_refusals(kw, ws, bytes_, code):
    got = gr.dion_norm_backward(ctypes.byref(_norm_grad(**kw)), ws, bytes_, None)
    assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()


def _source(**kw):
    s = gr.GradSource(kept=_kept(), d=FAKE, ldd=32, n=32, G=FAKE, ldg=32, transposed=0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(), None),
    (dict(transposed=1, ldg=64), None),
    (dict(d=FAKE + 2), dion.ERR_INVALID_ARG),                   # copied into the workspace: NULL
    (dict(n=0), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(n=(1 << 24) + 1, ldd=1 << 25, ldg=1 << 25), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(kept=_kept(features=(1 << 24) + 1)), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(kept=_kept(q=None)), dion.ERR_INVALID_ARG),
    (dict(kept=_kept(tokens=-4)), dion.ERR_INVALID_ARG),
    (dict(d=None), dion.ERR_INVALID_ARG),
    (dict(G=None), dion.ERR_INVALID_ARG),
    (dict(ldd=31), dion.ERR_INVALID_ARG),
    (dict(ldg=31), dion.ERR_INVALID_ARG),
    (dict(transposed=1), dion.ERR_INVALID_ARG),                 # rows of 64 need ldg >= 64
    (dict(d=FAKE + 1), dion.ERR_MISALIGNED),
    (dict(G=FAKE + 2), dion.ERR_MISALIGNED),
    (dict(kept=_kept(tokens=0, q=None, scale=None), d=None), None),
])
def test_weight_grad_refusals(kw, code):
    s = _source(**kw)
    got = gr.dion_weight_grad(ctypes.byref(s), 1, 0, None, 0, None, None)
    assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()


def test_weight_grad_list_refusals():
    two = (gr.GradSource * 2)(_source(), _source(G=None))
    assert gr.dion_weight_grad(two, 2, 0, None, 0, None, None) == dion.ERR_INVALID_ARG
    assert gr.dion_weight_grad(two, -1, 0, None, 0, None, None) == dion.ERR_INVALID_ARG
    assert gr.dion_weight_grad(None, 1, 0, None, 0, None, None) == dion.ERR_INVALID_ARG
    assert gr.dion_weight_grad(two, 1, 0, None, 0, FAKE + 2, None) == dion.ERR_MISALIGNED
    huge = (gr.GradSource * 1)(_source(n=(1 << 24) + 1))
    assert gr.dion_weight_grad_workspace(huge, 1) == 0
    # the size goes by the shapes: G need not be there yet
    no_g = _source(kept=_kept(tokens=1 << 14), G=None)
    assert gr.dion_weight_grad_workspace(ctypes.byref(no_g), 1) > 0
    # few tiles over many tokens: the split over the tokens needs a workspace
    long = _source(kept=_kept(tokens=1 << 14))
    need = gr.dion_weight_grad_workspace(ctypes.byref(long), 1)
    assert need > 0
    assert gr.dion_weight_grad(ctypes.byref(long), 1, 0, None, need, None, None) == dion.ERR_INVALID_ARG
    assert gr.dion_weight_grad(ctypes.byref(long), 1, 0, FAKE, need - 1, None,
                               None) == dion.ERR_WORKSPACE_TOO_SMALL
    assert gr.dion_weight_grad(ctypes.byref(long), 1, 0, FAKE, need, None, None) in REACHED


def test_step_from_saved_refusals():
    opt = dion.DionB200([(2, 64, 32, 16)])
    ptrs = (dion.BucketPtrs * 1)(dion.BucketPtrs(FAKE, FAKE, FAKE, FAKE))
    good = (gr.GradSource * 2)(_source(), _source())
    ws = gr.dion_step_from_saved_workspace(opt._h, good, 2)
    assert ws >= opt.workspace_bytes

    def call(sources, nb=1, lr=0.1, wsb=ws, status=None):
        return gr.dion_step_batched_from_saved(opt._h, ptrs, sources, nb, 0, lr, FAKE, wsb, status,
                                               None, None)

    assert call(good) in REACHED
    assert call(None) == dion.ERR_INVALID_ARG
    assert call(good, nb=2) == dion.ERR_INVALID_ARG
    assert call(good, lr=float("nan")) == dion.ERR_INVALID_ARG
    assert call(good, wsb=16) == dion.ERR_WORKSPACE_TOO_SMALL
    assert call((gr.GradSource * 2)(_source(), _source(n=40, ldd=40))) == dion.ERR_INVALID_ARG
    assert call((gr.GradSource * 2)(_source(), _source(transposed=1))) == dion.ERR_INVALID_ARG
    opt.close()
    assert call(good) == dion.ERR_NOT_INITIALIZED


def _embed(**kw):
    a = gr.Embed(tokens=4, vocab=10, features=16, ids=FAKE, id_bytes=8, table_dtype=2, out_dtype=0,
                 scale=1.0, table=FAKE, ldt=16, out=FAKE, ldo=16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(), None), (dict(tokens=0, ids=None, out=None), None),
    (dict(tokens=-1), dion.ERR_INVALID_ARG), (dict(vocab=0), dion.ERR_INVALID_ARG),
    (dict(vocab=(1 << 31) - 1), dion.ERR_INVALID_ARG),
    (dict(features=0), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(features=(1 << 24) + 1), dion.ERR_UNSUPPORTED_SHAPE),
    (dict(id_bytes=2), dion.ERR_INVALID_ARG), (dict(ids=None), dion.ERR_INVALID_ARG),
    (dict(ids=FAKE + 4), dion.ERR_MISALIGNED), (dict(ids=FAKE + 4, id_bytes=4), None),
    (dict(scale=float("nan")), dion.ERR_INVALID_ARG),
    (dict(table_dtype=5), dion.ERR_INVALID_ARG), (dict(out_dtype=-1), dion.ERR_INVALID_ARG),
    (dict(table=None), dion.ERR_INVALID_ARG), (dict(ldt=15), dion.ERR_INVALID_ARG),
    (dict(out=FAKE + 1), dion.ERR_MISALIGNED),
])
def test_embed_refusals(kw, code):
    got = gr.dion_embed_lookup(ctypes.byref(_embed(**kw)), None)
    assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()


@pytest.mark.parametrize("kw,ws,bytes_,code", [
    (dict(), FAKE, WS, None),
    (dict(tokens=0, ids=None, dout=None), None, 0, None),
    (dict(), None, WS, dion.ERR_INVALID_ARG),
    (dict(), FAKE, 8, dion.ERR_WORKSPACE_TOO_SMALL),
    (dict(), FAKE + 8, WS, dion.ERR_MISALIGNED),
    (dict(dtype=9), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(dout=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(dtable=None), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(ldo=3), FAKE, WS, dion.ERR_INVALID_ARG),
    (dict(dtable=FAKE + 2), FAKE, WS, dion.ERR_MISALIGNED),
    (dict(scale=float("inf")), FAKE, WS, dion.ERR_INVALID_ARG),
])
def test_embed_backward_refusals(kw, ws, bytes_, code):
    a = gr.EmbedGrad(tokens=4, vocab=10, features=16, ids=FAKE, id_bytes=4, dtype=0, scale=1.0,
                     dout=FAKE, ldo=16, dtable=FAKE, ldt=16)
    for k, v in kw.items():
        setattr(a, k, v)
    got = gr.dion_embed_backward(ctypes.byref(a), ws, bytes_, None)
    assert (got in REACHED) if code is None else (got == code), dion.dion_last_error()


def test_plans_check_their_tensors_on_the_host():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dion.NormPlan(x, u=x)
    with pytest.raises(ValueError, match="CUDA"):
        dion.NormGradPlan(x, du=x, dx=x)
    with pytest.raises(ValueError, match="CUDA"):
        dion.EmbedPlan(x, torch.zeros(3, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="CUDA"):
        dion.EmbedGradPlan(torch.zeros(3, dtype=torch.int64), x, x)
    with pytest.raises(ValueError, match="ActCheckpoint"):
        dion.WeightGradPlan([x], [x], [x])
    with pytest.raises(ValueError, match="one entry"):
        dion.WeightGradPlan([x], [], [])
    with pytest.raises(ValueError):
        dion.ActCheckpoint(-1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        dion.ActCheckpoint(4, 8, device="cpu")
    with pytest.raises(ValueError, match="bf16"):
        dion.NormPlan(x.double(), u=x)
    for bad in (torch.zeros(8), None):
        with pytest.raises(ValueError):
            dion.NormPlan(bad)


def test_c99_caller(tmp_path):
    import os
    import shutil
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    exe, libdir = tmp_path / "abi_gradients", os.path.dirname(dion.LIB_PATH)
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I",
                    os.path.join(root, "include"), os.path.join(root, "tests", "c", "abi_gradients.c"),
                    "-L", libdir, "-ldion_b200", f"-Wl,-rpath,{libdir}", "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def test_gradient_workloads_are_seeded():
    import torch
    import workloads as W
    gw = W.GRADIENT_WORKLOADS["layer_h256_ff128_t300"]
    a, b, c = W.gradient_inputs(gw), W.gradient_inputs(gw), W.gradient_inputs(gw, step=1)
    assert all(torch.equal(a[k], b[k]) for k in a) and not torch.equal(a["y"], c["y"])
    assert a["ids"].min() == -1 and a["ids"].max() < gw.vocab and a["d_mlp"].shape == (300, 128)
