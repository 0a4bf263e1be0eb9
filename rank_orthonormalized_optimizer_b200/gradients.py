"""Where the step's gradients come from: the fused norm, activations kept in 8 bits and the
weight gradient from them, the embedding lookup and its gradient (include/dion.h).

Each class marshals a fixed set of tensors once, as VecStepPlan does; a call then costs one
C call and its launches.  The tensors must stay allocated while the plan is used, lie on one
device, which must be the current one when the plan is called, and hold their rows with the
features contiguous (row strides are free).  Gradients of weights, gains and tables are
fp32: the buffers that DionB200.step and VecStepPlan.step read.  ``workspace`` (uint8) is
allocated by the plan unless it is given; two calls in flight must not share one.
"""
from __future__ import annotations

import ctypes

from . import (BucketPtrs, _check, _sig, c_float, c_int32, c_int64, c_size_t,
               c_void_p)

ACT_BLOCK = 32                       # DION_ACT_BLOCK of include/dion.h
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2


class ActKept(ctypes.Structure):
    _fields_ = [("q", c_void_p), ("scale", c_void_p), ("tokens", c_int64), ("features", c_int64)]


class GradSource(ctypes.Structure):
    _fields_ = [("kept", ActKept), ("d", c_void_p), ("ldd", c_int64), ("n", c_int64),
                ("G", c_void_p), ("ldg", c_int64), ("transposed", c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("tokens", c_int64), ("features", c_int64), ("dtype", c_int32),
                ("post_norm", c_int32), ("eps", c_float), ("residual_scale", c_float),
                ("x", c_void_p), ("ldx", c_int64), ("y", c_void_p), ("ldy", c_int64),
                ("h", c_void_p), ("ldh", c_int64), ("u", c_void_p), ("ldu", c_int64),
                ("pre_gain", c_void_p), ("post_gain", c_void_p), ("gate", c_void_p),
                ("kept", ctypes.POINTER(ActKept))]


class NormGrad(ctypes.Structure):
    _fields_ = [("tokens", c_int64), ("features", c_int64), ("dtype", c_int32),
                ("post_norm", c_int32), ("eps", c_float), ("residual_scale", c_float),
                ("h", c_void_p), ("ldh", c_int64), ("y", c_void_p), ("ldy", c_int64),
                ("du", c_void_p), ("lddu", c_int64), ("dh", c_void_p), ("lddh", c_int64),
                ("dx", c_void_p), ("lddx", c_int64), ("dy", c_void_p), ("lddy", c_int64),
                ("pre_gain", c_void_p), ("post_gain", c_void_p), ("gate", c_void_p),
                ("dpre_gain", c_void_p), ("dpost_gain", c_void_p), ("dgate", c_void_p),
                ("accumulate", c_int32)]


class Embed(ctypes.Structure):
    _fields_ = [("tokens", c_int64), ("vocab", c_int64), ("features", c_int64), ("ids", c_void_p),
                ("id_bytes", c_int32), ("table_dtype", c_int32), ("out_dtype", c_int32),
                ("scale", c_float), ("table", c_void_p), ("ldt", c_int64), ("out", c_void_p),
                ("ldo", c_int64)]


class EmbedGrad(ctypes.Structure):
    _fields_ = [("tokens", c_int64), ("vocab", c_int64), ("features", c_int64), ("ids", c_void_p),
                ("id_bytes", c_int32), ("dtype", c_int32), ("scale", c_float), ("dout", c_void_p),
                ("ldo", c_int64), ("dtable", c_void_p), ("ldt", c_int64), ("accumulate", c_int32)]


_P = ctypes.POINTER
dion_act_save = _sig("dion_act_save", c_int32, c_void_p, c_int64, c_int32, _P(ActKept), c_void_p)
dion_act_load = _sig("dion_act_load", c_int32, _P(ActKept), c_void_p, c_int64, c_int32, c_void_p)
dion_weight_grad_workspace = _sig("dion_weight_grad_workspace", c_size_t, _P(GradSource), c_int32)
dion_weight_grad = _sig("dion_weight_grad", c_int32, _P(GradSource), c_int32, c_int32, c_void_p,
                        c_size_t, c_void_p, c_void_p)
dion_step_from_saved_workspace = _sig("dion_step_from_saved_workspace", c_size_t, c_void_p,
                                      _P(GradSource), c_int32)
dion_step_batched_from_saved = _sig("dion_step_batched_from_saved", c_int32, c_void_p,
                                    _P(BucketPtrs), _P(GradSource), c_int32, c_int32, c_float,
                                    c_void_p, c_size_t, c_void_p, c_void_p, c_void_p)
dion_norm_forward = _sig("dion_norm_forward", c_int32, _P(Norm), c_void_p)
dion_norm_backward_workspace = _sig("dion_norm_backward_workspace", c_size_t, c_int64, c_int64)
dion_norm_backward = _sig("dion_norm_backward", c_int32, _P(NormGrad), c_void_p, c_size_t, c_void_p)
dion_embed_lookup = _sig("dion_embed_lookup", c_int32, _P(Embed), c_void_p)
dion_embed_backward_workspace = _sig("dion_embed_backward_workspace", c_size_t, c_int64, c_int64)
dion_embed_backward = _sig("dion_embed_backward", c_int32, _P(EmbedGrad), c_void_p, c_size_t,
                           c_void_p)

EXPORTED = ["dion_act_save", "dion_act_load", "dion_weight_grad_workspace", "dion_weight_grad",
            "dion_step_from_saved_workspace", "dion_step_batched_from_saved", "dion_norm_forward",
            "dion_norm_backward_workspace", "dion_norm_backward", "dion_embed_lookup",
            "dion_embed_backward_workspace", "dion_embed_backward"]


_CODES = {}     # torch dtype -> dion_dtype; filled on first use (torch is imported lazily)


def _dtype_codes() -> dict:
    if not _CODES:
        import torch
        _CODES.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16,
                       torch.float32: DTYPE_FP32})
    return _CODES


def _dtype(t) -> int:
    code = _dtype_codes().get(t.dtype)
    if code is None:
        raise ValueError(f"bf16, fp16 or fp32 expected, got {t.dtype}")
    return code


class _Owned:
    """Device memory that a plan allocates, on the stream that is current then (the home stream).
    Once freed, the caching allocator gives it to the home stream's next allocation at once, so
    every other stream that uses it is named to the allocator (record_stream), which then waits
    for that stream's work; and that stream waits for what the home stream had enqueued when the
    memory was handed out: the work of its last owner, and the zeroing of status words."""

    def __init__(self, *tensors):
        import torch
        self.tensors = tensors
        home = torch.cuda.current_stream(tensors[0].device)
        self.streams, self._made = {home.cuda_stream}, None
        # (made inside a capture, the memory is the graph's, whose streams all fork from this one)
        if not _capturing(home):
            self._made = torch.cuda.Event()
            self._made.record(home)

    def use(self, stream):
        for t in self.tensors:
            t.record_stream(stream)
        # an event of before a capture cannot be waited for inside it; the replays come after the
        # work before the capture, and the next call outside waits
        if not _capturing(stream):
            if self._made is not None:
                stream.wait_event(self._made)
            self.streams.add(stream.cuda_stream)


def _capturing(stream) -> bool:
    import torch
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


class _Bound:
    """Tensors of one plan: checked, kept alive, all on one device."""

    def __init__(self):
        self._device, self._keep, self._owned = None, [], []
        self._known = None      # the last call's stream, which may use all of _owned

    def _tensor(self, name, t, dtype=None):
        import torch
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if self._device is None:
            self._device = t.device
        elif t.device != self._device:
            raise ValueError(f"{name} is on {t.device}, the others on {self._device}")
        self._keep.append(t)
        return t

    def _rows(self, name, t, shape, dtype=None):
        """(pointer, row stride) of a 2-D tensor with contiguous features."""
        self._tensor(name, t, dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: the features must be contiguous")
        ld = t.stride(0) if shape[0] > 1 else shape[1]
        if ld < shape[1]:
            raise ValueError(f"{name}: its rows overlap (row stride {ld})")
        return t.data_ptr(), ld

    def _vector(self, name, t, n):
        """Pointer of a contiguous fp32 vector of n elements; None passes."""
        import torch
        if t is None:
            return None
        self._tensor(name, t, torch.float32)
        if tuple(t.shape) != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous vector of {n}")
        return t.data_ptr()

    def _workspace(self, workspace, nbytes, status_words=0):
        """(pointer, bytes) of the caller's workspace, or of one that the plan allocates; and the
        plan's zeroed status words."""
        import torch
        own = []
        if workspace is None:
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=self._device)
            own.append(workspace)
        self._tensor("workspace", workspace, torch.uint8)
        if workspace.numel() < nbytes or not workspace.is_contiguous():
            raise ValueError(f"workspace must be {nbytes} contiguous bytes, got {workspace.numel()}")
        self.workspace_bytes = nbytes
        status = None
        if status_words:
            status = torch.zeros(status_words, dtype=torch.int32, device=self._device)
            own.append(status)
        if own:
            self._owned.append(_Owned(*own))
        return c_void_p(workspace.data_ptr()), workspace.numel(), status

    def _checkpoint(self, k):
        """An ActCheckpoint that the plan reads or writes."""
        self._tensor("checkpoint", k.q)
        self._keep.append(k)
        self._owned += [o for o in k._owned if o not in self._owned]

    def _stream(self, stream):
        import torch
        device = torch.cuda.current_device()
        if device != self._device.index:
            raise ValueError(f"the plan's tensors are on {self._device}, the current device is "
                             f"cuda:{device}")
        # the handle alone: a Stream object takes longer than the launch
        raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
        if raw != self._known:
            self._other_stream(raw, torch.cuda.current_stream(device) if stream is None else stream)
        return raw

    def _other_stream(self, raw, stream):
        """The stream (another one than the last call's) may use the plan's own memory."""
        for owned in self._owned:
            if raw not in owned.streams:
                owned.use(stream)
        if all(raw in owned.streams for owned in self._owned):
            self._known = raw


# ------------------------------------------------------------------ activations in 8 bits
class ActCheckpoint(_Bound):
    """Activations [tokens, features] kept in 8 bits: e4m3 bytes ``q`` [tokens, ld] (ld =
    features rounded up to 32) and a power-of-two exponent byte per 32 features, ``scale``
    [tokens, ld / 32].  ``save`` fills them, ``load`` reads them back (exact in bf16)."""

    def __init__(self, tokens: int, features: int, *, q=None, scale=None, device=None):
        import torch
        super().__init__()
        if tokens < 0 or features < 1:
            raise ValueError("tokens >= 0 and features >= 1 expected")
        self.tokens, self.features = int(tokens), int(features)
        ld = -(-self.features // ACT_BLOCK) * ACT_BLOCK
        own = []
        if q is None:
            q = torch.empty(self.tokens, ld, dtype=torch.uint8, device=device or "cuda")
            own.append(q)
        if scale is None:
            scale = torch.empty(self.tokens, ld // ACT_BLOCK, dtype=torch.uint8, device=q.device)
            own.append(scale)
        for name, t, shape in (("q", q, (self.tokens, ld)),
                               ("scale", scale, (self.tokens, ld // ACT_BLOCK))):
            self._tensor(name, t, torch.uint8)
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {shape}, got {tuple(t.shape)}")
        self.q, self.scale = q, scale
        self.args = ActKept(q.data_ptr(), scale.data_ptr(), self.tokens, self.features)
        self._keep, self._shape = [q, scale], (self.tokens, self.features)
        if own:
            self._owned.append(_Owned(*own))
        self._ref = ctypes.byref(self.args)
        _dtype_codes()

    def _arg(self, name, x):
        """x's pointer, row stride and type; x itself is the caller's to keep."""
        import torch
        # the usual case in a few comparisons: this is a call a layer, not a plan
        code = _CODES.get(x.dtype) if isinstance(x, torch.Tensor) else None
        if code is not None and x.device == self._device and x.shape == self._shape:
            ld, one = x.stride()
            if one == 1 and ld >= self.features:
                return x.data_ptr(), ld, code
        kept = len(self._keep)
        try:
            ptr, ld = self._rows(name, x, self._shape)
            return ptr, ld, _dtype(x)
        finally:                     # refused or not, x is not kept
            del self._keep[kept:]

    def save(self, x, stream=None):
        """Keep x [tokens, features] (bf16, fp16 or fp32)."""
        ptr, ld, ty = self._arg("x", x)
        _check(dion_act_save(ptr, ld, ty, self._ref, self._stream(stream)),
               "dion_act_save")

    def load(self, out, stream=None):
        """Write what was kept into out [tokens, features] (bf16, fp16 or fp32)."""
        ptr, ld, ty = self._arg("out", out)
        _check(dion_act_load(self._ref, ptr, ld, ty, self._stream(stream)),
               "dion_act_load")
        return out


def _sources(bound, checkpoints, dys, transposed):
    """GradSource array of (kept, D) pairs; G is filled in by the caller."""
    import torch
    n = len(checkpoints)
    if len(dys) != n:
        raise ValueError("checkpoints and output gradients must have one entry per matrix")
    arr = (GradSource * max(n, 1))()
    for i, (k, d) in enumerate(zip(checkpoints, dys)):
        if not isinstance(k, ActCheckpoint):
            raise ValueError(f"matrix {i}: an ActCheckpoint is expected")
        bound._checkpoint(k)
        if getattr(d, "ndim", 0) != 2:
            raise ValueError(f"matrix {i}: dy must be [tokens, n]")
        arr[i].kept = k.args
        arr[i].d, arr[i].ldd = bound._rows("dy", d, (k.tokens, d.shape[1]), torch.bfloat16)
        arr[i].n = d.shape[1]
        arr[i].transposed = int(bool(transposed))
    return arr


class WeightGradPlan(_Bound):
    """G = A^T dY of each matrix, from its input A kept in 8 bits (an ActCheckpoint of
    [tokens, m]) and its output's gradient dY (bf16 [tokens, n]); G fp32 [m, n], or with
    ``transposed`` dY^T A, [n, m].  ``status`` (int32, one word per matrix) takes
    DION_MAT_TIMEOUT where a device wait ran out, and keeps it until it is zeroed."""

    def __init__(self, checkpoints, dys, grads, *, transposed=False, workspace=None):
        import torch
        super().__init__()
        arr = _sources(self, checkpoints, dys, transposed)
        if len(grads) != len(checkpoints):
            raise ValueError("one gradient per matrix is expected")
        for i, g in enumerate(grads):
            m, n = checkpoints[i].features, dys[i].shape[1]
            arr[i].G, arr[i].ldg = self._rows("G", g, (n, m) if transposed else (m, n),
                                              torch.float32)
        self.n, self._arr = len(grads), arr
        self._ws, self._ws_bytes = c_void_p(), 0
        self.status = None
        if self.n:
            need = dion_weight_grad_workspace(arr, self.n)
            self._ws, self._ws_bytes, self.status = self._workspace(workspace, need, self.n)

    def backward(self, accumulate=False, stream=None):
        if not self.n:
            return
        _check(dion_weight_grad(self._arr, self.n, int(bool(accumulate)), self._ws, self._ws_bytes,
                                c_void_p(self.status.data_ptr()), self._stream(stream)),
               "dion_weight_grad")


class SavedStep(_Bound):
    """A Dion step whose gradients come from kept activations: ``opt`` (a DionB200) and, per
    matrix in the step's order, an ActCheckpoint and dY.  ``step`` forms every gradient in
    its slot of G and takes the step (dion_step_batched_from_saved); a matrix whose gradient ran
    out of device waits is left alone, and marked DION_MAT_TIMEOUT in ``step``'s status and, until
    it is zeroed, in ``grad_status``."""

    def __init__(self, opt, checkpoints, dys, *, transposed=False, workspace=None):
        import torch
        super().__init__()
        self.opt = opt
        if len(checkpoints) != opt.num_matrices:
            raise ValueError(f"{opt.num_matrices} matrices are planned, {len(checkpoints)} given")
        self._arr = _sources(self, checkpoints, dys, transposed)
        i = 0
        for s in opt.shapes:
            for _ in range(s.count):
                shape = (checkpoints[i].features, dys[i].shape[1])
                if (shape[::-1] if transposed else shape) != (s.m, s.n):
                    raise ValueError(f"matrix {i}: its gradient is not {(s.m, s.n)}")
                i += 1
        need = dion_step_from_saved_workspace(opt._h, self._arr, opt.num_matrices)
        self._ws, self._ws_bytes, self.grad_status = self._workspace(workspace, need,
                                                                     opt.num_matrices)

    def step(self, X, M, G, Q, lr: float, status=None, accumulate=False, stream=None):
        import torch
        arr = self.opt._ptrs(X, M, G, Q)
        for name, ts in (("X", X), ("M", M), ("G", G), ("Q", Q)):
            for i, t in enumerate(ts):
                if t.device != self._device:
                    raise ValueError(f"bucket {i}: {name} is on {t.device}, the checkpoints are on "
                                     f"{self._device}")
        if status is not None:
            if not isinstance(status, torch.Tensor) or status.device != self._device \
                    or status.dtype != torch.int32 or not status.is_contiguous() \
                    or status.numel() < self.opt.num_matrices:
                raise ValueError(f"status must be {self.opt.num_matrices} contiguous int32 words on "
                                 f"{self._device}")
        _check(dion_step_batched_from_saved(
            self.opt._h, arr, self._arr, len(self.opt.shapes), int(bool(accumulate)), float(lr),
            self._ws, self._ws_bytes,
            c_void_p(status.data_ptr()) if status is not None else None,
            c_void_p(self.grad_status.data_ptr()), self._stream(stream)),
            "dion_step_batched_from_saved")


# ------------------------------------------------------------------ norm
def _post_norm(y, post_norm, post_gain):
    if post_norm is None:
        return post_gain is not None
    return bool(post_norm)


class NormPlan(_Bound):
    """h = x + residual_scale gate * (post_gain * y rms(y)) and u = pre_gain * h rms(h).

    Rows [tokens, features] of one dtype; ``pre_gain``, ``post_gain``, ``gate`` fp32
    [features] or None (ones).  y is normalised where ``post_norm`` (default: where
    post_gain is given).  ``checkpoint`` (ActCheckpoint) receives u in 8 bits as well."""

    def __init__(self, x, y=None, *, h=None, u=None, pre_gain=None, post_gain=None, gate=None,
                 residual_scale=1.0, eps=1e-6, post_norm=None, checkpoint=None):
        super().__init__()
        if getattr(x, "ndim", 0) != 2:
            raise ValueError("x must be [tokens, features]")
        a = Norm(tokens=x.shape[0], features=x.shape[1], dtype=_dtype(x), eps=eps,
                 residual_scale=residual_scale, post_norm=_post_norm(y, post_norm, post_gain))
        a.x, a.ldx = self._rows("x", x, x.shape)
        for name, t in (("y", y), ("h", h), ("u", u)):
            if t is not None:
                ptr, ld = self._rows(name, t, x.shape, x.dtype)
                setattr(a, name, ptr)
                setattr(a, "ld" + name, ld)
        for name, t in (("pre_gain", pre_gain), ("post_gain", post_gain), ("gate", gate)):
            setattr(a, name, self._vector(name, t, x.shape[1]))
        if checkpoint is not None:
            self._checkpoint(checkpoint)
            a.kept = ctypes.pointer(checkpoint.args)
        self._args = a
        self._ref = ctypes.byref(a)

    def forward(self, stream=None):
        _check(dion_norm_forward(self._ref, self._stream(stream)), "dion_norm_forward")


class NormGradPlan(_Bound):
    """The gradients of NormPlan's outputs at the stored h and y (h is x where there is no y).

    ``du``, ``dh``: gradients of u and, from elsewhere, of h.  Written where given: ``dx``,
    ``dy`` (rows), ``dpre_gain``, ``dpost_gain``, ``dgate`` (fp32 [features])."""

    def __init__(self, h, y=None, *, du=None, dh=None, dx=None, dy=None, pre_gain=None,
                 post_gain=None, gate=None, dpre_gain=None, dpost_gain=None, dgate=None,
                 residual_scale=1.0, eps=1e-6, post_norm=None, workspace=None):
        super().__init__()
        if getattr(h, "ndim", 0) != 2:
            raise ValueError("h must be [tokens, features]")
        a = NormGrad(tokens=h.shape[0], features=h.shape[1], dtype=_dtype(h), eps=eps,
                     residual_scale=residual_scale, post_norm=_post_norm(y, post_norm, post_gain))
        for name, t in (("h", h), ("y", y), ("du", du), ("dh", dh), ("dx", dx), ("dy", dy)):
            if t is not None:
                ptr, ld = self._rows(name, t, h.shape, h.dtype)
                setattr(a, name, ptr)
                setattr(a, "ld" + name, ld)
        for name, t in (("pre_gain", pre_gain), ("post_gain", post_gain), ("gate", gate),
                        ("dpre_gain", dpre_gain), ("dpost_gain", dpost_gain), ("dgate", dgate)):
            setattr(a, name, self._vector(name, t, h.shape[1]))
        need = dion_norm_backward_workspace(h.shape[0], h.shape[1])
        self._ws, self._ws_bytes, _ = self._workspace(workspace, need)
        self._args = a
        self._ref = ctypes.byref(a)

    def backward(self, accumulate=False, stream=None):
        """``accumulate`` adds to dpre_gain, dpost_gain and dgate."""
        self._args.accumulate = int(bool(accumulate))
        _check(dion_norm_backward(self._ref, self._ws, self._ws_bytes, self._stream(stream)),
               "dion_norm_backward")


# ------------------------------------------------------------------ embedding
def _ids(bound, ids):
    import torch
    bound._tensor("ids", ids)
    if ids.dtype not in (torch.int32, torch.int64) or ids.ndim != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous vector of int32 or int64")
    return ids.data_ptr(), ids.element_size()


class EmbedPlan(_Bound):
    """out[t] = scale * table[ids[t]]; an id outside the table gives a row of zeros."""

    def __init__(self, table, ids, out, *, scale=1.0):
        super().__init__()
        if getattr(table, "ndim", 0) != 2:
            raise ValueError("table must be [vocab, features]")
        a = Embed(vocab=table.shape[0], features=table.shape[1], tokens=ids.numel(), scale=scale,
                  table_dtype=_dtype(table))
        a.ids, a.id_bytes = _ids(self, ids)
        a.table, a.ldt = self._rows("table", table, table.shape)
        a.out, a.ldo = self._rows("out", out, (ids.numel(), table.shape[1]))
        a.out_dtype = _dtype(out)
        self._args = a
        self._ref = ctypes.byref(a)

    def lookup(self, stream=None):
        _check(dion_embed_lookup(self._ref, self._stream(stream)), "dion_embed_lookup")


class EmbedGradPlan(_Bound):
    """dtable[v] = scale * the sum of dout's rows whose id is v; fp32, every row written
    (with ``accumulate`` added to, rows without a token left alone)."""

    def __init__(self, ids, dout, dtable, *, scale=1.0, workspace=None):
        import torch
        super().__init__()
        if getattr(dtable, "ndim", 0) != 2:
            raise ValueError("dtable must be [vocab, features]")
        a = EmbedGrad(vocab=dtable.shape[0], features=dtable.shape[1], tokens=ids.numel(),
                      scale=scale)
        a.ids, a.id_bytes = _ids(self, ids)
        a.dout, a.ldo = self._rows("dout", dout, (ids.numel(), dtable.shape[1]))
        a.dtype = _dtype(dout)
        a.dtable, a.ldt = self._rows("dtable", dtable, dtable.shape, torch.float32)
        need = dion_embed_backward_workspace(ids.numel(), dtable.shape[1])
        self._ws, self._ws_bytes, _ = self._workspace(workspace, need)
        self._args = a
        self._ref = ctypes.byref(a)

    def backward(self, accumulate=False, stream=None):
        self._args.accumulate = int(bool(accumulate))
        _check(dion_embed_backward(self._ref, self._ws, self._ws_bytes, self._stream(stream)),
               "dion_embed_backward")
