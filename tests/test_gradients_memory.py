"""The device memory that a gradient plan allocates itself (workspace, status words, 8-bit rows),
used on other streams than the one it was allocated on.

On the host (no GPU): stand-ins for CUDA tensors and streams record which streams the allocator
is told of, and what they wait for.  On the GPU: plans dropped with their call still in flight."""
import types

import pytest
import torch

import rank_orthonormalized_optimizer_b200 as dion
from rank_orthonormalized_optimizer_b200 import gradients as gr


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it lies on cuda:0 and keeps the streams that it is recorded on."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.waited, self.capturing = handle, [], False

    def wait_event(self, event):
        self.waited.append(event.at)


class FakeEvent:
    def record(self, stream):
        self.at = (stream, stream.clock)


@pytest.fixture
def fake(monkeypatch):
    """torch's allocation and streams of a device that is not there; ``fake.current`` is the current
    stream, whose ``clock`` counts what was enqueued on it."""
    f = types.SimpleNamespace(current=FakeStream(1), made=[])
    f.current.clock = 0

    def tensor(make):
        def call(*shape, dtype=torch.float32, device=None):
            t = make(*shape, dtype=dtype).as_subclass(FakeCuda)
            if device is not None:
                f.made.append(t)
                f.current.clock += 1
            return t
        return call

    class Using:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, f.current = f.current, self.stream

        def __exit__(self, *_):
            f.current = self.before

    monkeypatch.setattr(torch, "empty", tensor(torch.empty))
    monkeypatch.setattr(torch, "zeros", tensor(torch.zeros))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: f.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", Using)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: f.current.capturing)
    monkeypatch.setattr(torch.cuda, "Event", FakeEvent)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: f.current.cuda_stream,
                        raising=False)
    for name in ("dion_embed_backward", "dion_norm_backward", "dion_norm_forward", "dion_weight_grad",
                 "dion_act_save", "dion_act_load", "dion_step_batched_from_saved"):
        monkeypatch.setattr(gr, name, lambda *a: dion.OK)
    return f


def _rows(t, d, dtype=torch.float32):
    return torch.ones(t, d, dtype=dtype).as_subclass(FakeCuda)


def _plans():
    """{name: (makes a plan and gives its call, how many tensors the plan allocates)}"""
    x, xb = _rows(64, 32), _rows(64, 32, torch.bfloat16)
    ids = torch.arange(64).as_subclass(FakeCuda)
    given = lambda: dion.ActCheckpoint(64, 32, q=_rows(64, 32, torch.uint8),  # noqa: E731
                                       scale=_rows(64, 1, torch.uint8))
    own = lambda: dion.ActCheckpoint(64, 32)  # noqa: E731
    opt = dion.DionB200([(1, 32, 32, 16)])
    X, M, G, Q = ([torch.ones(1, 32, n).as_subclass(FakeCuda)] for n in (32, 32, 32, 16))

    def saved():
        step = dion.SavedStep(opt, [given()], [xb])
        return lambda stream=None: step.step(X, M, G, Q, 0.1, stream=stream)

    def act(load):
        k = own()
        return lambda stream=None: (k.load if load else k.save)(x, stream=stream)

    return {
        "embed": (lambda: dion.EmbedGradPlan(ids, x, _rows(100, 32)).backward, 1),
        "norm": (lambda: dion.NormGradPlan(x, du=x, dx=x).backward, 1),
        "weight": (lambda: dion.WeightGradPlan([given()], [xb], [_rows(32, 32)]).backward, 2),
        "step": (saved, 2),
        "act": (lambda: act(False), 2),
        "act_load": (lambda: act(True), 2),
        "norm_kept": (lambda: dion.NormPlan(x, u=x, checkpoint=own()).forward, 2),
        "weight_kept": (lambda: dion.WeightGradPlan([own()], [xb], [_rows(32, 32)]).backward, 4),
    }


NAMES = ["embed", "norm", "weight", "step", "act", "act_load", "norm_kept", "weight_kept"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("how", ["argument", "current"])
def test_other_streams_are_named_to_the_allocator(fake, name, how):
    make, count = _plans()[name]
    call = make()
    home, side = fake.current, FakeStream(2)
    home.clock = 100                       # what is enqueued later is not waited for
    if how == "argument":
        call(stream=side)
    else:
        fake.current = side
        call()
    assert len(fake.made) == count
    for t in fake.made:
        assert getattr(t, "recorded", []) == [side]
    # the stream waits for what the home stream had enqueued by the last of the allocations (the
    # zeroing of a status among it)
    assert side.waited and side.waited[-1] == (home, count)


@pytest.mark.parametrize("name", NAMES)
def test_the_home_stream_needs_neither(fake, name):
    call = _plans()[name][0]()
    call()
    call(stream=fake.current)
    assert not fake.current.waited
    assert not any(hasattr(t, "recorded") for t in fake.made)


def test_a_stream_is_named_once_and_a_given_workspace_never(fake):
    ids, x = torch.arange(64).as_subclass(FakeCuda), _rows(64, 32)
    own = dion.EmbedGradPlan(ids, x, _rows(100, 32))
    fake.made.clear()
    given = torch.empty(1 << 20, dtype=torch.uint8).as_subclass(FakeCuda)
    plan = dion.EmbedGradPlan(ids, x, _rows(100, 32), workspace=given)
    side = FakeStream(2)
    for _ in range(3):
        own.backward(stream=side)
        plan.backward(stream=side)
    assert len(side.waited) == 1 and not hasattr(given, "recorded") and not fake.made


def test_a_capture_waits_for_nothing_outside(fake):
    """Inside a capture an event of before it may not be waited for; the first call after it is."""
    ids, x = torch.arange(64).as_subclass(FakeCuda), _rows(64, 32)
    plan = dion.EmbedGradPlan(ids, x, _rows(100, 32))
    side = FakeStream(2)
    side.capturing = True
    plan.backward(stream=side)
    assert not side.waited
    side.capturing = False
    plan.backward(stream=side)
    assert len(side.waited) == 1


def test_a_checkpoint_keeps_no_rows_that_it_is_given(fake):
    k = dion.ActCheckpoint(64, 32)
    mine = len(k._keep)
    for good in (_rows(64, 32), _rows(64, 40)[:, :32].as_subclass(FakeCuda)):
        k.save(good)
    for bad in (_rows(63, 32), _rows(64, 32).double().as_subclass(FakeCuda), torch.ones(64, 32),
                torch.ones(32, 64).as_subclass(FakeCuda).t(), "rows"):
        for call in (k.save, k.load):
            with pytest.raises(ValueError):
                call(bad)
    assert len(k._keep) == mine


# ------------------------------------------------------------------ on the GPU
@pytest.mark.gpu
@pytest.mark.parametrize("name", ["embed", "norm", "weight", "act"])
def test_a_plan_dropped_with_its_call_in_flight(name):
    """Built, called on a side stream behind a delay, and dropped: what the home stream allocates
    and fills meanwhile is other memory, and the result is the one of a quiet call."""
    g = torch.Generator().manual_seed(1)
    t, d = 3000, 256
    x = torch.randn(t, d, generator=g).cuda()
    xb = x.bfloat16()
    ids = torch.randint(0, 100, (t,), generator=g).cuda()

    def make(out):
        if name == "embed":
            p = dion.EmbedGradPlan(ids, x, out)
            return p.backward, p._keep[-1]
        if name == "norm":
            p = dion.NormGradPlan(x, du=x, dpre_gain=out)
            return p.backward, p._keep[-1]
        kept = dion.ActCheckpoint(t, d)
        kept.save(x)
        if name == "act":
            return lambda stream=None: kept.load(out, stream=stream), kept.q
        p = dion.WeightGradPlan([kept], [xb], [out])
        return p.backward, p._keep[-1]

    new = lambda: torch.empty({"embed": (100, d), "norm": (d,), "weight": (d, d),  # noqa: E731
                               "act": (t, d)}[name], device="cuda")
    want, out = new(), new()
    call, _ = make(want)
    call()
    torch.full((8,), 255, dtype=torch.uint8, device="cuda")   # its kernel is loaded
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call, mem = make(out)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)           # some 100 ms
    call(stream=side)
    where, size = mem.data_ptr(), mem.numel()
    del call, mem
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()                      # the call has not run yet
    assert all(j.data_ptr() != where for j in junk)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("inside", [True, False])
def test_plans_and_captures(inside):
    """A plan built inside a capture, and one of before it called on a stream that the capture has
    forked; both replayed, the second used outside as well."""
    t, v, d = 2000, 50, 128
    g = torch.Generator().manual_seed(3)
    ids, x = torch.randint(-1, v, (t,), generator=g).cuda(), torch.randn(t, d, generator=g).cuda()
    xb = x.bfloat16()
    want, out = [(torch.empty(v, d, device="cuda"), torch.empty(d, d, device="cuda")) for _ in range(2)]

    def make(table, G):
        kept = dion.ActCheckpoint(t, d)
        return kept, dion.WeightGradPlan([kept], [xb], [G]), dion.EmbedGradPlan(ids, x, table)

    def call(plans, stream=None):
        plans[0].save(x, stream=stream)
        plans[1].backward(stream=stream)
        plans[2].backward(stream=stream)

    call(make(*want))
    before = make(*out)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if inside:
            plans = make(*out)
            call(plans)
        else:
            side.wait_stream(torch.cuda.current_stream())
            call(before, side)
            torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for o in out:
            o.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    for o in out:
        o.fill_(9)
    side.wait_stream(torch.cuda.current_stream())
    call(before, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
