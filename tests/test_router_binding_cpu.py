"""The binding of the router's operators and of AdamW without a GPU: what has to be refused before the
library is called. Tensors, streams and the library are stand-ins, so that a call that is wrongly let
through is seen and not run."""
import types

import pytest
import torch

import load_recalibrated_expert_amd as lr


class Tensor:
    """What the binding asks of a device tensor."""

    def __init__(self, shape, dtype, dev, at=1 << 20):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at
        self.device = torch.device("cpu" if dev < 0 else f"cuda:{dev}")

    def get_device(self):
        return -1 if self.device.type == "cpu" else self.device.index

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def record_stream(self, stream):
        pass

    def copy_(self, values, non_blocking=False):
        pass

    @property
    def is_cuda(self):
        return self.device.type == "cuda"


class Library:
    """Counts the calls that would launch; the host-only ones are the real library's."""

    def __init__(self, real):
        self.real, self.launched = real, []

    def __getattr__(self, name):
        if name.endswith("_size") or name in ("lrmoe_adamw_step_scalars", "lrmoe_adamw_plan"):
            return getattr(self.real, name)
        return lambda *a: self.launched.append(name) or 0


@pytest.fixture
def gpu(monkeypatch):
    """A current device (gpu.here) with stand-ins behind the binding; gpu.lib.launched lists the launches."""
    g = types.SimpleNamespace(here=0, lib=Library(lr.library()))
    monkeypatch.setattr(lr, "library", lambda: g.lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: g.here, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 7000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def empty(shape, dtype, device, stream):
        d = torch.device(device)
        return Tensor(shape, dtype, -1 if d.type == "cpu" else g.here if d.index is None else d.index)

    monkeypatch.setattr(lr, "_empty", empty)
    return g


def _calls(r, dev=0):
    x, idx = Tensor((r.T, r.E), torch.float32, dev), Tensor((r.T, r.K), torch.int32, dev)
    bal = {"counts": Tensor((1, r.E), torch.int32, dev), "norm": Tensor((1,), torch.float32, dev)}
    return (lambda **kw: lr.route(r, x, **kw), lambda **kw: lr.balance_loss(r, x, idx, **kw),
            lambda **kw: lr.route_bwd(r, x, idx, balance=bal, **kw))


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_a_router_of_another_device_is_refused(gpu, device):
    """Its workspace and the outputs it allocates are not on the device that the kernels run on."""
    for call in _calls(lr.Router(T=8, E=4, K=2, device=device)):
        with pytest.raises(ValueError):
            call()
    assert gpu.lib.launched == []
    for call in _calls(lr.Router(T=8, E=4, K=2, device="cuda:0")):
        call()
    assert gpu.lib.launched == ["lrmoe_route", "lrmoe_balance_loss", "lrmoe_route_bwd"]


def test_a_router_stays_on_the_device_of_its_workspace(gpu):
    """device="cuda" is the current one: a workspace of device 0 is not used by a call on device 1."""
    r = lr.Router(T=8, E=4, K=2, device="cuda")
    route, balance, _ = _calls(r, 0)
    route()
    gpu.here = 1
    route, balance, _ = _calls(r, 1)
    for call in (route, balance):
        with pytest.raises(ValueError):
            call()
    assert gpu.lib.launched == ["lrmoe_route"]


class Stream:
    def __init__(self, dev, raw):
        self.device_index, self.cuda_stream = dev, raw
        self.device = torch.device("cuda", dev)


def test_a_stream_of_another_device_is_refused(gpu):
    """A kernel launched there would run on that device, with this one's buffers."""
    p = types.SimpleNamespace(T=8, K=2, D=8, N=9, torch_dtype=torch.bfloat16, device="cuda:0",
                              c=lr._lib.CProblem())
    rows, alpha = Tensor((9, 8), torch.bfloat16, 0), Tensor((9,), torch.float32, 0)
    opt = lr.AdamW([torch.zeros(64)], grads=[torch.zeros(64)])
    opt._check_place = lambda: None
    opt.m[0] = opt.v[0] = Tensor((64,), torch.float32, 0)
    calls = _calls(lr.Router(T=8, E=4, K=2, device="cuda:0")) + (
        lambda **kw: lr.alpha_grad(p, rows, rows, alpha, Tensor((8, 2), torch.int32, 0), **kw),
        lambda **kw: opt.step(**kw))
    for call in calls:
        with pytest.raises(ValueError):
            call(stream=Stream(1, 7001))
    assert gpu.lib.launched == [] and opt.t == 0


@pytest.fixture
def capture(gpu, monkeypatch):
    """gpu with a set of streams (None: the current one) that record into a graph."""
    gpu.capturing, at = set(), [None]

    class on:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, at[0] = at[0], self.stream

        def __exit__(self, *a):
            at[0] = self.before

    gpu.current = lambda: at[0]
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at[0] in gpu.capturing)
    return gpu


def _adamw(n=1):
    opt = lr.AdamW([torch.zeros(64) for _ in range(n)], grads=[torch.zeros(64) for _ in range(n)])
    opt._check_place = lambda: None
    opt._used_on = lr._stream
    return opt


def test_a_step_on_a_capturing_stream_is_refused(capture):
    """step(stream=s) while s, which is not the current stream, records a graph that would repeat this step."""
    opt, side = _adamw(), Stream(0, 7100)
    capture.capturing = {side}
    with pytest.raises(ValueError):
        opt.step(stream=side)
    assert opt.t == 0 and capture.lib.launched == []
    opt.step()
    opt.step(stream=Stream(0, 7200))
    assert opt.t == 2
    capture.capturing = {None}
    for s in (None, side):
        with pytest.raises(ValueError):
            opt.step(stream=s)
    assert opt.t == 2


def test_a_graph_of_a_side_stream_keeps_what_it_reads(capture):
    """step_captured(stream=s) while s records: the gradient buffers stay with the object when others are bound."""
    opt, side = _adamw(), Stream(0, 7100)
    opt.advance()
    grads = opt.grads
    capture.capturing = {side}
    opt.step_captured(stream=side)
    opt.bind([torch.zeros(64)])
    assert any(g is grads for _, g in opt._captured)


def test_a_plan_is_not_copied_while_its_stream_records(capture):
    """A copy to the device would be an error inside the capture, and would end it."""
    opt, side = _adamw(49), Stream(0, 7100)
    opt.advance()
    opt._plan = False  # as after a first step
    capture.capturing = {side}
    opt.step_captured(stream=side)
    assert opt._plan is False and capture.lib.launched == ["lrmoe_adamw"]


class Scalars(Tensor):
    """AdamW's scalars on the device: the stream of every copy into them."""

    def __init__(self, gpu, fails=False):
        super().__init__((8,), torch.int32, 0)
        self.gpu, self.fails, self.copies = gpu, fails, []

    def copy_(self, values, non_blocking=False):
        if self.fails:
            raise RuntimeError("no copy")
        self.copies.append(self.gpu.current())


def _on_device(opt, scalars, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
    opt.w = [Tensor((64,), torch.float32, 0)]
    opt._scalars = scalars
    return opt


def test_advance_copies_on_the_stream_of_the_replays(capture, monkeypatch):
    """Elsewhere the copy could overtake a replay that still reads the step before."""
    opt, side = _on_device(_adamw(), Scalars(capture), monkeypatch), Stream(0, 7100)
    opt.advance(stream=side)
    opt.advance()
    assert opt._scalars.copies == [side, None] and opt.t == 2
    with pytest.raises(ValueError):
        opt.advance(stream=Stream(1, 7001))
    assert opt._scalars.copies == [side, None] and opt.t == 2


def test_advance_inside_a_capture_counts_no_step(capture, monkeypatch):
    opt, side = _on_device(_adamw(), Scalars(capture), monkeypatch), Stream(0, 7100)
    for capturing, stream in ((None, None), (side, side), (None, side)):
        capture.capturing = {capturing}
        with pytest.raises(ValueError):
            opt.advance(stream=stream)
    assert opt.t == 0 and opt._scalars.copies == []


def test_an_advance_whose_copy_fails_counts_no_step(capture, monkeypatch):
    opt = _on_device(_adamw(), Scalars(capture, fails=True), monkeypatch)
    with pytest.raises(RuntimeError):
        opt.advance()
    assert opt.t == 0


def test_a_gradient_over_the_logits_is_refused(gpu):
    """Rows of the logits that other tokens still read would be overwritten."""
    r = lr.Router(T=8, E=5, K=2, device="cuda:0")
    idx = Tensor((8, 2), torch.int32, 0)
    at = 1 << 20
    x = Tensor((8, 5), torch.float32, 0, at)
    for shift in (0, 20, 159, -20, -159):
        with pytest.raises(ValueError):
            lr.route_bwd(r, x, idx, dalpha=Tensor((8, 2), torch.float32, 0), out=Tensor((8, 5), torch.float32, 0, at + shift))
    assert gpu.lib.launched == []
    for shift in (160, -160):
        lr.route_bwd(r, x, idx, dalpha=Tensor((8, 2), torch.float32, 0), out=Tensor((8, 5), torch.float32, 0, at + shift))
    assert gpu.lib.launched == ["lrmoe_route_bwd"] * 2


def test_an_outgrown_workspace_is_kept_for_graphs_alone(capture):
    """One that no captured call has used is given back; one that a graph may replay with is not."""
    r, side = lr.Router(T=8, E=4, K=2, device="cuda:0"), Stream(0, 7100)
    for n_seq in range(1, 3000, 97):
        r.workspace(n_seq)
    assert r._grown == []
    kept = []
    for n_seq, stream in ((4000, None), (6000, side)):
        capture.capturing = {stream}
        kept.append(r.workspace(1, stream))  # large enough already
        capture.capturing = set()
        for more in (0, 500, 1000):
            assert r.workspace(n_seq + more) is not kept[-1]
        assert all(a is b for a, b in zip(r._grown, kept)) and len(r._grown) == len(kept)
    capture.capturing = {side}
    kept.append(r.workspace(9000, side))  # allocated inside a capture; the one before it was never in one
    capture.capturing = set()
    r.workspace(10000)
    assert all(a is b for a, b in zip(r._grown, kept)) and len(r._grown) == 3


def test_adamw_notes_its_own_buffers_once_per_stream(capture, monkeypatch):
    """record_stream, once for each stream, of what the object allocated: not of moments that the caller gave,
    and not of everything again when a plan or the scalars are new."""
    noted = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: noted.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    n, current = 60, Stream(0, 7000)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: current)
    w, g = ([torch.zeros(64) for _ in range(n)] for _ in range(2))
    given = [torch.zeros(64) for _ in range(n)]
    opt = lr.AdamW(w, grads=g, m=given)
    opt._check_place = lambda: None
    side = Stream(0, 7100)
    for _ in range(4):  # the second one makes the plan
        opt.step()
    opt.step(stream=side)
    opt.step(stream=side)
    own = {t.data_ptr() for t in opt.v}
    plan = opt._plan.data_ptr()
    assert sorted(noted, key=str) == sorted([(p, s) for p in own | {plan} for s in (current, side)], key=str)
    opt.bind([t.clone() for t in g])
    opt.step()
    opt.step()  # another plan
    assert noted[-1] == (opt._plan.data_ptr(), current) and len(noted) == 2 * (n + 1) + 1


def test_offsets_copied_to_another_device_are_refused(gpu):
    """Host offsets go to the router's device: route_bwd with a given output uses nothing else that is there."""
    r = lr.Router(T=8, E=4, K=2, device="cpu")
    x, idx = Tensor((8, 4), torch.float32, 0), Tensor((8, 2), torch.int32, 0)
    bal = {"counts": Tensor((2, 4), torch.int32, 0), "norm": Tensor((2,), torch.float32, 0)}
    for off in ([0, 3, 8], torch.tensor([0, 3, 8])):
        with pytest.raises(ValueError):
            lr.route_bwd(r, x, idx, balance=bal, seq_off=off, out=Tensor((8, 4), torch.float32, 0, 1 << 30))
    assert gpu.lib.launched == []


def test_advance_on_another_device_is_refused(capture, monkeypatch):
    """Its stream, like step_captured's, is one of the current device."""
    opt = _on_device(_adamw(), Scalars(capture), monkeypatch)
    del opt._check_place
    monkeypatch.setattr(torch.cuda, "current_device", lambda: capture.here)
    opt.advance()
    capture.here = 1
    with pytest.raises(ValueError):
        opt.advance()
    assert opt.t == 1 and len(opt._scalars.copies) == 1
