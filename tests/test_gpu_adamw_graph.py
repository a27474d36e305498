"""AdamW in captured graphs on streams that are busy: nothing waits for the device between the steps."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr

from gpu_util import DEV, log

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SIZES = [1000, 257, 40000]


def _tensors(rng, std):
    return [torch.from_numpy((rng.standard_normal(n) * std).astype(np.float32)).to(DEV) for n in SIZES]


def _same(opt, twin):
    for a, b in zip(opt.w + opt.m + opt.v, twin.w + twin.m + twin.v):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("current", [False, True], ids=["argument", "current"])
def test_advance_and_replay_on_a_busy_stream(bits, current):
    """The replays wait behind long work of their stream while the host has advanced past all of them: each one
    takes its own step's number, learning rate and random key."""
    rng = np.random.default_rng(21)
    w, g = _tensors(rng, 0.05), _tensors(rng, 0.01)
    opt = lr.AdamW([t.clone() for t in w], grads=g, bits=bits, seed=3, **HYPER)
    twin = lr.AdamW([t.clone() for t in w], grads=g, bits=bits, seed=3, **HYPER)
    rates = [1e-2 / (k + 1) for k in range(6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    log(f"capture, {bits} bits")
    opt.advance(stream=side)
    opt.t -= 1  # the capture runs nothing: the first replay's advance counts this step
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step_captured()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    for k, rate in enumerate(rates):
        opt.lr = rate
        if current:
            with torch.cuda.stream(side):
                opt.advance(grad_scale=1.0 - k / 8)
                graph.replay()
        else:
            opt.advance(grad_scale=1.0 - k / 8, stream=side)
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for k, rate in enumerate(rates):
        twin.lr = rate
        twin.step(grad_scale=1.0 - k / 8)
    torch.cuda.synchronize()
    log(f"{len(rates)} replays")
    assert opt.t == twin.t == len(rates)
    _same(opt, twin)


def test_capture_on_a_stream_given_by_name():
    """step_captured(stream=s) while s records; step(stream=s) there is refused and leaves the capture whole."""
    rng = np.random.default_rng(22)
    w, g = _tensors(rng, 0.05), _tensors(rng, 0.01)
    opt = lr.AdamW([t.clone() for t in w], grads=g, **HYPER)
    twin = lr.AdamW([t.clone() for t in w], grads=g, **HYPER)
    side = torch.cuda.Stream()
    opt.advance()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    log("capture on a side stream")
    with torch.cuda.graph(graph, stream=side):
        main = torch.cuda.current_stream()
        with torch.cuda.stream(torch.cuda.default_stream()):
            for refused in (opt.step, opt.advance):
                with pytest.raises(ValueError):
                    refused(stream=main)
            opt.step_captured(stream=main)
    opt.bind(_tensors(rng, 0.5))
    trash = [torch.full((n,), 7.0, device=DEV) for n in SIZES for _ in range(20)]
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    twin.step()
    torch.cuda.synchronize()
    assert opt.t == 1 and len(trash) == 60
    _same(opt, twin)
