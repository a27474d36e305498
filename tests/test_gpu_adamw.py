"""GPU parity of the AdamW step (lrmoe_adamw): weights and 32-bit states against fp64 within the bound
of fp32 arithmetic, 8-bit states code by code against the header's formulas in f32."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import router_oracle as ro

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
SIZES = [1, 2, 3, 255, 256, 257, 1000, 4095, 4096, 4097, 12289, 70003]


def _tensors(sizes, dt, rng, std):
    out = []
    for n in sizes:
        a = (rng.standard_normal(n) * std * np.exp2(rng.integers(-8, 3, n))).astype(np.float32)
        a[rng.random(n) < 0.05] = 0
        out.append(torch.from_numpy(a).to(DEV).to(dt))
    return out


def _codes(t):
    return t.view(torch.uint8).cpu().view(torch.float8_e4m3fn).double().numpy()


def _check(opt, before, g, t, dt, master, bits, grad_scale, hyper, first, seed):
    for i, n in enumerate(len(a) for a in before["w"]):
        G = as_f64(g[i])
        w0, m0, v0 = (before[k][i] for k in ("w", "m", "v"))
        (w, m, v), (ew, em, ev) = ro.adamw(w0, G, m0, v0, t=t, grad_scale=grad_scale, **hyper)
        got = as_f64(opt.masters[i] if master else opt.w[i])
        e = ew if (master or dt == torch.float32) else ew + np.abs(w) * 2.0 ** -8 + 1e-38
        assert np.all(np.abs(got - w) <= e), (i, n, np.max(np.abs(got - w) / e))
        if master:  # the rounded copy, bit for bit
            assert torch.equal(opt.w[i], opt.masters[i].bfloat16())
        if bits == 32:
            assert np.all(np.abs(as_f64(opt.m[i]) - m) <= em) and np.all(np.abs(as_f64(opt.v[i]) - v) <= ev)
            continue
        m1, v1, r1 = ro.adamw_f32(as_f64(g[i]).astype(np.float32), m0.astype(np.float32), v0.astype(np.float32),
                                  hyper["betas"], grad_scale)
        lo, hi = ro.random_bits(n, first[i], seed, t)
        for name, x, rnd, signed in (("m", m1, lo, True), ("v", r1, hi, False)):
            q, s = ro.quantise(x, rnd, signed)
            assert np.array_equal(as_f64(getattr(opt, name + "_scale")[i]), s), (name, i)
            assert np.array_equal(_codes(getattr(opt, name)[i]), q, equal_nan=True), (name, i)


def _state(opt, master, bits):
    w = [as_f64(t) for t in (opt.masters if master else opt.w)]
    if bits == 32:
        return {"w": w, "m": [as_f64(t) for t in opt.m], "v": [as_f64(t) for t in opt.v]}
    m = [ro.dequantise(_codes(t), as_f64(s)) for t, s in zip(opt.m, opt.m_scale)]
    r = [ro.dequantise(_codes(t), as_f64(s)) for t, s in zip(opt.v, opt.v_scale)]
    return {"w": w, "m": m, "v": [(a.astype(np.float32) * a.astype(np.float32)).astype(np.float64) for a in r]}


KINDS = [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt,master", KINDS, ids=["f32", "bf16", "bf16_master"])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16], ids=["g32", "g16"])
def test_steps(bits, dt, master, gdt):
    rng = np.random.default_rng(bits + 10 * master)
    w = _tensors(SIZES, torch.float32, rng, 0.05)
    masters = w if master else None
    w = [t.to(dt) if master or dt != torch.float32 else t for t in w]
    opt = lr.AdamW(w, masters=masters, bits=bits, seed=77, **HYPER)
    at = np.cumsum([0] + [(n + 255) // 256 * 256 for n in SIZES])
    for t in range(1, 5):
        g = _tensors(SIZES, gdt, rng, 1e-3 * 4 ** t)
        scale = 1.0 if t < 3 else 0.37
        before = _state(opt, master, bits)
        log(f"adamw {bits} bits {dt} master={master} {gdt} step {t}")
        opt.step(g, grad_scale=scale)
        torch.cuda.synchronize()
        assert opt.t == t
        _check(opt, before, g, t, dt, master, bits, scale, HYPER, at, 77)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_equal_single_calls(bits):
    """More tensors than one launch takes, empty ones among them: the same as one call for each."""
    rng = np.random.default_rng(9)
    sizes = [int(n) for n in rng.integers(0, 3000, 131)]
    sizes[3] = sizes[48] = sizes[130] = 0
    w = _tensors(sizes, torch.float32, rng, 0.05)
    g = _tensors(sizes, torch.float32, rng, 0.01)
    one = [t.clone() for t in w]
    first = list(np.cumsum([0] + [(n + 255) // 256 * 256 for n in sizes[:-1]]))
    opt = lr.AdamW(w, grads=g, bits=bits, seed=5, **HYPER)
    log(f"adamw {len(sizes)} tensors")
    for _ in range(2):
        opt.step()
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        o = lr.AdamW([one[i]], grads=[g[i]], bits=bits, seed=5, first=[int(first[i])], **HYPER)
        for _ in range(2):
            o.step()
        assert torch.equal(o.w[0], opt.w[i]) and torch.equal(o.m[0].view(torch.uint8), opt.m[i].view(torch.uint8))
        assert torch.equal(o.v[0].view(torch.uint8), opt.v[i].view(torch.uint8))


def test_views_leave_their_neighbours():
    """Tensors that are views of one buffer: elements between and behind them stay as they were."""
    n, gap = 1001, 23
    step = 1024
    flat = torch.full((3 * step,), 9.0, device=DEV)
    g = torch.full((3 * step,), 0.5, device=DEV)
    cut = lambda b: [b[i * step:i * step + n] for i in range(3)]  # noqa: E731
    m8, r8 = (torch.full((3 * step,), 0x11, dtype=torch.uint8, device=DEV) for _ in range(2))
    scale = [torch.full((3 * 4,), 2.0, device=DEV) for _ in range(2)]
    per = lambda b: [b[i * 4:i * 4 + 4] for i in range(3)]  # noqa: E731
    opt = lr.AdamW(cut(flat), grads=cut(g), m=cut(m8.view(torch.float8_e4m3fn)), v=cut(r8.view(torch.float8_e4m3fn)),
                   m_scale=per(scale[0]), v_scale=per(scale[1]), bits=8, **HYPER)
    log("views of one buffer")
    opt.step()
    torch.cuda.synchronize()
    for i in range(3):
        assert torch.all(flat[i * step + n:(i + 1) * step] == 9.0) and gap == step - n
        assert torch.all(m8[i * step + n:(i + 1) * step] == 0x11) and torch.all(r8[i * step + n:(i + 1) * step] == 0x11)
        assert torch.all(flat[i * step:i * step + n] != 9.0)


@pytest.mark.parametrize("plan", [False, True])
def test_more_elements_than_one_launch_takes(plan):
    """18.3e9 elements, 8-bit states: more chunks than a launch has blocks, so that the update takes two,
    with the second one's start inside a tensor. The first step from zero states does the same to
    every element of a tensor, and what it does is checked on a small one."""
    if torch.cuda.mem_get_info()[0] < 96 << 30:
        pytest.skip("needs 96 GB of device memory")
    n, tensors = (1 << 30) + 256, 17
    sizes = [n] * tensors + [1000] * (40 if plan else 1)
    w = [torch.full((k,), 0.5 + i / 64, dtype=torch.bfloat16, device=DEV) for i, k in enumerate(sizes)]
    g = torch.full((n,), 0.25, dtype=torch.bfloat16, device=DEV)
    small = torch.full((1024,), 0.25, dtype=torch.bfloat16, device=DEV)
    opt = lr.AdamW(w, grads=[g] * tensors + [small[:1000]] * (len(sizes) - tensors), bits=8, **HYPER)
    small_w = [torch.full((64,), 0.5 + i / 64, dtype=torch.bfloat16, device=DEV) for i in range(len(sizes))]
    log(f"{sum(sizes)} elements in {len(sizes)} tensors, plan: {plan}")
    if plan:
        opt._plan = False  # as after a first step
    opt.step()
    assert isinstance(opt._plan, torch.Tensor) == plan
    torch.cuda.synchronize()
    twin = lr.AdamW(small_w, grads=[small[:64]] * len(sizes), bits=8, **HYPER)
    twin.step()
    for i, (a, b) in enumerate(zip(opt.w, twin.w)):
        lo, hi = a.aminmax()
        assert lo == hi == b[0] and b[0] != 0.5 + i / 64, i
        assert opt.v_scale[i].min() == opt.v_scale[i].max() == twin.v_scale[i][0], i
        assert opt.m_scale[i].min() == opt.m_scale[i].max() == twin.m_scale[i][0], i


def test_not_finite_gradients():
    """An infinite or NaN gradient spoils its own element only: the block's scale comes from the rest."""
    n = 700
    rng = np.random.default_rng(2)
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DEV)
    bad = [0, 5, 300, 699]
    g[0], g[5], g[300], g[699] = float("inf"), float("nan"), -float("inf"), 3e38
    for bits in (32, 8):
        w = torch.ones(n, device=DEV)
        opt = lr.AdamW([w], grads=[g], bits=bits, seed=1, **HYPER)
        before = _state(opt, False, bits)
        log(f"gradients that are not finite, {bits} bits")
        opt.step()
        torch.cuda.synchronize()
        good = np.ones(n, bool)
        good[bad] = False
        (wr, _, _), (ew, _, _) = ro.adamw(before["w"][0][good], as_f64(g)[good], before["m"][0][good],
                                          before["v"][0][good], t=1, **HYPER)
        assert np.all(np.abs(as_f64(w)[good] - wr) <= ew)
        if bits == 8:
            m1, _, r1 = ro.adamw_f32(as_f64(g).astype(np.float32), before["m"][0].astype(np.float32),
                                     before["v"][0].astype(np.float32), HYPER["betas"])
            lo, hi = ro.random_bits(n, 0, 1, 1)
            for got, sc, x, rnd, signed in ((opt.m, opt.m_scale, m1, lo, True), (opt.v, opt.v_scale, r1, hi, False)):
                q, s = ro.quantise(x, rnd, signed)
                assert np.array_equal(as_f64(sc[0]), s) and np.array_equal(_codes(got[0]), q, equal_nan=True)


def test_tiny_and_huge_states():
    """Blocks of subnormal and of very large moments: scales at both ends of their range."""
    n = 1024
    g = torch.full((n,), 1e-40, device=DEV)
    g[256:512], g[512:768], g[768:] = 1e-38, 1e19, 0.0
    w = torch.zeros(n, device=DEV)
    opt = lr.AdamW([w], grads=[g], bits=8, seed=4, **HYPER)
    before = _state(opt, False, 8)
    log("tiny and huge states")
    opt.step()
    torch.cuda.synchronize()
    m1, _, r1 = ro.adamw_f32(as_f64(g).astype(np.float32), before["m"][0].astype(np.float32),
                             before["v"][0].astype(np.float32), HYPER["betas"])
    lo, hi = ro.random_bits(n, 0, 4, 1)
    for got, sc, x, rnd, signed in ((opt.m, opt.m_scale, m1, lo, True), (opt.v, opt.v_scale, r1, hi, False)):
        q, s = ro.quantise(x, rnd, signed)
        assert np.array_equal(as_f64(sc[0]), s) and np.array_equal(_codes(got[0]), q)
    assert float(opt.m_scale[0][3]) == 1.0 and torch.all(w[768:] == 0)


def test_8bit_second_moment_follows_the_gradient():
    """With beta2 = 0.999 a step changes v by less than half a spacing of e4m3; the random rounding
    moves its mean all the same. Mean over 4096 elements after 300 steps of a gradient a quarter of
    the start's: sqrt(v)'s mean within 2 percent of the exact root."""
    n = 4096
    opt = lr.AdamW([torch.zeros(n, device=DEV)], bits=8, seed=8, lr=0.0, betas=(0.9, 0.999))
    opt.step([torch.full((n,), 1.0, device=DEV)])
    r0 = np.sqrt(0.001)
    g = torch.full((n,), 0.25 * r0, device=DEV)
    for _ in range(300):
        opt.step([g])
    torch.cuda.synchronize()
    v = 0.001 * 0.999 ** 300 + (0.25 * r0) ** 2 * (1 - 0.999 ** 300)
    r = ro.dequantise(_codes(opt.v[0]), as_f64(opt.v_scale[0]))
    log(f"mean root {r.mean():.6f}, exact {np.sqrt(v):.6f}, start {r0:.6f}")
    assert abs(r.mean() / np.sqrt(v) - 1) < 0.02


def test_python_checks():
    w = [torch.zeros(64, device=DEV)]
    g = [torch.zeros(64, device=DEV)]
    opt = lr.AdamW(w, grads=g)
    with pytest.raises(ValueError):
        opt.step([g[0].cpu()])
    with pytest.raises(ValueError):
        opt.step([g[0].half()])
    with pytest.raises(ValueError):
        lr.AdamW([torch.zeros(64, 2, device=DEV)[:, 0]])  # strided
    good = torch.ones(64, device=DEV)
    two = lr.AdamW([torch.zeros(64, device=DEV) for _ in range(2)], grads=[good, good])
    table = [e.grad for e in two._table]
    with pytest.raises(ValueError):  # the second is strided: the first is not taken either
        two.step([torch.ones(64, device=DEV), torch.ones(64, 2, device=DEV)[:, 0]])
    assert [e.grad for e in two._table] == table and two.t == 0
    odd = lr.AdamW([torch.zeros(65, device=DEV)[1:]], grads=g)
    with pytest.raises(lr.LrmoeError):  # not 16-byte aligned
        odd.step()
    assert odd.t == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_replayed_graph(bits):
    """A captured step on a side stream: advance() before each replay, new gradients in the buffers, eager
    steps of a twin between the replays. Every replay equals the twin."""
    rng = np.random.default_rng(6)
    sizes = [1000, 257, 40000]
    w = _tensors(sizes, torch.float32, rng, 0.05)
    g = _tensors(sizes, torch.float32, rng, 0.01)
    twin = lr.AdamW([t.clone() for t in w], grads=g, bits=bits, seed=3, **HYPER)
    opt = lr.AdamW(w, grads=g, bits=bits, seed=3, **HYPER)
    side = torch.cuda.Stream()
    opt.step()
    twin.step()
    opt.advance()  # the first replay's scalars; a capture alone runs nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step_captured()
    for rep in range(4):
        if rep:
            for t, new in zip(g, _tensors(sizes, torch.float32, rng, 0.01)):
                t.copy_(new)
            opt.lr = twin.lr = 1e-2 / (rep + 1)
            opt.advance(grad_scale=0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        twin.step(grad_scale=0.5 if rep else 1.0)
        torch.cuda.synchronize()
        log(f"replay {rep}")
        assert opt.t == twin.t
        for a, b in zip(opt.w + opt.m + opt.v, twin.w + twin.m + twin.v):
            assert torch.equal(a.view(torch.uint8) if a.dtype != torch.float32 else a,
                               b.view(torch.uint8) if b.dtype != torch.float32 else b), rep


def test_rebinding_keeps_a_captured_graph():
    """A graph of more tensors than one launch's arguments take reads its plan: binding other gradient
    buffers afterwards leaves the graph, which still uses those it was captured with."""
    rng = np.random.default_rng(8)
    sizes = [300] * 60
    w = _tensors(sizes, torch.float32, rng, 0.05)
    g = _tensors(sizes, torch.float32, rng, 0.01)
    opt = lr.AdamW(w, grads=g, **HYPER)
    twin = lr.AdamW([t.clone() for t in w], grads=g, **HYPER)
    for o in (opt, twin):
        o.step()
        o.step()  # the second step makes the plan
    opt.advance()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            opt.step()
        opt.step_captured()
    opt.bind(_tensors(sizes, torch.float32, rng, 0.5))
    trash = [torch.full((100000,), 77, dtype=torch.uint8, device=DEV) for _ in range(50)]  # what bind freed
    log(f"replay after binding others, {len(trash)} buffers written")
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    twin.step()
    for a, b in zip(opt.w + opt.m + opt.v, twin.w + twin.m + twin.v):
        assert torch.equal(a, b)


def test_other_stream():
    """Steps on a side stream, the gradients written there: equal to steps on the current one."""
    rng = np.random.default_rng(12)
    w = _tensors([5000, 70001], torch.float32, rng, 0.05)
    g = _tensors([5000, 70001], torch.float32, rng, 0.01)
    twin = lr.AdamW([t.clone() for t in w], grads=[t.clone() for t in g], bits=8, **HYPER)
    opt = lr.AdamW(w, grads=g, bits=8, **HYPER)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    log("side stream")
    for _ in range(3):
        with torch.cuda.stream(side):
            for t in g:
                t.mul_(0.5)
        opt.step(stream=side)
        for t in twin.grads:
            t.mul_(0.5)
        twin.step()
    torch.cuda.synchronize()
    for a, b in zip(opt.w, twin.w):
        assert torch.equal(a, b)


def test_plan_and_states_freed_while_a_side_stream_uses_them():
    """Work queued on a side stream still reads the plan that bind drops and the states of an object that
    is gone: their memory is not given out before that work is done."""
    rng = np.random.default_rng(13)
    sizes = [300] * 60
    w = _tensors(sizes, torch.float32, rng, 0.05)
    g = _tensors(sizes, torch.float32, rng, 0.01)
    twin = lr.AdamW([t.clone() for t in w], grads=g, **HYPER)
    opt = lr.AdamW(w, grads=g, **HYPER)
    side = torch.cuda.Stream()
    for o in (opt, twin):
        o.step()
        o.step()  # makes the plan
    torch.cuda.synchronize()
    log("two steps behind a wait on the side stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # well over the host's time for what follows
        opt.step()
    opt.step(stream=side)
    held = {t.data_ptr() for t in [opt._plan] + opt.m + opt.v}
    bytes_ = [t.numel() * t.element_size() for t in [opt._plan, opt.m[0]]]
    opt.bind([t.clone() for t in g])
    del opt
    trash = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in bytes_ for _ in range(200)]
    assert not side.query(), "the side stream ended before the buffers were asked for"
    assert held.isdisjoint(t.data_ptr() for t in trash)
    torch.cuda.synchronize()
    twin.step()
    twin.step()
    for a, b in zip(w, twin.w):
        assert torch.equal(a, b)
