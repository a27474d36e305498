"""GPU parity of activation checkpoints in 8 bits and of the steps that read them.

Codes, scales and restored values are compared bit for bit with the definition (oracle/checkpoint_oracle.py). Scores
and packed rows carry the oracle's element bounds of fp32 arithmetic. The backward from checkpoints is held to the bounds
of the backward from stored rows (bf16: dH per element 2^-8 |ref| + 2e-5 rms of the row, weight and input gradients rel.
Frobenius 5e-3 as PhiW and dH are stored in bf16, the FC2 weight gradient 1e-5 against the stored PhiW; f32: 1e-5)
against the exact oracle on the restored values."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
import oracle
import synth
from oracle import checkpoint_oracle as co

from gpu_util import DEV, Staged, as_f64, bits, check_selection, log, rel_fro
from test_gpu_parity import SMALL, _make

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rows(n, width, dt, kind, seed=0):
    rng = np.random.default_rng(n * 7 + width + seed)
    x = rng.standard_normal((n, width))
    if kind == "ties":  # whole and half steps of scales with few bits, most of them exact ties
        x = rng.integers(-254, 255, (n, width)) / 2.0
        x[:, ::128] = 127.0
        x *= 2.0 ** rng.integers(-40, 40, (n, 1)) * rng.choice([1.0, 1.5, 1.25, 1 + 2.0 ** -7], (n, 1))
    elif kind == "near_ties":  # a last place beside the halves
        x = rng.integers(-253, 254, (n, width)) / 2.0
        x[:, ::128] = 127.0
        x = x * rng.choice([1.0, 1 + 2.0 ** -7, 1.1640625], (n, 1)) * (1 + rng.integers(-2, 3, (n, width)) * 2.0 ** -23)
    elif kind == "spread":
        x *= np.exp(rng.standard_normal((n, width)) * 4)
    elif kind == "tiny_ties":  # ties and their neighbours of scales just over the smallest
        x = rng.integers(-254, 255, (n, width)) / 2.0
        x[:, ::128] = 127.0
        x *= rng.integers(128, 160, (n, 1)) * 2.0 ** (rng.integers(0, 4, (n, 1)) - 133.0)
    elif kind == "tiny":  # down to subnormal values, and rows of zeros
        x *= 2.0 ** rng.integers(-150, -115, (n, 1))
        x[::5] = 0
    elif kind == "huge":
        x *= 2.0 ** rng.integers(118, 127, (n, 1))
        m = 3.3895313892515355e38 if dt == "bf16" else np.finfo(np.float32).max
        x = np.clip(x, -m, m)
        x[::3, ::131] = m
    elif kind == "bad":
        for v in (np.nan, np.inf, -np.inf):
            x[rng.random((n, width)) < 1e-3] = v
    return torch.from_numpy(x.astype(np.float32)).to(DEV).to(TYPES[dt])


def _same(got, ref):
    assert np.array_equal(got, ref, equal_nan=True), np.argwhere(~((got == ref) | (np.isnan(got) & np.isnan(ref))))[:5]


@pytest.mark.parametrize("n,parts,width,dt,kind", [
    (1, 1, 8, "f32", "normal"), (1, 1, 8, "bf16", "normal"), (3, 2, 8, "bf16", "spread"), (70, 1, 120, "f32", "spread"),
    (65, 1, 128, "bf16", "ties"), (64, 2, 128, "f32", "ties"), (33, 1, 136, "bf16", "near_ties"),
    (50, 1, 1536, "f32", "near_ties"), (257, 2, 768, "bf16", "normal"), (257, 2, 768, "bf16", "ties"),
    (100, 2, 1408, "bf16", "spread"), (999, 1, 520, "f32", "normal"), (40, 3, 264, "bf16", "tiny"),
    (40, 3, 264, "f32", "tiny"), (3000, 1, 256, "bf16", "tiny_ties"), (3000, 1, 256, "f32", "tiny_ties"), (40, 2, 264, "bf16", "huge"), (40, 1, 384, "f32", "huge"), (300, 2, 256, "bf16", "bad"),
    (300, 1, 200, "f32", "bad"), (5, 1, 20000, "bf16", "normal"), (30011, 1, 24, "f32", "spread"),
    (3001, 2, 640, "bf16", "near_ties")])
def test_codes_and_values(n, parts, width, dt, kind):
    x = _rows(n, parts * width, dt, kind)
    log(f"checkpoint {n} rows of {parts} x {width} {dt} {kind}")
    c = lr.checkpoint(x, parts=parts)
    torch.cuda.synchronize()
    q, s = co.checkpoint(as_f64(x), parts)
    _same(as_f64(c.scale), s)
    _same(c.q.cpu().numpy().astype(np.float64), q)
    v = co.values(q, s)
    with np.errstate(over="ignore"):  # 127 scales may round past the largest number
        exact = v.astype(np.float32)
    _same(as_f64(lr.restore(c, dtype=torch.float32)), exact.astype(np.float64))
    _same(as_f64(lr.restore(c)), torch.from_numpy(exact).bfloat16().double().numpy())


def test_few_bits_lose_nothing():
    """Values that are codes already come back as they were."""
    x = torch.randint(-127, 128, (64, 256), device=DEV).float()
    x[:, ::128] = 127.0
    log("codes as they were")
    c = lr.checkpoint(x)
    assert torch.equal(c.scale, torch.ones_like(c.scale)) and torch.equal(c.q.float(), x)
    assert torch.equal(lr.restore(c, dtype=torch.float32), x)


def test_no_rows_and_given_buffers():
    log("no rows")
    c = lr.checkpoint(torch.empty(0, 64, device=DEV), parts=2)
    assert c.q.shape == (0, 64) and c.scale.shape == (0, 2, 1) and lr.restore(c).shape == (0, 64)
    x = _rows(20, 264, "bf16", "normal")
    big = lr.Checkpoint(torch.full((23, 264), 99, dtype=torch.int8, device=DEV),
                        torch.full((23, 1, 3), 7.0, dtype=torch.bfloat16, device=DEV))
    assert lr.checkpoint(x, out=big) is big
    a = lr.checkpoint(x)
    assert torch.equal(big.q[:20], a.q) and torch.equal(big.scale[:20], a.scale)
    assert torch.all(big.q[20:] == 99) and torch.all(big.scale[20:] == 7)  # rows behind are left as they were
    out = torch.empty(20, 264, dtype=torch.bfloat16, device=DEV)
    assert lr.restore(a, out=out) is out and torch.equal(out, lr.restore(a))
    with pytest.raises(ValueError):
        lr.checkpoint(x.t().contiguous().t())
    with pytest.raises(lr.LrmoeError):  # rows that start in the middle of a 16-byte unit
        lr.checkpoint(x.view(-1)[4:4 + 264].view(1, 264))


def _saved(s, pr):
    """The checkpoint of a staged problem's saved rows, and the same in fp64."""
    sw = pr.cfg.swiglu
    c = lr.checkpoint(s.H if sw else s.Phi, parts=2 if sw else 1)
    q, scale = c.q.cpu().numpy().astype(np.float64), as_f64(c.scale)
    return c, q, scale


@pytest.fixture(scope="module", params=sorted(SMALL))
def case(request):
    log(f"case {request.param}: generating")
    pr = _make(request.param)
    s = Staged(pr)
    return request.param, pr, s, *_saved(s, pr)


def test_score(case):
    name, pr, s, c, q, scale = case
    log(f"score {name}")
    R = lr.score_checkpoint(s.P, s.G, c, s.alpha, s.tok)
    ref, err = co.score(as_f64(s.G), q, scale, pr.routing.alpha, pr.routing.tok, pr.cfg.swiglu)
    d = np.abs(as_f64(R) - ref)
    assert np.all(d <= err), np.max(d / err)


@pytest.mark.parametrize("swiglu,dt", [(True, "bf16"), (False, "bf16"), (True, "f32")])
def test_score_by_launch_plan(swiglu, dt):
    """Many gradient words: both norms in one launch where the workspace has room for the pairs', else in two; and few
    words, each pair on its own. Tokens outside [0, T) score 0 in each."""
    T, K, E, D, F = 1100, 8, 3, 2048 if dt == "bf16" else 1024, 136
    rng = np.random.default_rng(9)
    seg = np.array([0, 3000, 3000, T * K])
    H = _rows(T * K, F * (2 if swiglu else 1), dt, "normal")
    G = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(DEV).to(TYPES[dt])
    tok = rng.integers(0, T, T * K).astype(np.int32)
    tok[::97], tok[5] = -1, T
    alpha = rng.random(T * K).astype(np.float32)
    c = lr.checkpoint(H, parts=2 if swiglu else 1)
    q, scale = c.q.cpu().numpy().astype(np.float64), as_f64(c.scale)
    out = (tok < 0) | (tok >= T)
    ref, err = co.score(as_f64(G), q, scale, alpha, np.where(out, 0, tok), swiglu)
    for t_of, few in ((T, False), (T // 10, True)):  # the fewer tokens: pairs of the first T // 10 tokens' count
        n = t_of * K
        p = lr.Problem(E=E, T=T if not few else t_of, K=K, D=D, F=F, swiglu=swiglu, dtype=lr.BF16 if dt == "bf16" else lr.F32,
                       seg_off=np.minimum(seg, n), quota=np.diff(np.minimum(seg, n)), device=DEV)
        tk = torch.from_numpy(np.where(tok[:n] < p.T, tok[:n], -1)).to(DEV)
        part = lr.Checkpoint(c.q[:n], c.scale[:n])
        gone = tk.cpu().numpy() < 0
        for room in (8 * (p.T + 64), 8 * (p.T + 64 + p.N)):
            log(f"score plan {swiglu} {dt} {p.T} tokens, {room} bytes")
            p.workspace = lambda mode=0, b=room: torch.empty(b, dtype=torch.uint8, device=DEV)
            R = as_f64(lr.score_checkpoint(p, G[:p.T], part, torch.from_numpy(alpha[:n]).to(DEV), tk))
            assert not R[gone].any()
            assert np.all((np.abs(R - ref[:n]) <= err[:n])[~gone])


def test_compact(case):
    name, pr, s, c, q, scale = case
    N = s.P.N
    rng = np.random.default_rng(3)
    sel = np.sort(rng.permutation(N)[:s.P.K_tot]).astype(np.int32)
    sel[rng.random(len(sel)) < 0.05] = -1
    sel[rng.random(len(sel)) < 0.05] = N
    log(f"compact {name}")
    dt = TYPES[pr.cfg.dtype]
    out = torch.full((s.P.K_tot + 3, pr.cfg.F), -7.0, dtype=dt, device=DEV)
    got = lr.compact_checkpoint(s.P, torch.from_numpy(sel).to(DEV), c, s.alpha, out=out)
    ref, err = co.compact(sel, q, scale, pr.routing.alpha, pr.cfg.swiglu, pr.cfg.dtype == "bf16")
    d = np.abs(as_f64(got) - ref)
    assert np.all(d <= err), np.max(d / np.maximum(err, 1e-300))
    assert torch.all(out[s.P.K_tot:] == -7)


def _reference(pr, sel, q, scale, X):
    """The exact oracle's steps 3 to 5 on the restored values (fp64)."""
    r, c = pr.routing, pr.cfg
    cseg = np.concatenate([[0], np.cumsum(pr.quota)]).astype(np.int64)
    v = co.values(q, scale)[sel]
    P, t = co.phi(v, c.swiglu)[0], r.tok[sel].astype(np.int64)
    D = r.alpha[sel].astype(np.float64)[:, None] * oracle.widen(pr.G, c.dtype)[t]
    if c.swiglu:
        dW1, dW2, dH, dX = oracle.swiglu_expert_backward(cseg, D, P, X[t], v, oracle.widen(pr.W1, c.dtype),
                                                         oracle.widen(pr.W2, c.dtype))
        return {"dW1": dW1, "dW2": dW2, "dH": dH, "dIn": dX, "out": oracle.scatter_tokens(dX, t, c.T), "cseg": cseg}
    dW2, dPhi = oracle.linear_expert_backward(cseg, D, P, oracle.widen(pr.W2, c.dtype))
    return {"dW2": dW2, "dIn": dPhi, "out": oracle.scatter_tokens(dPhi, t, c.T), "cseg": cseg}


def _run(s, pr, c, X, **kw):
    sw = pr.cfg.swiglu
    return lr.backward(s.P, G=s.G, Phi=None if sw else c, H=c if sw else None, X=X, alpha=s.alpha, tok=s.tok,
                       slot=s.slot, W2=s.W2, W1=s.W1, **kw)


@pytest.mark.parametrize("x8", [False, True])
def test_backward(case, x8):
    name, pr, s, c, q, scale = case
    x8 = x8 and pr.cfg.swiglu  # FC2-only problems read no X
    bf = pr.cfg.dtype == "bf16"
    X = lr.checkpoint(s.X) if x8 else s.X
    log(f"backward {name} {'X in 8 bits' if x8 else ''}")
    bufs = {}
    for again in range(2):  # the second with the first's buffers
        res = _run(s, pr, c, X, bufs=bufs)
    torch.cuda.synchronize()
    R, _ = co.score(as_f64(s.G), q, scale, pr.routing.alpha, pr.routing.tok, pr.cfg.swiglu)
    sel = res["sel"].cpu().numpy().astype(np.int64)
    check_selection(sel, R, pr.routing.seg_off, pr.quota)
    xs = None if s.X is None else as_f64(lr.restore(X, dtype=TYPES[pr.cfg.dtype]) if x8 else s.X)
    ref = _reference(pr, sel, q, scale, xs)
    cseg = ref["cseg"]
    PhiW = as_f64(res["PhiW"])
    tol = 5e-3 if bf else 1e-5
    t = pr.routing.tok[sel].astype(np.int64)
    G = oracle.widen(pr.G, pr.cfg.dtype)
    for e in range(pr.cfg.E):
        a, b = cseg[e], cseg[e + 1]
        for k in ("dW2", "dW1") if pr.cfg.swiglu else ("dW2",):
            assert rel_fro(as_f64(res[k][e]), ref[k][e]) <= tol, (k, e)
        if b > a:
            assert rel_fro(as_f64(res["dW2"][e]), PhiW[a:b].T @ G[t[a:b]]) <= 1e-5
            assert rel_fro(as_f64(res["dIn"][a:b]), ref["dIn"][a:b]) <= tol
    if pr.cfg.swiglu and len(sel):
        dH, want = as_f64(res["dH"]), ref["dH"]
        rms = np.sqrt(np.mean(want * want, axis=1, keepdims=True))
        bound = (2.0 ** -8 * np.abs(want) + 2e-5 * rms) if bf else 2e-5 * rms + 1e-5 * np.abs(want)
        assert np.all(np.abs(dH - want) <= bound), np.max(np.abs(dH - want) / bound)
    assert rel_fro(as_f64(res["out"][:pr.cfg.T]), ref["out"]) <= tol


def test_overlapped_scatter_gives_the_same(case):
    name, pr, s, c, q, scale = case
    log(f"overlapped scatter {name}")
    a, b = _run(s, pr, c, s.X), _run(s, pr, c, s.X, overlap_scatter=True)
    torch.cuda.synchronize()
    for k in ("out", "dW2", "sel") + (("dW1", "dH") if pr.cfg.swiglu else ()):
        n = pr.cfg.T if k == "out" else None
        assert torch.equal(a[k][:n], b[k][:n]), k


def test_pairs_outside_and_a_bad_first_row():
    """Packed rows of no pair give zeros though row 0, whose words their loads read, is NaN."""
    pr = _make("swiglu_ragged")
    s = Staged(pr)
    H = s.H.clone()
    H[0, 3] = float("inf")
    H[0, pr.cfg.F + 130] = float("nan")
    c = lr.checkpoint(H, parts=2)
    p = s.P
    sel, _, maps = lr.select(p, lr.score(p, s.G, s.Phi, s.alpha, s.tok), tok=s.tok, slot=s.slot)
    sel, ctok = sel.clone(), maps["ctok"].clone()
    keep0 = (sel == 0).nonzero()
    sel[keep0] = 1
    out_of = torch.tensor([2, 300, 301], device=DEV)
    sel[out_of], ctok[out_of] = torch.tensor([-1, p.N, -5], dtype=torch.int32, device=DEV), -1
    log("pairs outside")
    PhiW = lr.compact_checkpoint(p, sel, c, s.alpha)
    g = lr.grouped_gemm_bwd_checkpoint(p, s.G, s.alpha, sel, ctok, PhiW, s.W2, s.X, c, s.W1)
    torch.cuda.synchronize()
    for t in (PhiW, g["dH"], g["dIn"]):
        assert not t[out_of].any() and torch.isfinite(t.float()).all()
    assert torch.isfinite(g["dW1"]).all() and torch.isfinite(g["dW2"]).all()


@pytest.mark.parametrize("pairs,quota", [(0, 0), (40, 0)])
def test_nothing_retained(pairs, quota):
    """No pairs at all, and pairs of which none is kept: zero gradients."""
    T, K, D, F = 30, 2, 64, 40
    bf = lambda *d: torch.randn(*d, device=DEV).bfloat16()  # noqa: E731
    p = lr.Problem(E=2, T=T, K=K, D=D, F=F, swiglu=True, dtype=lr.BF16, seg_off=[0, pairs // 4, pairs],
                   quota=[quota, quota], device=DEV)
    tok = torch.arange(max(pairs, 1), dtype=torch.int32, device=DEV) % T
    slot = torch.arange(max(pairs, 1), dtype=torch.int32, device=DEV) // T
    alpha, X, W1, W2 = torch.rand(max(pairs, 1), device=DEV), bf(T, D), bf(2, D, 2 * F), bf(2, F, D)
    log(f"nothing retained of {pairs}")
    f = lr.expert_forward_checkpoint(p, X, tok, alpha, W1, W2)
    assert f["H"].q.shape == (pairs, 2 * F)
    res = lr.backward(p, G=bf(T, D), H=f["H"], X=lr.checkpoint(X), alpha=alpha, tok=tok, slot=slot, W2=W2, W1=W1)
    torch.cuda.synchronize()
    assert res["sel"].numel() == 0 and not res["dW1"].any() and not res["dW2"].any() and not res["out"][:T].any()


def test_offsets_past_32_bits():
    """Codes, rows and packed rows behind the 2^32nd value."""
    T, K, F = 360_000, 8, 768
    N = T * K  # 2880000 rows of 1536: 4.4e9 values
    keep = 5000
    x = torch.zeros(N, 2 * F, dtype=torch.bfloat16, device=DEV)
    x[-keep:] = _rows(keep, 2 * F, "bf16", "spread")
    log("checkpoint of 4.4e9 values")
    c = lr.checkpoint(x, parts=2)
    q, s = co.checkpoint(as_f64(x[-keep:]), 2)
    _same(c.q[-keep:].cpu().numpy().astype(np.float64), q)
    _same(as_f64(c.scale[-keep:]), s)
    assert not c.q[:-keep].any()
    lr.restore(c, out=x)
    _same(as_f64(x[-keep:]), torch.from_numpy(co.values(q, s).astype(np.float32)).bfloat16().double().numpy())
    assert not x[:-keep].any()
    del x
    p = lr.Problem(E=2, T=T, K=K, D=8, F=F, swiglu=True, dtype=lr.BF16, seg_off=[0, 100, N], quota=[0, N - 100], device=DEV)
    G = torch.ones(T, 8, dtype=torch.bfloat16, device=DEV)
    tok = (torch.arange(N, device=DEV) // K).int()
    alpha = torch.rand(N, device=DEV)
    log("scores and packed rows")
    R = lr.score_checkpoint(p, G, c, alpha, tok)
    a = alpha[-keep:].cpu().numpy()
    ref, err = co.score(np.ones((1, 8)), q, s, a, np.zeros(keep, np.int64), True)
    assert np.all(np.abs(as_f64(R[-keep:]) - ref) <= err) and not R[:-keep].any()
    P = lr.compact_checkpoint(p, torch.arange(100, N, dtype=torch.int32, device=DEV), c, alpha)
    ref, err = co.compact(np.arange(keep), q, s, a, True, True)
    assert np.all(np.abs(as_f64(P[-keep:]) - ref) <= err) and not P[:-keep].any()


FORWARD = {
    "ragged": synth.custom("ckpt_fwd_ragged", T=600, K=4, E=6, D=512, F=384, counts=(700, 0, 513, 300, 257, 1), seed=31),
    "odd_dims": synth.custom("ckpt_fwd_odd", T=100, K=2, E=4, D=136, F=72, counts=(50, 17, 0, 90), seed=32),
    "wide": synth.custom("ckpt_fwd_wide", T=150, K=3, E=3, D=2304, F=136, counts=(200, 90, 110), seed=34),
    "small": synth.custom("ckpt_fwd_small", T=3, K=1, E=2, D=40, F=8, counts=(0, 1), seed=36),
}


@pytest.mark.parametrize("name", sorted(FORWARD))
def test_forward_saves_the_checkpoint_of_its_rows(name):
    pr = synth.make_problem(FORWARD[name], rho="0.6")
    s = Staged(pr)
    log(f"forward {name}")
    a = lr.expert_forward(s.P, s.X, s.tok, s.alpha, s.W1, s.W2)
    H = lr.Checkpoint(torch.full((s.P.N + 2, 2 * pr.cfg.F), 99, dtype=torch.int8, device=DEV),
                      torch.full((s.P.N + 2, 2, co.groups(pr.cfg.F)), 7.0, dtype=torch.bfloat16, device=DEV))
    b = lr.expert_forward_checkpoint(s.P, s.X, s.tok, s.alpha, s.W1, s.W2, out={"H": H})
    c = lr.checkpoint(a["H"], parts=2)
    torch.cuda.synchronize()
    assert torch.equal(b["H"].q, c.q) and torch.equal(b["H"].scale, c.scale)
    assert torch.equal(a["Phi"], b["Phi"]) and torch.equal(a["Y"], b["Y"])
    assert torch.all(H.q[s.P.N:] == 99) and torch.all(H.scale[s.P.N:] == 7)


def _step(s, c, x8, bufs):
    """Forward with checkpoints, then the backward from them."""
    lr.checkpoint(s.X, out=x8)
    f = lr.expert_forward_checkpoint(s.P, s.X, s.tok, s.alpha, s.W1, s.W2, out={"H": c, "Phi": bufs["Phi"], "Y": bufs["Y"]})
    return lr.backward(s.P, G=s.G, H=f["H"], X=x8, alpha=s.alpha, tok=s.tok, slot=s.slot, W2=s.W2, W1=s.W1,
                       bufs=bufs["bwd"])


def test_captured_step_replays():
    """A layer's forward and backward through checkpoints as one graph, replayed with new inputs in its buffers."""
    pr = synth.make_problem(FORWARD["ragged"], rho="0.6")
    s, P = Staged(pr), pr.cfg
    c = lr.Checkpoint(torch.empty(s.P.N, 2 * P.F, dtype=torch.int8, device=DEV),
                      torch.empty(s.P.N, 2, co.groups(P.F), dtype=torch.bfloat16, device=DEV))
    x8 = lr.checkpoint(s.X)
    bf = torch.bfloat16
    bufs = {"Phi": torch.empty(s.P.N, P.F, dtype=bf, device=DEV), "Y": torch.empty(s.P.N, P.D, dtype=bf, device=DEV),
            "bwd": {}}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(s, c, x8, bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(s, c, x8, bufs)
    X0, G0 = s.X.clone(), s.G.clone()
    for i in range(3):
        s.X.copy_(X0 * (1 + i))
        s.G.copy_(G0.roll(i, 0))
        log(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        got = {k: out[k].clone() for k in ("sel", "PhiW", "dH", "dW1", "dW2", "out")}
        other = {"Phi": torch.empty_like(bufs["Phi"]), "Y": torch.empty_like(bufs["Y"]), "bwd": {}}
        ref = _step(s, lr.Checkpoint(torch.empty_like(c.q), torch.empty_like(c.scale)), lr.checkpoint(s.X), other)
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], ref[k]), (i, k)


def test_on_another_stream():
    pr = synth.make_problem(FORWARD["ragged"], rho="0.6")
    s = Staged(pr)
    ref = lr.checkpoint(s.X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    log("checkpoint on a stream")
    c = lr.checkpoint(s.X, stream=side)
    back = lr.restore(c, stream=side)
    f = lr.expert_forward_checkpoint(s.P, s.X, s.tok, s.alpha, s.W1, s.W2, stream=side)
    R = lr.score_checkpoint(s.P, s.G, f["H"], s.alpha, s.tok, stream=side)
    side.synchronize()
    assert torch.equal(c.q, ref.q) and torch.equal(back, lr.restore(ref))
    f2 = lr.expert_forward_checkpoint(s.P, s.X, s.tok, s.alpha, s.W1, s.W2)
    assert torch.equal(f["H"].q, f2["H"].q) and torch.equal(R, lr.score_checkpoint(s.P, s.G, f2["H"], s.alpha, s.tok))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_largest_values(dt):
    """Groups whose largest magnitude is at or next to the type's largest finite number: codes are the definition's, and
    f32 values stay finite; bf16 ones may round to an infinity, as the nearest bf16 number of code times scale does."""
    rng = np.random.default_rng(3)
    big = torch.finfo(TYPES[dt]).max
    x = rng.uniform(-1, 1, (40, 256)) * big
    x[:, 5] = big * np.where(np.arange(40) % 2, 1.0, -1.0)
    x[:, 200] = big * (1 - 2.0 ** -np.arange(40).clip(1, 22 if dt == "f32" else 8))
    rows = torch.from_numpy(x).to(TYPES[dt]).to(DEV)
    log("rows at the end of the range")
    c = lr.checkpoint(rows)
    back, back16 = lr.restore(c, dtype=torch.float32), lr.restore(c, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    q, scale = co.checkpoint(as_f64(rows), 1)
    assert np.array_equal(c.q.cpu().numpy(), q) and np.array_equal(as_f64(c.scale), scale)
    v = co.values(q, scale)
    assert np.isfinite(as_f64(back)).all() and np.array_equal(as_f64(back), v)
    assert torch.equal(back16.cpu(), torch.from_numpy(v).float().bfloat16())
