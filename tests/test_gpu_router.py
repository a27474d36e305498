"""GPU parity of the router's operators against their fp64 definitions (oracle/router_oracle.py,
which also gives each value's error bound in fp32 arithmetic): routing and pair lists, balance
loss, both gradients, at the sizes, masks and values where they can go wrong."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import router_oracle as ro

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu

# T, E, K, first, local, dtype, renorm, mask share, what the logits hold
CASES = {
    "one_token": (1, 8, 2, 0, 8, "f32", False, 0.0, "normal"),
    "one_expert": (37, 1, 1, 0, 1, "f32", True, 0.0, "normal"),
    "all_chosen": (50, 7, 7, 0, 7, "f32", True, 0.0, "normal"),
    "share": (1111, 128, 8, 0, 128, "f32", True, 0.0, "normal"),
    "share_bf16": (1111, 128, 8, 16, 16, "bf16", False, 0.2, "normal"),
    "odd_bf16": (300, 61, 5, 7, 20, "bf16", True, 0.3, "normal"),
    "odd_f32": (515, 257, 6, 200, 57, "f32", False, 0.1, "normal"),
    "two_groups": (130, 66, 32, 0, 66, "f32", False, 0.0, "normal"),
    "wide": (129, 600, 16, 3, 590, "bf16", False, 0.0, "normal"),
    "ten_bf16": (200, 128, 10, 0, 128, "bf16", True, 0.1, "ties"),
    "sixteen": (311, 200, 16, 40, 100, "f32", False, 0.0, "bad"),
    "sixteen_small": (140, 33, 16, 0, 33, "bf16", True, 0.0, "normal"),
    "thirty_two": (150, 300, 32, 0, 300, "bf16", True, 0.0, "few"),
    "eight_of_300": (150, 300, 8, 0, 300, "f32", True, 0.0, "bad"),
    "eight_of_400": (150, 400, 8, 0, 400, "bf16", False, 0.0, "normal"),
    "eight_of_180": (150, 180, 8, 0, 180, "f32", False, 0.0, "ties"),
    "widest": (77, 1024, 32, 0, 1024, "f32", True, 0.1, "normal"),
    "ties": (400, 48, 6, 0, 48, "bf16", True, 0.0, "ties"),
    "constant": (70, 16, 4, 2, 9, "f32", False, 0.0, "constant"),
    "bad_values": (333, 40, 6, 0, 40, "f32", False, 0.1, "bad"),
    "bad_values_bf16": (333, 40, 6, 0, 40, "bf16", True, 0.1, "bad"),
    "infinite_bf16": (257, 40, 6, 0, 40, "bf16", True, 0.0, "infinite"),
    "infinite_bf16_all": (257, 40, 6, 0, 40, "bf16", False, 0.0, "infinite"),
    "infinite_f32": (257, 40, 12, 0, 40, "f32", True, 0.0, "infinite"),
    "all_masked": (90, 12, 3, 0, 12, "f32", True, 1.0, "normal"),
    "few_left": (64, 24, 8, 4, 16, "f32", True, 0.0, "few"),
    "lowest": (64, 24, 8, 0, 24, "f32", True, 0.0, "lowest"),
    "large": (96, 32, 4, 0, 32, "f32", False, 0.0, "large"),
    "many_chunks": (40000, 5, 2, 1, 3, "f32", False, 0.1, "normal"),
    "two_chunks": (129, 20, 3, 0, 20, "f32", False, 0.0, "normal"),
}


def _inputs(name):
    T, E, K, first, local, dt, renorm, masked, kind = CASES[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    x = rng.standard_normal((T, E)) * 2
    if kind == "ties":
        x = np.round(x)
        x[::7] = np.where(rng.random((len(x[::7]), E)) < 0.5, 0.0, -0.0)
    elif kind == "constant":
        x[:] = 1.5
    elif kind == "bad":
        for v, share in ((np.nan, 0.1), (np.inf, 0.02), (-np.inf, 0.2), (-3e38, 0.1), (3e38, 0.02)):
            x[rng.random((T, E)) < share] = v
        x[5], x[6], x[7] = np.nan, -np.inf, np.inf
        x[8] = -3.3e38
    elif kind == "infinite":  # beside the largest and lowest finite values of either type
        for v in (np.inf, 3.3895314e38, np.finfo(np.float32).max, -3.3895314e38, np.finfo(np.float32).min, -np.inf):
            x[rng.random((T, E)) < 0.08] = v
    elif kind == "few":
        x[rng.random((T, E)) < 0.85] = -np.inf
    elif kind == "lowest":  # masked by the type's lowest value instead of -inf
        x[rng.random((T, E)) < 0.85] = np.finfo(np.float32).min
    elif kind == "large":
        x *= 40
    t = torch.from_numpy(x.astype(np.float32))
    t = (t.bfloat16() if dt == "bf16" else t).to(DEV)
    mask = None
    if masked:
        mask = (torch.from_numpy(rng.random(T)) >= masked).to(torch.uint8).to(DEV)
    r = lr.Router(T=T, E=E, K=K, dtype=lr.BF16 if dt == "bf16" else lr.F32, first=first, local=local, renorm=renorm,
                  scale=1.25, device=DEV)
    return r, t, mask, rng


def _host(t):
    return None if t is None else as_f64(t)


def _outs(r, fill=-7):
    i32 = lambda *s: torch.full(s, fill, dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.full(s, float(fill), device=DEV)  # noqa: E731
    return {"idx": i32(r.T, r.K), "w": f32(r.T, r.K), "counts": i32(r.E),
            "seg_off": torch.full((r.local + 1,), fill, dtype=torch.int64, device=DEV), "tok": i32(r.T * r.K),
            "slot": i32(r.T * r.K), "alpha": f32(r.T * r.K), "pmap": i32(r.T, r.K)}


def _check_route(r, o, ref):
    for k in ("idx", "counts", "seg_off", "pmap"):
        assert np.array_equal(o[k].cpu().numpy(), ref[k]), k
    N = int(ref["seg_off"][-1])
    for k in ("tok", "slot"):
        assert np.array_equal(o[k][:N].cpu().numpy(), ref[k]), k
        assert torch.all(o[k][N:] == -7), k  # rows behind the last pair are left as they were
    assert torch.all(o["alpha"][N:] == -7)
    w = as_f64(o["w"])
    assert np.all(np.abs(w - ref["w"]) <= ref["w_err"]), np.max(np.abs(w - ref["w"]) / ref["w_err"])
    t, k = np.nonzero(ref["pmap"] >= 0)
    alpha = as_f64(o["alpha"])
    assert np.array_equal(alpha[ref["pmap"][t, k]], w[t, k])


@pytest.mark.parametrize("name", sorted(CASES))
def test_route(name):
    r, x, mask, _ = _inputs(name)
    log(f"route {name}")
    ref = ro.route(_host(x), r.K, _host(mask), r.first, r.local, r.renorm, r.scale)
    o = lr.route(r, x, mask=mask, out=_outs(r))
    torch.cuda.synchronize()
    _check_route(r, o, ref)
    again = lr.route(r, x, mask=mask, out=_outs(r))
    for k in o:
        assert torch.equal(o[k], again[k]), k


@pytest.mark.parametrize("T,E,K,first,local,dt", [
    (32769, 9, 3, 2, 5, "bf16"), (33000, 9, 3, 0, 9, "f32"), (70001, 6, 2, 1, 1, "f32"), (20000, 330, 2, 5, 33, "bf16"),
    (140001, 3, 1, 0, 3, "f32"), (600007, 2, 1, 1, 1, "bf16")])
def test_route_chunk_sizes(T, E, K, first, local, dt):
    """Lengths whose chunks are no power of two (72 to 1024 tokens), with last ones that are nearly empty."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32))
    x = (x.bfloat16() if dt == "bf16" else x).to(DEV)
    mask = torch.from_numpy(rng.random(T) >= 0.2).to(DEV)
    r = lr.Router(T=T, E=E, K=K, dtype=lr.BF16 if dt == "bf16" else lr.F32, first=first, local=local, renorm=True,
                  device=DEV)
    log(f"route {T} x {E}")
    o = lr.route(r, x, mask=mask, out=_outs(r))
    torch.cuda.synchronize()
    _check_route(r, o, ro.route(_host(x), K, mask.cpu().numpy(), first, local, True, 1.0))


def test_route_no_tokens():
    r = lr.Router(T=0, E=9, K=2, first=3, local=4, device=DEV)
    log("route without tokens")
    o = lr.route(r, torch.empty(0, 9, device=DEV))
    assert o["counts"].tolist() == [0] * 9 and o["seg_off"].tolist() == [0] * 5
    b = lr.balance_loss(r, torch.empty(0, 9, device=DEV), o["idx"], seq_off=[0, 0, 0])
    assert b["loss"].item() == 0 and not b["counts"].any() and not b["psum"].any() and not b["norm"].any()
    assert lr.route_bwd(r, torch.empty(0, 9, device=DEV), o["idx"], balance=b, seq_off=[0, 0, 0]).shape == (0, 9)


def _sequences(name, T, rng):
    yield None
    yield [0, T]
    yield sorted([0, 0, T, T] + rng.integers(0, T + 1, size=9).tolist())
    if T > 3:
        yield [1, T // 2, T - 1]  # tokens before the first and behind the last sequence
        yield [2 * T // 3, 3 * T // 4, T]


@pytest.mark.parametrize("name", sorted(CASES))
def test_balance_and_gradient(name):
    r, x, mask, rng = _inputs(name)
    X, M = _host(x), _host(mask)
    idx = lr.route(r, x, mask=mask)["idx"]
    I = idx.cpu().numpy()
    dalpha = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    gloss = torch.tensor([0.7], device=DEV)
    g7 = float(np.float32(0.7))
    for off in _sequences(name, r.T, rng):
        log(f"balance {name} {None if off is None else len(off) - 1}")
        ref = ro.balance(X, I, float(np.float32(0.3)), M, off)
        b = lr.balance_loss(r, x, idx, coef=0.3, mask=mask, seq_off=off)
        again = lr.balance_loss(r, x, idx, coef=0.3, mask=mask, seq_off=off)
        assert all(torch.equal(b[k], again[k]) for k in b)
        assert np.array_equal(b["counts"].cpu().numpy(), ref["counts"])
        assert np.all(np.abs(as_f64(b["psum"]) - ref["psum"]) <= ref["psum_err"])
        assert np.all(np.abs(as_f64(b["norm"]) - ref["norm"]) <= 2 * ro.U * ref["norm"])
        assert abs(float(b["loss"]) - ref["loss"]) <= ref["loss_err"] + 1e-37
        N = as_f64(b["norm"])
        for y, bal in ((None, True), (dalpha, False), (dalpha, True)):
            got = lr.route_bwd(r, x, idx, dalpha=y, balance=b if bal else None, gloss=gloss, mask=mask, seq_off=off)
            dx, err = ro.route_bwd(X, I, y=None if y is None else as_f64(y), counts=ref["counts"],
                                   norm=N if bal else None, gloss=g7, mask=M, seq_off=off, renorm=r.renorm,
                                   scale=r.scale)
            if x.dtype == torch.bfloat16:
                err = err + np.abs(dx) * 2.0 ** -8
            d = np.abs(as_f64(got) - dx)
            assert np.all(d <= err), (off, y is None, bal, np.max(d / err))


def test_gradient_through_pair_rows():
    """dalpha by pair row: local pairs through pmap, the others and rows past the end give nothing."""
    r, x, mask, rng = _inputs("share_bf16")
    o = lr.route(r, x, mask=mask)
    n = int(o["seg_off"][-1])
    d = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DEV)
    slots = torch.where(o["pmap"] >= 0, d[o["pmap"].clamp(min=0).long()], 0.0)
    log("gradient by pair row")
    a = lr.route_bwd(r, x, o["idx"], dalpha=d, pmap=o["pmap"], mask=mask)
    b = lr.route_bwd(r, x, o["idx"], dalpha=slots, mask=mask)
    assert torch.equal(a, b)
    short = lr.route_bwd(r, x, o["idx"], dalpha=d[:n // 2].contiguous(), pmap=o["pmap"], mask=mask)
    cut = torch.where(o["pmap"] < n // 2, slots, 0.0)
    assert torch.equal(short, lr.route_bwd(r, x, o["idx"], dalpha=cut, mask=mask))


def test_indexes_outside_the_experts_are_empty_slots():
    r, x, mask, rng = _inputs("odd_f32")
    idx = lr.route(r, x, mask=mask)["idx"].clone()
    idx[::3, 2], idx[1::5, 0] = r.E, -5
    idx[4, 1] = 2 ** 31 - 1
    I = np.where((idx.cpu().numpy() < 0) | (idx.cpu().numpy() >= r.E), -1, idx.cpu().numpy())
    y = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    log("indexes outside the experts")
    b = lr.balance_loss(r, x, idx, mask=mask)
    assert np.array_equal(b["counts"].cpu().numpy(), ro.balance(_host(x), I, 1.0, _host(mask))["counts"])
    dx, err = ro.route_bwd(_host(x), I, y=as_f64(y), mask=_host(mask), scale=r.scale)
    assert np.all(np.abs(as_f64(lr.route_bwd(r, x, idx, dalpha=y, mask=mask)) - dx) <= err)


def test_offsets_outside_the_tokens_are_clamped():
    r, x, _, _ = _inputs("odd_f32")
    idx = lr.route(r, x)["idx"]
    log("device offsets outside [0, T]")
    wild = torch.tensor([-9, 100, 10 ** 12], device=DEV)
    a = lr.balance_loss(r, x, idx, seq_off=wild)
    b = lr.balance_loss(r, x, idx, seq_off=[0, 100, r.T])
    assert all(torch.equal(a[k], b[k]) for k in a)
    with pytest.raises(ValueError):
        lr.balance_loss(r, x, idx, seq_off=[0, 10 ** 12])
    with pytest.raises(ValueError):
        lr.balance_loss(r, x, idx, seq_off=[0, 9, 3, r.T])


def test_gradients_add_over_the_expert_shares():
    """Each GPU's pairs give a part of the routing gradient; the parts add up to the whole."""
    _, x, _, rng = _inputs("share")
    T, E, K = 1111, 128, 8
    whole = lr.Router(T=T, E=E, K=K, renorm=True, device=DEV)
    o = lr.route(whole, x)
    y = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(DEV)
    parts = np.zeros((T, E))
    log("expert shares")
    for first in range(0, E, 32):
        r = lr.Router(T=T, E=E, K=K, renorm=True, first=first, local=32, device=DEV)
        p = lr.route(r, x)
        n = int(p["seg_off"][-1])
        row = p["pmap"].long()
        d = torch.zeros(n, device=DEV)
        d[row[row >= 0]] = y[row >= 0]
        parts += as_f64(lr.route_bwd(r, x, p["idx"], dalpha=d, pmap=p["pmap"]))
    X, I = _host(x), o["idx"].cpu().numpy()
    dx, err = ro.route_bwd(X, I, y=as_f64(y), renorm=True)
    bound = sum(ro.route_bwd(X, I, y=np.where((I >= f) & (I < f + 32), as_f64(y), 0), renorm=True)[1]
                for f in range(0, E, 32))
    assert np.all(np.abs(parts - dx) <= bound)


@pytest.mark.parametrize("T,K,D,dt,keep", [(1, 1, 8, "f32", None), (37, 3, 8, "bf16", 0.5), (200, 8, 520, "bf16", None),
                                           (90, 10, 2048, "f32", 0.6), (65, 4, 4104, "bf16", 0.9),
                                           (130, 17, 264, "f32", None), (700, 2, 1032, "bf16", 0.0)])
def test_alpha_grad(T, K, D, dt, keep):
    rng = np.random.default_rng(T + D)
    E = K + 3
    x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    r = lr.Router(T=T, E=E, K=K, first=1, local=E - 1, device=DEV)
    o = lr.route(r, x)
    seg = o["seg_off"].cpu().numpy()
    N = int(seg[-1])
    p = lr.Problem(E=E - 1, T=T, K=K, D=D, F=8, swiglu=True, dtype=lr.BF16 if dt == "bf16" else lr.F32, seg_off=seg,
                   quota=np.zeros(E - 1, np.int32), device=DEV)
    td = torch.bfloat16 if dt == "bf16" else torch.float32
    G = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).to(DEV).to(td)
    Y = torch.from_numpy(rng.standard_normal((max(N, 1), D)).astype(np.float32)).to(DEV).to(td)
    alpha = o["alpha"].clone()
    alpha[:N][::5] = 0
    k = None if keep is None else torch.from_numpy((rng.random(max(N, 1)) < keep).astype(np.uint8)).to(DEV)
    log(f"alpha gradient T={T} K={K} D={D} {dt}")
    out = torch.full((N + 3,), -7.0, device=DEV)
    lr.alpha_grad(p, G, Y, alpha, o["pmap"], keep=k, out=out)
    ref, err = ro.alpha_grad(as_f64(G), as_f64(Y)[:N], as_f64(alpha)[:N], o["tok"][:N].cpu().numpy(),
                             None if k is None else k.cpu().numpy()[:N])
    assert np.all(np.abs(as_f64(out[:N]) - ref) <= err + 1e-37)
    assert torch.all(out[N:] == -7)


@pytest.mark.parametrize("T,K,D,dt", [(1024, 2, 24, "f32"), (1025, 2, 24, "f32"), (1030, 9, 1024, "f32"),
                                      (1030, 17, 2056, "bf16"), (8192, 1, 2048, "bf16"), (8193, 1, 2048, "bf16")])
def test_alpha_grad_of_few_and_many_tokens(T, K, D, dt):
    """On both sides of the sizes up to which a block shares a token's columns, more than eight slots among
    them."""
    test_alpha_grad(T, K, D, dt, 0.7)


def test_alpha_grad_leaves_pairs_without_a_position():
    p = lr.Problem(E=1, T=2, K=2, D=8, F=8, swiglu=True, dtype=lr.F32, seg_off=[0, 4], quota=[4], device=DEV)
    one = torch.ones(4, 8, device=DEV)
    out = torch.full((4,), -7.0, device=DEV)
    pmap = torch.tensor([[3, -1], [4, 1]], dtype=torch.int32, device=DEV)  # 4 is past the last pair
    log("pairs without a position")
    lr.alpha_grad(p, one[:2], one, torch.full((4,), 0.5, device=DEV), pmap, out=out)
    assert out.tolist() == [-7.0, 16.0, -7.0, 16.0]


def test_python_checks():
    r, x, mask, _ = _inputs("share")
    idx = lr.route(r, x)["idx"]
    b = lr.balance_loss(r, x, idx)
    for call in (lambda: lr.route(r, x.bfloat16()), lambda: lr.route(r, x[:-1]), lambda: lr.route(r, x.t()),
                 lambda: lr.route(r, x.cpu()), lambda: lr.route(r, x, mask=torch.ones(3, dtype=torch.uint8, device=DEV)), lambda: lr.route(r, x, mask=torch.ones(r.T, dtype=torch.uint8)),
                 lambda: lr.route(r, x, mask=torch.ones(r.T, device=DEV)),
                 lambda: lr.route(r, x, out={"idx": idx.long()}), lambda: lr.route(r, x, out={"tok": idx}),
                 lambda: lr.balance_loss(r, x, idx[:5]), lambda: lr.balance_loss(r, x, idx.float()),
                 lambda: lr.balance_loss(r, x, idx, seq_off=[0]), lambda: lr.balance_loss(r, x, idx, out={"loss": x}),
                 lambda: lr.route_bwd(r, x, idx, dalpha=b["psum"]), lambda: lr.route_bwd(r, x, idx, dalpha=x.double()),
                 lambda: lr.route_bwd(r, x, idx, balance=b, seq_off=[0, 4, 9]),
                 lambda: lr.route_bwd(r, x, idx, balance=b, gloss=torch.ones((), device=DEV)),
                 lambda: lr.route_bwd(r, x, idx, balance=b, out=x),
                 lambda: lr.route_bwd(r, x, idx, balance=b, out=x.bfloat16())):
        with pytest.raises(ValueError):
            call()


def test_replayed_graph_and_other_stream():
    """Routing, loss and gradient captured on a side stream: every replay on new logits equals the eager
    calls, with eager work of another Router between the replays."""
    r, x, mask, rng = _inputs("share_bf16")
    off = torch.tensor([0, 400, 400, 900, r.T], device=DEV)
    y = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)

    def step(rt):
        o = lr.route(rt, x, mask=mask)
        b = lr.balance_loss(rt, x, o["idx"], mask=mask, seq_off=off)
        return {**o, **b, "dx": lr.route_bwd(rt, x, o["idx"], dalpha=y, balance=b, mask=mask, seq_off=off)}

    eager = lr.Router(T=r.T, E=r.E, K=r.K, dtype=r.dtype, first=r.first, local=r.local, scale=r.scale, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(r)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = step(r)
    for rep in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)).to(DEV))
        for t in got.values():
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step(eager)
        n = int(want["seg_off"][-1])
        log(f"replay {rep}: {n} pairs")
        for k in want:
            a, b = (t[k][:n] if k in ("tok", "slot", "alpha") else t[k] for t in (got, want))
            assert torch.equal(a, b), (rep, k)


def test_side_stream_argument():
    """Calls on a stream that is not the current one, outputs allocated by them: the logits are written there
    just before, so a call on the current stream would not see them."""
    r, x, mask, rng = _inputs("share")
    want = lr.route(r, x)
    wb = lr.balance_loss(r, x, want["idx"], seq_off=[0, 100, r.T])
    wg = lr.route_bwd(r, x, want["idx"], balance=wb, seq_off=[0, 100, r.T])
    side = torch.cuda.Stream()
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    big = torch.zeros(1 << 28, device=DEV)
    log("side stream")
    with torch.cuda.stream(side):
        for _ in range(4):
            big.add_(1.0)
        late.copy_(x)
    o = lr.route(r, late, stream=side)
    b = lr.balance_loss(r, late, o["idx"], seq_off=[0, 100, r.T], stream=side)
    g = lr.route_bwd(r, late, o["idx"], balance=b, seq_off=[0, 100, r.T], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in ("idx", "w", "counts", "seg_off", "tok", "alpha", "pmap"):
        assert torch.equal(o[k], want[k]), k
    assert torch.equal(b["loss"], wb["loss"]) and torch.equal(b["psum"], wb["psum"]) and torch.equal(g, wg)


def test_a_grown_workspace_leaves_a_captured_graph():
    """A graph captured with one sequence keeps its workspace when a later call with many needs a larger one."""
    r, x, mask, rng = _inputs("share")
    idx = lr.route(r, x)["idx"]
    want = lr.balance_loss(r, x, idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lr.balance_loss(r, x, idx)
    log("workspace grows")
    lr.balance_loss(r, x, idx, seq_off=list(range(r.T + 1)))
    trash = [torch.full((r.workspace_size(1),), 99, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert all(bool(torch.all(t == 99)) for t in trash)


def test_wide_local_share_with_many_slots():
    """Bits and pairs of a placing block that do not fit its LDS together: the pairs are stored directly."""
    T, E, K = 70001, 1024, 16
    x = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    r = lr.Router(T=T, E=E, K=K, dtype=lr.BF16, device=DEV)
    log("wide local share")
    o = lr.route(r, x)
    top, order = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(o["idx"].long(), order[:, :K])
    flat = o["idx"].reshape(-1).long()
    by = torch.argsort(flat, stable=True)
    assert torch.equal(o["tok"].long(), by // K) and torch.equal(o["slot"].long(), by % K)
    assert torch.equal(o["alpha"], o["w"].reshape(-1)[by])
    assert torch.equal(o["counts"].long(), torch.bincount(flat, minlength=E))
    back = torch.empty_like(by)
    back[by] = torch.arange(T * K, device=DEV)
    assert torch.equal(o["pmap"].reshape(-1).long(), back)


@pytest.mark.parametrize("E", [6, 24, 60, 100])
@pytest.mark.parametrize("off", [None, [0, 30000, 30001, 100000]])
def test_balance_of_long_sequences(off, E):
    """Tiles of more than one pass: counts and sums against torch in fp64."""
    T, K = 100003, 3
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, E, generator=gen, device=DEV)
    mask = (torch.rand(T, generator=gen, device=DEV) < 0.7).to(torch.uint8)
    r = lr.Router(T=T, E=E, K=K, device=DEV)
    idx = lr.route(r, x, mask=mask)["idx"]
    log("long sequences")
    b = lr.balance_loss(r, x, idx, coef=0.5, mask=mask, seq_off=off)
    again = lr.balance_loss(r, x, idx, coef=0.5, mask=mask, seq_off=off)
    assert all(torch.equal(b[k], again[k]) for k in b)
    p, on = torch.softmax(x.double(), 1), mask.bool()
    ends = [0, T] if off is None else off
    loss, S = 0.0, len(ends) - 1
    for s, (lo, hi) in enumerate(zip(ends, ends[1:])):
        rows = on[lo:hi]
        want = p[lo:hi][rows].sum(0)
        count = torch.bincount(idx[lo:hi][rows].reshape(-1).long(), minlength=E)
        assert torch.equal(b["counts"][s].long(), count)
        # each p to 60 x 2^-24 (|x - max| is under 12), 128 sums of a lane and 80 over lanes in fp32,
        # at the most: fewer of a lane with four or eight lanes to a token
        assert torch.all((b["psum"][s].double() - want).abs() <= want * 270 * 2.0 ** -24)
        n = int(rows.sum())
        if n:
            loss += 0.5 * E / (K * n * n) * float((count.double() * want).sum()) / sum(
                int(on[a:c].sum()) > 0 for a, c in zip(ends, ends[1:]))
    assert abs(float(b["loss"]) - loss) <= 280 * 2.0 ** -24 * loss


def test_workspace_freed_while_a_side_stream_uses_it():
    """A router that is gone while a call of it waits on a side stream: its workspace, allocated on the current
    stream, is not given out before that call is done."""
    r = lr.Router(T=9000, E=64, K=4, dtype=lr.BF16)
    x = torch.randn(r.T, r.E, device=DEV).bfloat16()
    want = lr.route(r, x)
    n, at = r.workspace().numel(), r.workspace().data_ptr()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    log("a call behind a wait on the side stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # well over the host's time for what follows
    got = lr.route(r, x, stream=side)
    del r
    trash = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(50)]
    assert not side.query(), "the side stream ended before the buffers were asked for"
    assert at not in {t.data_ptr() for t in trash}
    torch.cuda.synchronize()
    pairs = int(want["seg_off"][-1])
    for name in want:
        a, b = (o[name][:pairs] if name in ("tok", "slot", "alpha") else o[name] for o in (got, want))
        assert torch.equal(a, b), name


@pytest.mark.parametrize("E,S,masked", [(9, 64, 0.2), (9, 65, 0.2), (130, 22, 0.0), (130, 700, 0.3), (64, 3000, 0.9),
                                        (20, 100, 1.0)])
def test_balance_of_many_sequences(E, S, masked):
    """On both sides of the number of sequences whose loss has a launch of its own, empty and long ones
    among them."""
    rng = np.random.default_rng(E + S)
    T, K = 6001, 3
    x = torch.from_numpy((rng.standard_normal((T, E)) * 2).astype(np.float32)).to(DEV)
    mask = torch.from_numpy(rng.random(T) >= masked).to(DEV)
    off = np.sort(np.concatenate([[0], rng.integers(0, T // 3, size=S - 1), [T]])).tolist()
    r = lr.Router(T=T, E=E, K=K, device=DEV)
    idx = lr.route(r, x, mask=mask)["idx"]
    log(f"{S} sequences of {E} experts")
    b = lr.balance_loss(r, x, idx, coef=0.3, mask=mask, seq_off=off)
    again = lr.balance_loss(r, x, idx, coef=0.3, mask=mask, seq_off=off)
    assert all(torch.equal(b[k], again[k]) for k in b)
    M = mask.cpu().numpy()
    ref = ro.balance(_host(x), idx.cpu().numpy(), float(np.float32(0.3)), M, off)
    assert np.array_equal(b["counts"].cpu().numpy(), ref["counts"])
    assert np.all(np.abs(as_f64(b["psum"]) - ref["psum"]) <= ref["psum_err"])
    assert np.all(np.abs(as_f64(b["norm"]) - ref["norm"]) <= 2 * ro.U * ref["norm"])
    assert abs(float(b["loss"]) - ref["loss"]) <= ref["loss_err"] + 1e-37
    dx, err = ro.route_bwd(_host(x), idx.cpu().numpy(), counts=ref["counts"], norm=as_f64(b["norm"]), mask=M,
                           seq_off=off)
    got = lr.route_bwd(r, x, idx, balance=b, mask=mask, seq_off=off)
    assert np.all(np.abs(as_f64(got) - dx) <= err)


@pytest.mark.parametrize("E,dt", [(17, "f32"), (61, "bf16"), (130, "f32"), (257, "bf16"), (601, "f32")])
def test_logits_from_a_later_row(E, dt):
    """Logits and their gradient as views that start at rows 1 to 3 of a buffer: as a copy of them gives."""
    rng = np.random.default_rng(E)
    T, K = 400, 3
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    whole = torch.from_numpy((rng.standard_normal((T + 3, E)) * 2).astype(np.float32)).to(DEV).to(t)
    r = lr.Router(T=T, E=E, K=K, dtype=lr.BF16 if dt == "bf16" else lr.F32, device=DEV)
    y = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(DEV)
    for row in (1, 2, 3):
        x = whole[row:row + T]
        log(f"logits of {E} {dt} from row {row}")
        got, want = [], []
        grad = torch.full((T + 6, E), 5.0, dtype=t, device=DEV)
        for to, logits, out in ((got, x, grad[row:row + T]), (want, x.clone(), None)):
            o = lr.route(r, logits)
            b = lr.balance_loss(r, logits, o["idx"])
            to += [*o.values(), *b.values(), lr.route_bwd(r, logits, o["idx"], dalpha=y, balance=b, out=out)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.all(grad[:row] == 5.0) and torch.all(grad[row + T:] == 5.0)


def test_a_workspace_outgrown_while_a_side_stream_uses_it():
    """A call that waits on a side stream keeps its workspace when a call on the current stream needs a larger
    one; afterwards the smaller one is given back."""
    r = lr.Router(T=9000, E=64, K=4, dtype=lr.BF16, device=DEV)
    x = torch.randn(r.T, r.E, device=DEV).bfloat16()
    want = lr.route(r, x)
    n = r.workspace().numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    log("a call behind a wait on the side stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = lr.route(r, x, stream=side)
    lr.balance_loss(r, x, want["idx"], seq_off=list(range(r.T + 1)))
    assert r.workspace().numel() > n and r._grown == []
    trash = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(50)]
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert all(bool(torch.all(t == 255)) for t in trash)
