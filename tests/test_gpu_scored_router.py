"""GPU parity of routing by scores against the fp64 definitions (oracle/scored_oracle.py, which also gives each
value's error bound in fp32 arithmetic): choices, weights and pair lists, the balance loss of sigmoid scores, both
gradients and the bias update."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import scored_oracle as so

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu

# T, E, K, first, local, dtype, score, bias, groups, top, best, renorm, mask share, what the logits hold
CASES = {
    "one_token": (1, 128, 8, 0, 128, "f32", "sigmoid", "steps", 1, 1, 1, True, 0.0, "normal"),
    "one_token_groups": (1, 160, 6, 40, 21, "bf16", "sigmoid", "steps", 8, 3, 2, False, 0.0, "normal"),
    "one_expert": (37, 1, 1, 0, 1, "f32", "sigmoid", "normal", 1, 1, 2, True, 0.0, "normal"),
    "all_chosen": (50, 7, 7, 0, 7, "f32", "sigmoid", "normal", 1, 1, 1, True, 0.0, "normal"),
    "share": (1111, 128, 8, 0, 128, "f32", "sigmoid", "steps", 1, 1, 1, True, 0.0, "normal"),
    "share_bf16": (1111, 128, 8, 16, 16, "bf16", "sigmoid", "steps", 1, 1, 1, False, 0.2, "normal"),
    "by_logit": (500, 61, 5, 7, 20, "bf16", "sigmoid", None, 1, 1, 1, True, 0.3, "ties"),
    "by_logit_f32": (500, 61, 5, 7, 20, "f32", "sigmoid", None, 1, 1, 1, False, 0.1, "large"),
    "softmax_bias": (515, 257, 6, 200, 57, "f32", "softmax", "normal", 1, 1, 1, False, 0.1, "normal"),
    "softmax_bias_renorm": (515, 40, 6, 0, 40, "bf16", "softmax", "steps", 1, 1, 1, True, 0.1, "normal"),
    "softmax_groups": (300, 64, 6, 0, 64, "f32", "softmax", None, 8, 3, 1, False, 0.1, "normal"),
    "groups": (700, 160, 6, 40, 21, "bf16", "sigmoid", "steps", 8, 3, 2, False, 0.15, "normal"),
    "groups_f32": (700, 256, 8, 0, 256, "f32", "sigmoid", "normal", 8, 4, 2, True, 0.0, "normal"),
    "groups_of_one": (130, 16, 4, 0, 16, "f32", "sigmoid", "normal", 16, 5, 2, True, 0.0, "normal"),
    "groups_all_kept": (130, 24, 4, 0, 24, "f32", "sigmoid", None, 4, 4, 2, True, 0.0, "ties"),
    "most_groups": (99, 128, 10, 0, 128, "bf16", "sigmoid", None, 64, 9, 2, True, 0.1, "normal"),
    "odd_groups": (333, 105, 3, 1, 99, "f32", "sigmoid", "normal", 5, 1, 2, False, 0.0, "bad"),
    "few_in_groups": (200, 48, 6, 0, 48, "f32", "sigmoid", "normal", 6, 2, 2, True, 0.1, "few"),
    "group_ties": (300, 60, 5, 0, 60, "bf16", "sigmoid", None, 6, 2, 2, True, 0.0, "ties"),
    "constant": (70, 16, 4, 2, 9, "f32", "sigmoid", "steps", 4, 2, 2, False, 0.0, "constant"),
    "constant_negative": (70, 16, 4, 2, 9, "f32", "sigmoid", "below", 4, 2, 2, False, 0.0, "constant"),
    "negative_scores": (300, 40, 6, 0, 40, "f32", "sigmoid", "below", 1, 1, 1, True, 0.0, "normal"),
    "bad_bias": (300, 40, 6, 0, 40, "f32", "sigmoid", "bad", 1, 1, 1, True, 0.0, "normal"),
    "bad_bias_groups": (300, 40, 6, 0, 40, "bf16", "softmax", "bad", 5, 2, 2, True, 0.0, "normal"),
    "bad_values": (333, 40, 6, 0, 40, "f32", "sigmoid", "normal", 1, 1, 1, False, 0.1, "bad"),
    "bad_values_bf16": (333, 40, 6, 0, 40, "bf16", "sigmoid", "normal", 8, 4, 1, True, 0.1, "bad"),
    "all_masked": (90, 12, 3, 0, 12, "f32", "sigmoid", "normal", 3, 2, 2, True, 1.0, "normal"),
    "lowest": (64, 24, 8, 0, 24, "f32", "sigmoid", "normal", 1, 1, 1, True, 0.0, "lowest"),
    "deep": (96, 32, 4, 0, 32, "f32", "sigmoid", None, 1, 1, 1, True, 0.0, "deep"),
    "large": (96, 32, 4, 0, 32, "f32", "sigmoid", None, 4, 2, 2, False, 0.0, "large"),
    "sixteen": (311, 200, 16, 40, 100, "f32", "sigmoid", "normal", 1, 1, 1, False, 0.0, "bad"),
    "sixteen_groups": (140, 330, 16, 0, 33, "bf16", "sigmoid", "normal", 11, 4, 2, True, 0.0, "normal"),
    "eight_of_300": (150, 300, 8, 0, 300, "f32", "sigmoid", "normal", 1, 1, 1, True, 0.0, "normal"),
    "eight_of_380": (150, 380, 8, 0, 380, "f32", "sigmoid", "normal", 4, 2, 2, True, 0.0, "normal"),
    "eight_of_500": (150, 500, 8, 0, 500, "bf16", "sigmoid", "normal", 4, 3, 1, True, 0.0, "normal"),
    "eight_of_180": (150, 180, 8, 0, 180, "f32", "sigmoid", "normal", 1, 1, 1, True, 0.0, "normal"),
    "eight_of_600": (150, 600, 8, 0, 600, "f32", "softmax", "normal", 1, 1, 1, True, 0.0, "normal"),
    "thirty_two": (150, 300, 32, 0, 300, "bf16", "sigmoid", "normal", 3, 2, 2, True, 0.0, "normal"),
    "widest": (77, 1024, 32, 0, 1024, "f32", "sigmoid", "normal", 1, 1, 1, True, 0.1, "normal"),
    "widest_groups": (77, 1024, 32, 0, 1024, "f32", "sigmoid", "normal", 64, 5, 2, True, 0.1, "normal"),
    "widest_few": (200, 1024, 8, 3, 590, "bf16", "sigmoid", "normal", 4, 2, 2, True, 0.1, "normal"),
    "widest_sixteen": (40, 1000, 12, 0, 1000, "f32", "sigmoid", "normal", 10, 2, 1, False, 0.1, "normal"),
    "many_chunks": (40000, 5, 2, 1, 3, "f32", "sigmoid", "normal", 1, 1, 1, False, 0.1, "normal"),
    "many_chunks_groups": (33001, 6, 2, 1, 3, "bf16", "sigmoid", "normal", 3, 1, 2, False, 0.1, "normal"),
}


def _inputs(name):
    T, E, K, first, local, dt, score, bias, groups, top, best, renorm, masked, kind = CASES[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    x = rng.standard_normal((T, E)) * 2
    if kind == "ties":
        x = np.round(x)
        x[::7] = np.where(rng.random((len(x[::7]), E)) < 0.5, 0.0, -0.0)
    elif kind == "constant":
        x[:] = 1.5
    elif kind == "bad":
        for v, share in ((np.nan, 0.1), (np.inf, 0.02), (-np.inf, 0.2), (-3e38, 0.05)):
            x[rng.random((T, E)) < share] = v
        x[5], x[6], x[7] = np.nan, -np.inf, np.inf
        x[8] = -3.3e38
    elif kind == "few":
        x[rng.random((T, E)) < 0.85] = -np.inf
    elif kind == "lowest":  # masked by the type's lowest value instead of -inf
        x[rng.random((T, E)) < 0.85] = np.finfo(np.float32).min
    elif kind == "deep":  # all scores far below the smallest f32
        x = x * 30 - 900
    elif kind == "large":  # to both ends of what a score in f32 can tell apart
        x *= 15
    t = torch.from_numpy(x.astype(np.float32))
    t = (t.bfloat16() if dt == "bf16" else t).to(DEV)
    mask = None
    if masked:
        mask = (torch.from_numpy(rng.random(T)) >= masked).to(torch.uint8).to(DEV)
    b = {None: None, "normal": rng.standard_normal(E) * 0.2, "steps": np.round(rng.standard_normal(E) * 4) * 1e-3,
         "below": np.full(E, -3.0), "bad": np.where(rng.random(E) < 0.3, rng.choice([np.nan, -np.inf, np.inf], E), 0.1)}[bias]
    b = None if b is None else torch.from_numpy(b.astype(np.float32)).to(DEV)
    r = lr.Router(T=T, E=E, K=K, dtype=lr.BF16 if dt == "bf16" else lr.F32, first=first, local=local, renorm=renorm,
                  scale=1.25, score=score, groups=groups, top_groups=top, group_best=best, device=DEV)
    return r, t, b, mask, rng


def _host(t):
    return None if t is None else as_f64(t)


def _outs(r, fill=-7):
    i32 = lambda *s: torch.full(s, fill, dtype=torch.int32, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.full(s, float(fill), device=DEV)  # noqa: E731
    return {"idx": i32(r.T, r.K), "w": f32(r.T, r.K), "counts": i32(r.E),
            "seg_off": torch.full((r.local + 1,), fill, dtype=torch.int64, device=DEV), "tok": i32(r.T * r.K),
            "slot": i32(r.T * r.K), "alpha": f32(r.T * r.K), "pmap": i32(r.T, r.K)}


def _reference(r, x, b, mask, o):
    # group sums of scores that differ by less than 2^-41 come from logits over 28 here ("large"): exp(-28) = 7e-13
    return so.route(_host(x), r.K, r.score, _host(b), r.groups, r.top_groups, r.group_best, _host(mask), r.first, r.local,
                    r.renorm, r.scale, given=o["idx"].cpu().numpy())


def _check(r, o, ref):
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
    assert np.array_equal(as_f64(o["alpha"])[ref["pmap"][t, k]], w[t, k])


@pytest.mark.parametrize("name", sorted(CASES))
def test_route(name):
    r, x, b, mask, _ = _inputs(name)
    log(f"scored route {name}")
    o = lr.route(r, x, mask=mask, bias=b, out=_outs(r))
    torch.cuda.synchronize()
    _check(r, o, _reference(r, x, b, mask, o))
    again = lr.route(r, x, mask=mask, bias=b, out=_outs(r))
    for k in o:
        assert torch.equal(o[k], again[k]), k


def _sequences(T, rng):
    yield None
    yield sorted([0, 0, T, T] + rng.integers(0, T + 1, size=9).tolist())
    if T > 3:
        yield [1, T // 2, T - 1]  # tokens before the first and behind the last sequence


SIGMOID = sorted(n for n in CASES if CASES[n][6] == "sigmoid")


@pytest.mark.parametrize("name", SIGMOID)
def test_balance_and_gradient(name):
    r, x, b, mask, rng = _inputs(name)
    X, M = _host(x), _host(mask)
    idx = lr.route(r, x, mask=mask, bias=b)["idx"]
    I = idx.cpu().numpy()
    dalpha = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    gloss = torch.tensor([0.7], device=DEV)
    for off in _sequences(r.T, rng):
        log(f"scored balance {name} {None if off is None else len(off) - 1}")
        ref = so.balance(X, I, float(np.float32(0.3)), "sigmoid", M, off)
        bal = lr.balance_loss(r, x, idx, coef=0.3, mask=mask, seq_off=off)
        assert np.array_equal(bal["counts"].cpu().numpy(), ref["counts"])
        assert np.all(np.abs(as_f64(bal["psum"]) - ref["psum"]) <= ref["psum_err"])
        assert np.all(np.abs(as_f64(bal["norm"]) - ref["norm"]) <= 2 * so.U * ref["norm"])
        assert abs(float(bal["loss"]) - ref["loss"]) <= ref["loss_err"] + 1e-37
        N = as_f64(bal["norm"])
        for y, on in ((None, True), (dalpha, False), (dalpha, True)):
            got = lr.route_bwd(r, x, idx, dalpha=y, balance=bal if on else None, gloss=gloss, mask=mask, seq_off=off)
            dx, err = so.sigmoid_bwd(X, I, y=None if y is None else as_f64(y), counts=ref["counts"],
                                     norm=N if on else None, gloss=float(np.float32(0.7)), mask=M, seq_off=off,
                                     renorm=r.renorm, scale=r.scale)
            if x.dtype == torch.bfloat16:
                err = err + np.abs(dx) * 2.0 ** -8
            d = np.abs(as_f64(got) - dx)
            assert np.all(d <= err), (off, y is None, on, np.max(d / err))


def test_softmax_gradient_with_bias_is_the_plain_one():
    r, x, b, mask, rng = _inputs("softmax_bias_renorm")
    o = lr.route(r, x, mask=mask, bias=b)
    plain = lr.Router(T=r.T, E=r.E, K=r.K, dtype=r.dtype, renorm=True, scale=1.25, device=DEV)
    grouped = lr.Router(T=r.T, E=r.E, K=r.K, dtype=r.dtype, renorm=True, scale=1.25, groups=4, top_groups=2, device=DEV)
    y = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    log("softmax gradient")
    assert torch.equal(lr.route_bwd(plain, x, o["idx"], dalpha=y, mask=mask),
                       lr.route_bwd(grouped, x, o["idx"], dalpha=y, mask=mask))
    a, b2 = lr.balance_loss(plain, x, o["idx"], mask=mask), lr.balance_loss(grouped, x, o["idx"], mask=mask)
    assert all(torch.equal(a[k], b2[k]) for k in a)


def test_gradient_through_pair_rows():
    r, x, b, mask, rng = _inputs("share_bf16")
    o = lr.route(r, x, mask=mask, bias=b)
    n = int(o["seg_off"][-1])
    d = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DEV)
    slots = torch.where(o["pmap"] >= 0, d[o["pmap"].clamp(min=0).long()], 0.0)
    log("scored gradient by pair row")
    assert torch.equal(lr.route_bwd(r, x, o["idx"], dalpha=d, pmap=o["pmap"], mask=mask),
                       lr.route_bwd(r, x, o["idx"], dalpha=slots, mask=mask))


def test_indexes_outside_the_experts_are_empty_slots():
    r, x, b, mask, rng = _inputs("all_chosen")
    idx = lr.route(r, x, bias=b)["idx"].clone()
    idx[::3, 2], idx[1::5, 0], idx[4, 1] = r.E, -5, 2 ** 31 - 1
    I = np.where((idx.cpu().numpy() < 0) | (idx.cpu().numpy() >= r.E), -1, idx.cpu().numpy())
    y = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    log("scored gradient, indexes outside the experts")
    dx, err = so.sigmoid_bwd(_host(x), I, y=as_f64(y), renorm=True, scale=r.scale)
    assert np.all(np.abs(as_f64(lr.route_bwd(r, x, idx, dalpha=y)) - dx) <= err)


def test_near_scores_are_told_apart():
    """Scores that agree to 2^-30, which f32 scores could not order."""
    E, T = 64, 50
    rng = np.random.default_rng(5)
    x = np.full((T, E), 0.75, np.float32)
    place = np.argsort(rng.random((T, E)), axis=1)
    x += (place * 2.0 ** -24).astype(np.float32) * 8  # a step of x is 2^-24 here; scores differ by 2^-23
    bias = np.zeros(E, np.float32)
    bias[::2] = np.float32(2.0 ** -40)
    r = lr.Router(T=T, E=E, K=8, score="sigmoid", device=DEV)
    log("near scores")
    o = lr.route(r, torch.from_numpy(x).to(DEV), bias=torch.from_numpy(bias).to(DEV))
    ref = so.route(x, 8, "sigmoid", bias=bias)
    assert np.array_equal(o["idx"].cpu().numpy(), ref["idx"])


def test_route_no_tokens():
    r = lr.Router(T=0, E=9, K=2, first=3, local=4, score="sigmoid", device=DEV)
    log("scored route without tokens")
    empty = torch.empty(0, 9, device=DEV)
    o = lr.route(r, empty, bias=torch.zeros(9, device=DEV))
    assert o["counts"].tolist() == [0] * 9 and o["seg_off"].tolist() == [0] * 5
    b = lr.balance_loss(r, empty, o["idx"], seq_off=[0, 0, 0])
    assert b["loss"].item() == 0 and not b["counts"].any() and not b["psum"].any() and not b["norm"].any()
    assert lr.route_bwd(r, empty, o["idx"], balance=b, seq_off=[0, 0, 0]).shape == (0, 9)


@pytest.mark.parametrize("T,E,K,score", [(600007, 96, 1, "softmax"), (600007, 96, 1, "sigmoid"), (66001, 128, 3, "sigmoid"),
                                         (24000, 128, 2, "sigmoid"), (49999, 130, 2, "softmax")])
def test_many_rows_of_counts(T, E, K, score):
    """Numbers of chunks on both sides of what the placing blocks sum themselves, and more than a scan keeps in registers.
    The lists against stable sorts by torch."""
    x = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T))
    r = lr.Router(T=T, E=E, K=K, first=1, local=E - 2, score=score, device=DEV)
    log(f"pair lists of {T} x {E}")
    o = lr.route(r, x)
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :K].contiguous()
    assert torch.equal(o["idx"].long(), idx) and torch.equal(o["counts"].long(), torch.bincount(idx.view(-1), minlength=E))
    e = idx.reshape(-1) - 1
    here = (e >= 0) & (e < E - 2)
    order = torch.argsort(torch.where(here, e, E), stable=True)[:int(here.sum())]
    n = len(order)
    assert torch.equal(o["seg_off"][1:], torch.cumsum(o["counts"][1:-1].long(), 0)) and int(o["seg_off"][-1]) == n
    assert torch.equal(o["tok"][:n].long(), order // K) and torch.equal(o["slot"][:n].long(), order % K)
    assert torch.equal(o["alpha"][:n], o["w"].view(-1)[order])
    row = torch.full((T * K,), -1, device=DEV)
    row[order] = torch.arange(n, device=DEV)
    assert torch.equal(o["pmap"].view(-1).long(), row)


@pytest.mark.parametrize("E", [1, 3, 64, 65, 1024])
def test_bias_update(E):
    rng = np.random.default_rng(E)
    r = lr.Router(T=4, E=E, K=1, score="sigmoid", device=DEV)
    log(f"bias update of {E}")
    for high in (3, 2 ** 31 - 1):  # sums past 32 bits
        counts = rng.integers(0, high, E, endpoint=True).astype(np.int32)
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        b, c = torch.from_numpy(bias).to(DEV), torch.from_numpy(counts).to(DEV)
        ref = so.bias_update(bias, counts, 1e-3)
        assert np.array_equal(lr.bias_update(r, b, c, 1e-3).cpu().numpy(), ref)
        assert np.array_equal(b.cpu().numpy(), bias)
        assert lr.bias_update(r, b, c, 1e-3, out=b) is b and np.array_equal(b.cpu().numpy(), ref)


def test_captured_step_replays():
    """Routing, loss, gradients and the bias update in place as one graph: each replay is the next step."""
    r, x, b, mask, rng = _inputs("groups")
    y = torch.from_numpy(rng.standard_normal((r.T, r.K)).astype(np.float32)).to(DEV)
    start = b.clone()

    def step():
        o = lr.route(r, x, mask=mask, bias=b)
        bal = lr.balance_loss(r, x, o["idx"], coef=0.1, mask=mask)
        g = lr.route_bwd(r, x, o["idx"], dalpha=y, balance=bal, mask=mask)
        lr.bias_update(r, b, o["counts"], 0.05, out=b)
        return o["idx"], o["w"], bal["loss"], g, b

    eager = []
    for _ in range(4):
        eager.append([t.clone() for t in step()])
    b.copy_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    b.copy_(start)
    for i in range(4):
        log(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, eager[i]):
            assert torch.equal(a, e)
        lr.route(lr.Router(T=r.T, E=r.E, K=2, dtype=r.dtype, device=DEV), x)  # eager work between the replays


def test_on_another_stream():
    r, x, b, mask, _ = _inputs("share")
    ref = lr.route(r, x, bias=b)
    s = torch.cuda.Stream()
    log("scored route on a stream")
    r2 = lr.Router(T=r.T, E=r.E, K=r.K, renorm=True, scale=1.25, score="sigmoid", device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    o = lr.route(r2, x, bias=b, stream=s)
    n = lr.bias_update(r2, b, o["counts"], 1e-3, stream=s)
    s.synchronize()
    N = int(ref["seg_off"][-1])
    for k in o:
        cut = slice(0, N) if k in ("tok", "slot", "alpha") else slice(None)
        assert torch.equal(o[k][cut], ref[k][cut]), k
    assert torch.equal(n, lr.bias_update(r, b, ref["counts"], 1e-3))
