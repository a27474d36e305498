"""The router's gradients and weights at the ends of their range, against fp64: counts that are large and
nearly equal, products that f32 cannot hold, logits far below the largest."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import router_oracle as ro

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu

DTYPES = {"f32": (torch.float32, lr.F32), "bf16": (torch.bfloat16, lr.BF16)}


def _logits(rng, T, E, dt, std=2.0):
    return torch.from_numpy((rng.standard_normal((T, E)) * std).astype(np.float32)).to(DEV).to(DTYPES[dt][0])


@pytest.mark.parametrize("spread", [0, 1, 360, "one"])
@pytest.mark.parametrize("E,dt", [(1, "f32"), (2, "f32"), (5, "bf16"), (16, "f32"), (31, "f32"), (64, "f32"), (128, "f32"),
                                  (128, "bf16"), (257, "f32"), (600, "bf16"), (1024, "f32")])
def test_balance_gradient_of_nearly_equal_counts(E, dt, spread):
    """The gradient is that of the counts' differences: sum_e p_e = 1, so what all counts have in common has
    no part in it, nor in its error. The bound takes the counts relative to that of the token's most
    probable expert: each p (rel), conversion, product, a sum of up to 32 of a lane and six over
    lanes, difference, factor and last rounding are under rel + 48 half steps of both terms."""
    rng = np.random.default_rng(E + (7 if spread == "one" else spread))
    T = 301
    x = _logits(rng, T, E, dt)
    mask = torch.from_numpy(rng.random(T) >= 0.1).to(DEV)
    off = [0, 100, 100, 250, T]
    base = np.array([1 << 16, 1, 5_000_011, (1 << 30) + 12345])[:, None]
    if spread == "one":  # one expert's count stands out
        c = np.repeat(base, E, 1)
        c[:, E // 2] += 1 << 20
    else:
        c = base + rng.integers(-spread, spread + 1, size=(4, E))
    c = np.maximum(c, 0)
    norm = (1.0 / base[:, 0]).astype(np.float32)
    bal = {"counts": torch.from_numpy(c.astype(np.int32)).to(DEV), "norm": torch.from_numpy(norm).to(DEV)}
    r = lr.Router(T=T, E=E, K=1, dtype=DTYPES[dt][1], device=DEV)
    idx = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    gloss = torch.tensor([0.75], device=DEV)
    log(f"balance gradient of {E} {dt}, spread {spread}")
    got = as_f64(lr.route_bwd(r, x, idx, balance=bal, gloss=gloss, mask=mask, seq_off=off))
    p, rel = ro.softmax(ro.clean(as_f64(x), mask.cpu().numpy()))
    top = p.argmax(1)
    seq = np.searchsorted(off, np.arange(T), side="right") - 1
    d = (c[seq] - c[seq, top][:, None]).astype(np.float64)
    dot = (p * d).sum(1, keepdims=True)
    f = 0.75 * norm.astype(np.float64)[seq][:, None]
    want = f * p * (d - dot)
    pr = rel + 48 * ro.U
    err = f * p * (np.abs(d) * pr + (p * np.abs(d) * pr).sum(1, keepdims=True) + np.abs(dot) * pr) + 1e-37
    if dt == "bf16":
        err = err + np.abs(want) * 2.0 ** -8
    live = mask.cpu().numpy()
    assert np.all(got[~live] == 0)
    worst = float(np.max((np.abs(got - want) / err)[live]))
    assert worst <= 1


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("g,y,a", [(1e-7, 1e-36, 1e-36), (1e-25, 1e-20, 1e-20), (1e-30, 1e-30, 1e-38), (1e25, 1e20, 1e20),
                                   (1e30, 1e-38, 1e-38), (1e-39, 1e-3, 1e-3), (1.0, 1e-39, 1e-39), (1e30, 1e30, 3e38)])
@pytest.mark.parametrize("T,D", [(5, 264), (1100, 64)])
def test_alpha_grad_products_that_f32_does_not_hold(T, D, g, y, a, dt):
    """G, Y and alpha of ordinary and subnormal values whose products vanish in f32 or pass its largest value,
    and whose quotients do neither. The bound is the definition's for products and sums in fp64, the f32
    result's own rounding below 2^-126 added."""
    rng = np.random.default_rng(T + D)
    K = 3
    N = T * K
    td, code = DTYPES[dt]
    G = torch.from_numpy((rng.standard_normal((T, D)) * g).astype(np.float32)).to(DEV).to(td)
    Y = torch.from_numpy((rng.standard_normal((N, D)) * y).astype(np.float32)).to(DEV).to(td)
    alpha = torch.from_numpy(((rng.random(N) * 0.5 + 0.5) * a).astype(np.float32)).to(DEV)
    pmap = torch.from_numpy(rng.permutation(N).astype(np.int32).reshape(T, K)).to(DEV)
    p = lr.Problem(E=1, T=T, K=K, D=D, F=8, swiglu=True, dtype=code, seg_off=[0, N], quota=[0], device=DEV)
    log(f"alpha gradient T={T} {dt} G {g:g} Y {y:g} alpha {a:g}")
    got = as_f64(lr.alpha_grad(p, G, Y, alpha, pmap))
    tok = np.empty(N, np.int64)
    tok[pmap.cpu().numpy().reshape(-1)] = np.repeat(np.arange(T), K)
    want, err = ro.alpha_grad(as_f64(G), as_f64(Y), as_f64(alpha), tok)
    worst = float(np.max(np.abs(got - want) / (err + 2.0 ** -149)))
    assert worst <= 1 and np.abs(want).max() > 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 8, 3), (50, 16, 4), (333, 60, 8), (200, 128, 8), (40, 300, 16), (33, 1024, 32),
                                   (5000, 24, 4)])
@pytest.mark.parametrize("least", [80, 92])
def test_chosen_logits_far_below_the_largest(least, T, E, K, renorm, dt):
    """Chosen experts 80 to 104 below the maximum: weights from 2^-115 to the smallest subnormal number, and
    their share of the logits' gradient. The bounds are the definition's; below 2^-126 the exponential,
    the quotient and the product with scale are each off by up to half of 2^-149 more. What is not
    chosen counts as 0 below 2^-126, so scale * sum_k p_k y_k reaches a slot within that."""
    rng = np.random.default_rng(T + E)
    td, code = DTYPES[dt]
    x = -least - (104 - least) * rng.random((T, E))
    x[np.arange(T), rng.integers(0, E, T)] = rng.standard_normal(T)
    x = torch.from_numpy(x.astype(np.float32)).to(DEV).to(td)
    r = lr.Router(T=T, E=E, K=K, dtype=code, renorm=renorm, scale=1.5, device=DEV)
    log(f"route {T} x {E} {dt} with far logits")
    ref = ro.route(as_f64(x), K, renorm=renorm, scale=1.5)
    o = lr.route(r, x)
    assert np.array_equal(o["idx"].cpu().numpy(), ref["idx"])
    w, tiny = as_f64(o["w"]), 2.0 ** -149
    rel = (ref["w_err"] - 1e-37) / ref["w"]
    worst = float(np.max(np.abs(w - ref["w"]) / (ref["w"] * rel + 3 * tiny)))
    assert worst <= 1
    assert np.all(w[ref["w"] > 4 * tiny] > 0)
    y = torch.from_numpy((rng.standard_normal((T, K)) * 1e30).astype(np.float32)).to(DEV)
    y[:, 0] *= 1e-30  # the largest's is ordinary, so that the others' part is seen
    got = as_f64(lr.route_bwd(r, x, o["idx"], dalpha=y))
    want, err = ro.route_bwd(as_f64(x), ref["idx"], y=as_f64(y), renorm=renorm, scale=1.5)
    d = np.zeros((T, E))
    np.put_along_axis(d, ref["idx"], np.abs(1.5 * as_f64(y)), 1)
    # q to 2 tiny at each slot and in the sum; the sum times what counts as 0
    err = err + 2 * tiny * d + ref_p(as_f64(x), ref["idx"], renorm) * 2 * tiny * d.sum(1, keepdims=True)
    err = err + 2.0 ** -126 * np.abs(ref_sum(as_f64(x), ref["idx"], as_f64(y), renorm))
    if dt == "bf16":
        err = err + np.abs(want) * 2.0 ** -8
    worst = float(np.max(np.abs(got - want) / err))
    assert worst <= 1


def ref_p(x, idx, renorm):
    """fp64 softmax over all experts, or over the chosen ones."""
    if renorm:
        chosen = np.zeros(x.shape, bool)
        np.put_along_axis(chosen, idx, True, 1)
        x = np.where(chosen, x, -np.inf)
    return ro.softmax(x)[0]


def ref_sum(x, idx, y, renorm):
    return 1.5 * (np.take_along_axis(ref_p(x, idx, renorm), idx, 1) * y).sum(1, keepdims=True)
