"""The balance gradient of sigmoid scores with counts that are large, nearly equal or far apart, and scores of any size, against
fp64."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import router_oracle as ro
from oracle import scored_oracle as so

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu

DTYPES = {"f32": (torch.float32, lr.F32), "bf16": (torch.bfloat16, lr.BF16)}


def _logits(rng, kind, T, E):
    x = rng.standard_normal((T, E)) * 2
    if kind == "low":  # 1 - s is 1 in f32 for all of them
        x = x - 40
    elif kind == "lowest":
        x = x * 10 - 500
    elif kind == "one_leads":  # the probability of one expert is nearly 1, however low its score is
        x = x - rng.uniform(30, 50, (T, 1))
        x[np.arange(T), rng.integers(0, E, T)] = rng.uniform(-22, -17, T)
    elif kind == "one_leads_high":
        x = x - rng.uniform(10, 20, (T, 1))
        x[np.arange(T), rng.integers(0, E, T)] = rng.uniform(-8, 3, T)
    return x.astype(np.float32)


@pytest.mark.parametrize("kind", ["normal", "low", "lowest", "one_leads", "one_leads_high"])
@pytest.mark.parametrize("counts", ["equal", "near", "apart"])
@pytest.mark.parametrize("E,dt", [(1, "f32"), (2, "f32"), (5, "bf16"), (16, "f32"), (31, "f32"), (64, "f32"), (128, "f32"),
                                  (128, "bf16"), (257, "f32"), (600, "bf16"), (1024, "f32")])
def test_balance_gradient_is_of_the_counts_differences(E, dt, counts, kind):
    """sum_e p_e = 1, so what all counts have in common has no part in the gradient, nor in its error. The bound takes the
    counts relative to that of the token's most probable expert: each p (rel), the factor 1 - s (12 half steps), conversion,
    products, a sum of up to 32 of a lane and six over lanes, difference and last rounding are under rel + 60 half steps of both
    terms. A p below 2^-126 counts as 0, so p may be off by that much: f 2^-126 |d - dot| of its own gradient, and
    f p 2^-126 |d| of dot's."""
    rng = np.random.default_rng(E + 3 * len(kind) + 5 * len(counts))
    T = 301
    x = torch.from_numpy(_logits(rng, kind, T, E)).to(DEV).to(DTYPES[dt][0])
    mask = torch.from_numpy(rng.random(T) >= 0.1).to(DEV)
    off = [0, 100, 100, 250, T]
    base = np.array([1 << 17, 1, 5_000_011, (1 << 30) + 12345])[:, None]
    c = {"equal": np.repeat(base, E, 1), "near": base + rng.integers(-1, 2, (4, E)),
         "apart": rng.integers(0, 200_001, (4, E))}[counts]
    norm = (1.0 / base[:, 0]).astype(np.float32)
    bal = {"counts": torch.from_numpy(c.astype(np.int32)).to(DEV), "norm": torch.from_numpy(norm).to(DEV)}
    r = lr.Router(T=T, E=E, K=1, dtype=DTYPES[dt][1], score="sigmoid", device=DEV)
    idx = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    gloss = torch.tensor([0.75], device=DEV)
    log(f"sigmoid balance gradient of {E} {dt}, counts {counts}, logits {kind}")
    got = as_f64(lr.route_bwd(r, x, idx, balance=bal, gloss=gloss, mask=mask, seq_off=off))
    live = mask.cpu().numpy()
    X = ro.clean(as_f64(x), live)
    p, rel = so.shares(X, "sigmoid")
    away = np.where(X > -np.inf, so.sigmoid(-X), 0.0)
    top = p.argmax(1)
    seq = np.searchsorted(off, np.arange(T), side="right") - 1
    d = (c[seq] - c[seq, top][:, None]).astype(np.float64)
    dot = (p * d).sum(1, keepdims=True)
    f = 0.75 * norm.astype(np.float64)[seq][:, None] * away
    want = f * p * (d - dot)
    pr = rel + 60 * ro.U
    err = f * p * (np.abs(d) * pr + (p * np.abs(d) * pr).sum(1, keepdims=True) + np.abs(dot) * pr) + 1e-37
    err = err + f * 2.0 ** -126 * (np.abs(d - dot) + p * np.abs(d).sum(1, keepdims=True))
    if dt == "bf16":
        err = err + np.abs(want) * 2.0 ** -8
    assert np.all(got[~live] == 0)
    worst = float(np.max((np.abs(got - want) / err)[live]))
    assert worst <= 1


@pytest.mark.parametrize("shift", [1, 63, 64, 65, 500])
@pytest.mark.parametrize("ahead", [True, False])
def test_bias_update_into_a_part_of_the_bias(ahead, shift):
    """``out`` and ``bias`` as two rows of one buffer that share elements: every bias is read before any is written."""
    E = 1024
    rng = np.random.default_rng(shift)
    buf = (rng.standard_normal(E + shift) * 0.1).astype(np.float32)
    counts = rng.integers(0, 50, E).astype(np.int32)
    t = torch.from_numpy(buf).to(DEV)
    low, high = t[:E], t[shift:shift + E]
    out, bias = (high, low) if ahead else (low, high)
    ref = so.bias_update(bias.cpu().numpy(), counts, 1e-3)
    r = lr.Router(T=4, E=E, K=1, score="sigmoid", device=DEV)
    log(f"bias update, {shift} apart")
    assert np.array_equal(lr.bias_update(r, bias, torch.from_numpy(counts).to(DEV), 1e-3, out=out).cpu().numpy(), ref)
