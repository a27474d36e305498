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
