"""The backward from checkpoints of [gate | up] and of X holds no more than the estimate of quota admission."""
import gc

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
import synth

from gpu_util import Staged, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [0, 4000])
def test_backward_from_checkpoints_fits_its_estimate(more):
    """``more``: rows that X's checkpoint has behind the T tokens', which are not restored."""
    cfg = synth.custom("plan_codes", T=12000, K=2, E=3, D=1024, F=256, counts=(9000, 8000, 5000), seed=43)
    pr = synth.make_problem(cfg, rho="0.5")
    s = Staged(pr)
    H = lr.checkpoint(s.H, parts=2)
    rows = s.X if not more else torch.cat([s.X, torch.full((more, cfg.D), float("nan"), dtype=s.X.dtype, device=s.X.device)])
    X8 = lr.checkpoint(rows)
    del rows
    est = lr.backward_bytes(s.P, restored_x=True)
    torch.cuda.synchronize()
    gc.collect()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    # bytes asked for: the allocator adds up to 1 MiB to a large block (here 540672 to dIn and 589824 to X's rows, whose
    # segments of whole 2 MiB it does not split)
    base = torch.cuda.memory_stats()["requested_bytes.all.current"]
    log(f"backward from checkpoints, estimate {est}, of it {cfg.T * cfg.D * 2} for X")
    res = lr.backward(s.P, G=s.G, H=H, X=X8, alpha=s.alpha, tok=s.tok, slot=s.slot, W2=s.W2, W1=s.W1)
    torch.cuda.synchronize()
    grown = torch.cuda.memory_stats()["requested_bytes.all.peak"] - base
    log(f"the backward asked for {grown} bytes")
    assert 0.99 * est <= grown <= est
    assert res["sel"].numel() == int(np.sum(pr.quota)) and bool(torch.isfinite(res["dW1"]).all())
