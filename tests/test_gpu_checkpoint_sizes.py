"""Activation checkpoints of more groups than one launch takes."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import checkpoint_oracle as co

from gpu_util import DEV, as_f64, log

pytestmark = pytest.mark.gpu


def test_more_groups_than_a_launch_takes():
    """2^29 + 4000 groups: the second launch begins inside a row. Values on both sides of its first group and at the end."""
    n, parts, width = (2 ** 29 + 4000) // 7, 7, 8
    seam = (2 ** 29 - 32) // parts
    x = torch.zeros(n, parts * width, dtype=torch.bfloat16, device=DEV)
    places = (slice(0, 50), slice(seam - 50, seam + 50), slice(n - 20, n))
    rng = np.random.default_rng(8)
    for at in places:
        v = rng.standard_normal((at.stop - at.start, parts * width)) * np.exp(rng.standard_normal((at.stop - at.start, 1)) * 5)
        x[at] = torch.from_numpy(v.astype(np.float32)).to(DEV).bfloat16()
    given = [x[at].clone() for at in places]
    log(f"codes of {n * parts} groups")
    c = lr.checkpoint(x, parts=parts)
    torch.cuda.synchronize()
    log("and back")
    lr.restore(c, out=x)
    torch.cuda.synchronize()
    for at, rows in zip(places, given):
        q, s = co.checkpoint(as_f64(rows), parts)
        assert np.array_equal(c.q[at].cpu().numpy(), q) and np.array_equal(as_f64(c.scale[at]), s)
        back = torch.from_numpy(co.values(q, s).astype(np.float32)).bfloat16()
        assert torch.equal(x[at].cpu(), back)
    for a, b in ((50, seam - 50), (seam + 50, n - 20)):  # the rest is zeros: codes 0 and the smallest scale
        assert not c.q[a:b].any() and not x[a:b].any()
        assert torch.all(c.scale[a:b] == 2.0 ** -126)
