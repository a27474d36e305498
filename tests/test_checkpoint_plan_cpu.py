"""Quota admission where the backward restores X from a checkpoint: its rows count, whatever the quotas."""
import numpy as np
import pytest

import load_recalibrated_expert_amd as lr

T, K, D, F, SEG = 300, 2, 64, 32, [0, 250, 400, 600]
RHOS = ["1", "0.5", "0.1"]


def _plan(avail, dtype=lr.BF16, **kw):
    return lr.plan_quotas(3, T, K, D, F, True, dtype, SEG, RHOS, avail, **kw)


@pytest.mark.parametrize("dtype,size", [(lr.BF16, 2), (lr.F32, 4)])
def test_restored_rows_are_counted(dtype, size):
    rows, most = T * D * size, 1 << 40
    i, q, b = _plan(most, dtype)
    assert _plan(most, dtype, restored_x=True) == (i, pytest.approx(q), b + rows)
    p = lr.Problem(E=3, T=T, K=K, D=D, F=F, swiglu=True, dtype=dtype, seg_off=SEG, quota=q, device="cpu")
    assert lr.backward_bytes(p, restored_x=True) == lr.backward_bytes(p) + rows == b + rows
    # a budget that the restored rows do not fit beside the buffers admits a lower ratio
    assert _plan(b, dtype)[0] == 0
    j, q2, b2 = _plan(b + rows - 1, dtype, restored_x=True)
    assert j > 0 and b2 <= b + rows - 1 and np.all(q2 < q)
    assert _plan(b + rows, dtype, restored_x=True)[0] == 0


def test_nothing_fits_beside_the_restored_rows():
    rows = T * D * 2
    for avail in (0, rows - 1, rows, rows + 1):
        with pytest.raises(lr.InfeasibleQuotaError):
            _plan(avail, restored_x=True)
