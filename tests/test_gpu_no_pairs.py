"""A layer without pairs has no saved rows: its backward needs none and gives zero gradients."""
import pytest
import torch

import load_recalibrated_expert_amd as lr

from gpu_util import DEV, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("mode", [lr.COMPACT_PHYSICAL, lr.COMPACT_ZERO_MASKED])
@pytest.mark.parametrize("swiglu", [True, False])
def test_backward_without_saved_rows(swiglu, mode, packed):
    T, D, F = 30, 64, 40
    bf = lambda *d: torch.ones(*d, device=DEV).bfloat16()  # noqa: E731
    p = lr.Problem(E=2, T=T, K=2, D=D, F=F, swiglu=swiglu, dtype=lr.BF16, seg_off=[0, 0, 0], quota=[0, 0], device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    log(f"no pairs, swiglu {swiglu}, mode {mode}, packed {packed}")
    kw = dict(X=bf(T, D), W1=bf(2, D, 2 * F)) if swiglu else {}
    r = lr.backward(p, G=bf(T, D), Phi=None, H=None, alpha=one.float(), tok=one, slot=one, W2=bf(2, F, D), mode=mode,
                    packed_dlt=packed, **kw)
    torch.cuda.synchronize()
    assert not r["dW2"].any() and not r["out"][:T].any() and (not swiglu or not r["dW1"].any())
