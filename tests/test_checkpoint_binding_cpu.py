"""The binding of activation checkpoints without a GPU: calls that it refuses, or lets through, before the library is called."""
import types

import pytest
import torch

import load_recalibrated_expert_amd as lr
from load_recalibrated_expert_amd import _lib

from test_router_binding_cpu import Tensor, gpu  # noqa: F401


class Rows(Tensor):
    """Of which a call gives the first rows back."""

    def __getitem__(self, rows):
        return self


@pytest.mark.parametrize("parts,width", [(1, 2 ** 31), (1, 2 ** 32 + 8), (2, 2 ** 32 + 8), (2 ** 16, 8), (2 ** 32 + 1, 8)])
def test_columns_that_32_bits_do_not_count(gpu, parts, width):  # noqa: F811
    """Cut to 32 bits the call would be one of fewer columns."""
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        lr.checkpoint(Tensor((1, parts * width), bf, 0), parts=parts)
    with pytest.raises(ValueError):
        c = lr.Checkpoint(Tensor((1, parts * width), torch.int8, 0), Tensor((1, parts, -(-width // 128)), bf, 0))
        lr.restore(c)
    assert gpu.lib.launched == []


@pytest.mark.parametrize("parts,width", [(1, 8), (1, 2 ** 31 - 8), (2 ** 16 - 1, 8)])
def test_most_columns(gpu, parts, width):  # noqa: F811
    lr.checkpoint(Tensor((1, parts * width), torch.bfloat16, 0), parts=parts)
    lr.restore(lr.Checkpoint(Tensor((1, parts * width), torch.int8, 0), Tensor((1, parts, -(-width // 128)), torch.bfloat16, 0)))
    assert gpu.lib.launched == ["lrmoe_checkpoint", "lrmoe_restore"]


@pytest.mark.parametrize("device", [0, 1, -1])
def test_a_problem_of_another_device(gpu, device, monkeypatch):  # noqa: F811
    """Its offsets, workspace and outputs are there, not on the device that the kernels run on."""
    bf, f32 = torch.bfloat16, torch.float32
    monkeypatch.setattr(lr, "_gemm_outputs", lambda p, rows, out: out)  # it allocates
    where = "cpu" if device < 0 else f"cuda:{device}"
    p = types.SimpleNamespace(N=9, T=8, K=2, D=8, F=32, K_tot=5, E=2, swiglu=True, torch_dtype=bf, device=where,
                              c=_lib.CProblem(), workspace=lambda mode=0: Tensor((512,), torch.uint8, device),
                              seg_off_d=Tensor((3,), torch.int64, device), cseg_off_d=Tensor((3,), torch.int64, device))
    H = lr.Checkpoint(Tensor((9, 64), torch.int8, 0), Tensor((9, 2, 1), bf, 0))
    t, o = Tensor((9,), f32, 0), Rows((9, 8), bf, 0)
    calls = (lambda: lr.score_checkpoint(p, t, H, t, t, R=t), lambda: lr.compact_checkpoint(p, t, H, t, out=o),
             lambda: lr.grouped_gemm_bwd_checkpoint(p, t, t, t, t, t, t, t, H, t, out=dict(dW2=o, dW1=o, dH=o, dIn=o)),
             lambda: lr.expert_forward_checkpoint(p, t, t, t, t, t, out=dict(H=lr.Checkpoint(
                 Rows((9, 64), torch.int8, 0), Rows((9, 2, 1), bf, 0)), Phi=o, Y=o)))
    for call in calls:
        if device == 0:
            call()
        else:
            with pytest.raises(ValueError):
                call()
    assert len(gpu.lib.launched) == (4 if device == 0 else 0)
