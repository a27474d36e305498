"""The binding of activation checkpoints without a GPU: calls that it refuses, or lets through, before the library is called."""
import pytest
import torch

import load_recalibrated_expert_amd as lr

from test_router_binding_cpu import Tensor, gpu  # noqa: F401


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
