"""A backward call needs what its forward call left in the workspace: without one it is refused (no GPU needed, the check
comes before those of the tensors)."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece


@pytest.mark.parametrize("n", [0, 10])
def test_attention_backward_refuses_no_workspace(n):
    op = rece.SequenceAttention(n, 2, 4, 32)
    t, offs = torch.zeros(n, 4, 32, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace"):
        op.backward(t, t, t, offs, t, None, t)


def test_log_probabilities_backward_refuses_no_workspace():
    op = rece.LogProb(10, 50, 64)
    X, Y = torch.zeros(10, 64, dtype=torch.bfloat16), torch.zeros(50, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        op.backward(X, Y, torch.zeros(10, dtype=torch.int32), None, torch.zeros(10))
