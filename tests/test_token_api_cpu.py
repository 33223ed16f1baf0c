"""Refusals of the torch layer of the token operators that need no GPU."""
import pytest
import torch

from ppo_policy_loss_gb300 import torch_api


@pytest.mark.parametrize("stream", [None, 0, "side"])
def test_distill_wrapper_takes_no_stream(stream):
    """Its backward pass would not wait for a stream of its own."""
    leaf = torch.zeros((2, 8), requires_grad=True)
    ids, lq = torch.zeros((2, 1), dtype=torch.int64), torch.zeros((2, 1))
    with pytest.raises(ValueError, match="must not name stream"):
        torch_api.FusedTopkDistill.apply(leaf, ids, lq, None, dict(stream=stream))
