"""Refusals of the token operators that need no GPU."""
import ctypes
import os
import shutil

import pytest
import torch

import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api

FAKE = 0x7F0000000000
needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="no CUDA toolkit")


@pytest.mark.parametrize("stream", [None, 0, "side"])
def test_distill_wrapper_takes_no_stream(stream):
    """Its backward pass would not wait for a stream of its own."""
    leaf = torch.zeros((2, 8), requires_grad=True)
    ids, lq = torch.zeros((2, 1), dtype=torch.int64), torch.zeros((2, 1))
    with pytest.raises(ValueError, match="must not name stream"):
        torch_api.FusedTopkDistill.apply(leaf, ids, lq, None, dict(stream=stream))


@needs_nvcc
@pytest.mark.parametrize("R", [(1 << 28) + 1, (1 << 31) - 1])
def test_more_masked_rows_than_the_waits_allow_for(R):
    """Looking through so many rows' mask could outlast a bounded wait."""
    rl.build()
    lib = rl.load()
    assert lib.rl_token_logprobs(FAKE, rl.RL_BF16, R, 8, 8, None, 0, FAKE + (1 << 42), 1.0, 0, None, FAKE + (2 << 42), None, None,
                                 None, None, None) == rl.RL_ERR_SHAPE
    d = rl.rl_topk_distill_desc_init()
    d.logits, d.R, d.V, d.ld, d.K = FAKE, R, 8, 8, 1
    d.teacher_ids, d.teacher_logp, d.mask = FAKE + (1 << 42), FAKE + (2 << 42), FAKE + (3 << 42)
    d.stats_dev, d.workspace, d.workspace_bytes = FAKE + (4 << 42), FAKE + (5 << 42), rl.rl_topk_distill_workspace_size()
    assert lib.rl_topk_distill_fwd_bwd(ctypes.byref(d), None) == rl.RL_ERR_SHAPE
