"""The position of AttentionBlock's first token, on the CPU."""
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build


def test_first_position():
    """0 without a cache, whatever k_len a call gives; behind the cached tokens with one."""
    spr_build.build()
    w, wo = torch.zeros(3 * 128, 64, dtype=torch.bfloat16), torch.zeros(64, 128, dtype=torch.bfloat16)
    for causal in (False, True):
        assert spr.AttentionBlock((2, 10, 64), 2, 64, w, wo, causal=causal)._attend.q_start == 0
    assert spr.AttentionBlock((2, 10, 64), 2, 64, w, wo, cache=20)._attend.q_start == -2 ** 31
