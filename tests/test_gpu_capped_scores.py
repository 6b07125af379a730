"""Capped scores: the same call gives the same bits whatever ran before it."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from test_gpu_attend_masked import run, tensors

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def fill_shared_memory(value):
    """A projection whose tiles leave `value` in the shared memory of every SM."""
    x = torch.full((1, 1, 148 * 256, 512), value, device="cuda", dtype=BF)
    w = torch.full((256, 512), value, device="cuda", dtype=BF)
    y = torch.empty(1, 1, 148 * 256, 256, device="cuda", dtype=BF)
    prm = spr.make_project(x, w, y)
    spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm))
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hk,Nk", [(1, 4, 1, 500), (1, 8, 2, 5000), (3, 12, 4, 200), (20, 6, 2, 900),
                                         (200, 4, 2, 900)])
@pytest.mark.parametrize("slopes", [False, True])
def test_bits_do_not_depend_on_left_over_shared_memory(Nq, Hq, Hk, Nk, d, slopes):
    """Few query tokens and shared key heads: a tile's rows behind the packed ones hold anything."""
    Q, K, V = tensors(2, Hq, Hk, Nq, Nk, d, BF, seed=50)
    kw = dict(softcap=30.0, causal=True)
    if slopes:
        kw["slopes"] = torch.linspace(0, 0.2, Hq, device="cuda")
    got = []
    for value in (0.0, 1e4, 0.0, -3e18, 1.0):
        fill_shared_memory(value)
        got.append(run(Q, K, V, **kw))
    for O, L in got[1:]:
        assert torch.equal(O, got[0][0]) and torch.equal(L, got[0][1])
