"""What a workspace may be: elements one after the other, or its size says nothing."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build

BF = torch.bfloat16


def calls(dev):
    q = torch.zeros(2, 4, 10, 64, device=dev, dtype=BF)
    x, w = torch.zeros(2, 1, 10, 64, device=dev, dtype=BF), torch.zeros(64, 64, device=dev, dtype=BF)
    am, pj = spr.make_masked(q, q, q, torch.empty_like(q)), spr.make_project(x, w, torch.empty_like(x))
    o, y = torch.empty_like(q), torch.empty_like(x)
    return [(am, lambda ws: spr.sparsepr_attend_masked(am, q, q, q, o, ws)),
            (pj, lambda ws: spr.sparsepr_project(pj, x, w, y, ws))]


@pytest.mark.parametrize("dev", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_workspaces_that_are_less_than_they_say(dev):
    """One byte expanded, every other byte, no tensor at all."""
    spr_build.build()
    for prm, call in calls(dev):
        ws = spr.alloc_workspace(prm, device=dev)
        big = torch.empty(2 * ws.numel() + 512, device=dev, dtype=torch.uint8)
        off = -big.data_ptr() % 256
        for bad in (ws[:1].expand(1 << 30), big[off:off + 2 * ws.numel():2], None, 5):
            with pytest.raises(ValueError, match="^ws must be"):
                call(bad)
        with pytest.raises((ValueError, RuntimeError)):
            call(ws.to_sparse())


@pytest.mark.gpu
def test_workspaces_of_any_type():
    for prm, call in calls("cuda"):
        n = spr.alloc_workspace(prm).numel()
        call(torch.empty(-(-n // 4), device="cuda"))
        call(torch.empty(-(-n // 64), 16, device="cuda", dtype=torch.int32))
    torch.cuda.synchronize()
