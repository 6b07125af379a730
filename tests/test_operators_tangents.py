"""Forward only: a forward-mode tangent is refused, not silently cut off."""
import pytest
import torch
from torch.autograd import forward_ad

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build

BF = torch.bfloat16


def calls(dev):
    """Each operator as a function of one of its inputs, with that input."""
    q = torch.zeros(2, 4, 10, 64, device=dev, dtype=BF)
    x, w = torch.zeros(2, 1, 10, 64, device=dev, dtype=BF), torch.zeros(64, 64, device=dev, dtype=BF)
    o, y = torch.empty_like(q), torch.empty_like(x)
    am, nr, pj = spr.make_masked(q, q, q, o), spr.make_norm_rotate(q, None, o, None, rot=0), \
        spr.make_project(x, w, y)
    wa, wp = spr.alloc_workspace(am, device=dev), spr.alloc_workspace(pj, device=dev)
    return [(q, lambda t: spr.sparsepr_attend_masked(am, q, t, q, o, wa)),
            (q, lambda t: spr.sparsepr_norm_rotate(nr, t, None, o, None)),
            (w, lambda t: spr.sparsepr_project(pj, x, t, y, wp)),
            (w[0].contiguous(), lambda t: spr.sparsepr_project(pj, x, w, y, wp, bias=t))]


def refused(dev):
    for t, call in calls(dev):
        with forward_ad.dual_level():
            dual = forward_ad.make_dual(t, torch.ones_like(t))
            with pytest.raises(ValueError, match="tangent"):
                call(dual)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                call(dual)


def test_tangents_are_refused():
    spr_build.build()
    refused("cpu")


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu():
    """Also where the extension module would make the call; without a tangent it is made."""
    refused("cuda")
    for t, call in calls("cuda"):
        with forward_ad.dual_level():
            call(t)
        with pytest.raises((ValueError, RuntimeError)):
            torch.func.jvp(lambda u: call(u) or u, (t,), (torch.ones_like(t),))
    torch.cuda.synchronize()
