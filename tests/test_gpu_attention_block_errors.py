"""Errors that AttentionBlock's calls meet on the device are kept until they are asked for."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from synthetic import workload
from test_gpu_attention_block import randn, tables, weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("cache", [0, 40])
@pytest.mark.parametrize("row", [-1, 30, 1 << 30])
def test_position_outside_the_tables(cache, row):
    """Also when good calls follow; and one good call gives what it gives without positions."""
    B, N, C, heads, d = 2, 10, 128, 2, 64
    W, (cos, sin) = weights(heads, heads, d, C, BF), tables(30, d)
    block = spr.AttentionBlock((B, N, C), heads, d, cache=cache, **W)
    x = randn((B, N, C), BF, 20)
    good = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1)
    bad = good.clone()
    bad[1, 7] = row
    want = block(x, cos, sin)
    block.check()
    assert torch.equal(block(x, cos, sin, positions=good), want)
    block.check()
    block(x, cos, sin, positions=bad)
    block(x, cos, sin, positions=good)
    out = block(x, cos, sin)
    assert block.status.tolist() == [1, 1, 7, row]
    with pytest.raises(spr.SparsePRError, match=f"position {row} of token 7, batch 1") as e:
        block.check()
    assert e.value.status == 5
    block.check()  # told once
    assert torch.equal(out, want)


def test_captured_positions():
    """A replayed graph keeps the error of the positions that it finds."""
    B, N, C, heads, d = 1, 4, 128, 2, 64
    W, (cos, sin) = weights(heads, heads, d, C, BF), tables(30, d)
    block = spr.AttentionBlock((B, N, C), heads, d, **W)
    x = randn((B, N, C), BF, 21)
    pos = torch.arange(N, device="cuda", dtype=torch.int32).repeat(B, 1)
    out = torch.empty_like(x)
    block(x, cos, sin, positions=pos, out=out)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(x, cos, sin, positions=pos, out=out)
    pos[0, 2] = 99
    g.replay()
    pos[0, 2] = 2
    g.replay()
    with pytest.raises(spr.SparsePRError, match="position 99 of token 2"):
        block.check()
    g.replay()
    block.check()
    assert torch.equal(out, want)


def test_a_wait_that_gave_up_is_told():
    """The word that a kernel writes then, written by hand."""
    W, (cos, sin) = weights(2, 2, 64, 128, BF), tables(10, 64)
    block = spr.AttentionBlock((1, 10, 128), 2, 64, **W)
    x = randn((1, 10, 128), BF, 22)
    block.ws[:4].view(torch.int32)[0] = 4
    block(x, cos, sin)
    with pytest.raises(spr.SparsePRError, match="gave up"):
        block.check()
    block.check()


def test_sparse_block():
    wl = workload("tiny")
    kw = dict(Ms=wl.Ms, p=wl.p, Gk=wl.Gk, Gq=wl.Gq, iters=wl.iters, seed=wl.index,
              route_mode=wl.route_mode, tau=wl.tau, M=wl.M, r=wl.r, lam=wl.lam)
    W, (cos, sin) = weights(wl.H, wl.H, wl.d, 128, BF), tables(wl.N, wl.d)
    block = spr.AttentionBlock((1, wl.N, 128), wl.H, wl.d, sparse=kw, **W)
    block.check()
    block(randn((1, wl.N, 128), BF, 23), cos, sin)
    block.check()
