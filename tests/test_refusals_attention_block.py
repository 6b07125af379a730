"""What AttentionBlock refuses, on the CPU."""
import copy
import pickle

import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    spr_build.build()


def weights(heads, kv, d, C, dtype=BF):
    return torch.zeros((heads + 2 * kv) * d, C, dtype=dtype), torch.zeros(C, heads * d, dtype=dtype)


def test_construction():
    w, wo = weights(4, 4, 64, 128)
    sparse = dict(Ms=16, p=4, Gk=4, Gq=4)
    for kw in (dict(sparse=sparse, causal=True), dict(sparse=sparse, softcap=5.0),
               dict(sparse=sparse, cache=64), dict(sparse=sparse, slopes=torch.ones(4)),
               dict(sparse=sparse, kv_heads=2), dict(cache=5), dict(kv_heads=2),
               dict(pairing="both")):
        with pytest.raises(ValueError):
            spr.AttentionBlock((2, 10, 128), 4, 64, w, wo, **kw)
    with pytest.raises(ValueError):
        spr.AttentionBlock((2, 10, 128), 4, 64, w, wo[:, :192])
    cached = spr.AttentionBlock((2, 10, 128), 4, 64, w, wo, cache=40)
    plain = spr.AttentionBlock((2, 10, 128), 4, 64, w, wo)
    assert spr.AttentionBlock((2, 1, 128), 4, 64, w, wo, cache=cached).keys is cached.keys
    for shape, of in (((3, 10, 128), cached), ((2, 41, 128), cached), ((2, 10, 128), plain)):
        with pytest.raises(ValueError):
            spr.AttentionBlock(shape, 4, 64, w, wo, cache=of)
    with pytest.raises(ValueError):
        spr.AttentionBlock((2, 10, 128), 4, 64, w.half(), wo.half(), sparse=sparse)
    with pytest.raises(spr.SparsePRError):  # attention has no heads of 96 channels
        spr.AttentionBlock((2, 10, 128), 4, 192, *weights(4, 4, 192, 128))


def test_calls():
    w, wo = weights(4, 2, 64, 128)
    x, cos = torch.zeros(2, 10, 128, dtype=BF), torch.zeros(40, 32)
    i32 = dict(dtype=torch.int32)
    dense = spr.AttentionBlock((2, 10, 128), 4, 64, w, wo, kv_heads=2)
    cached = spr.AttentionBlock((2, 10, 128), 4, 64, w, wo, kv_heads=2, cache=30)
    for block, args, kw in (
            (dense, (x[:, :9], cos, cos), {}), (dense, (x,), {}), (dense, (x, cos[:9], cos[:9]), {}),
            (dense, (x, cos, cos), dict(at=1)), (dense, (x, cos, cos), dict(residual=x[:1])),
            (dense, (x, cos, cos), dict(out=x[:, :, :64])),
            (dense, (x, cos, cos), dict(prefix=torch.zeros(2, **i32))),  # not causal
            (cached, (x, cos, cos), dict(at=21)), (cached, (x, cos, cos), dict(at=-1)),
            (cached, (x, cos[:25], cos[:25]), dict(at=20)),
            (cached, (x, cos, cos), dict(k_len=torch.zeros(2, **i32))),
            (cached, (x, cos, cos), dict(doc=torch.zeros(2, 10, **i32))),
            (dense, (x, cos, cos), {})):  # the last: not on a GPU
        with pytest.raises(ValueError):
            block(*args, **kw)


def test_strides_that_no_tensor_map_describes():
    """One row for all tokens, or one query head for all heads, is refused; batches and key heads
    may share."""
    x, w, y = torch.zeros(2, 1, 40, 64, dtype=BF), torch.zeros(64, 64, dtype=BF), \
        torch.zeros(2, 1, 40, 64, dtype=BF)
    with pytest.raises(spr.SparsePRError):
        spr.alloc_workspace(spr.make_project(x[:, :, :1].expand(2, 1, 40, 64), w, y), device="cpu")
    assert spr.alloc_workspace(spr.make_project(x[:1].expand(2, 1, 40, 64), w, y),
                               device="cpu").numel() > 0
    q, k = torch.zeros(2, 4, 10, 64, dtype=BF), torch.zeros(2, 4, 30, 64, dtype=BF)
    with pytest.raises(spr.SparsePRError):
        spr.alloc_workspace(spr.make_masked(q[:, :1].expand(2, 4, 10, 64), k, k, q), device="cpu")
    one = k[:1, :1].expand(2, 4, 30, 64)
    assert spr.alloc_workspace(spr.make_masked(q, one, one, q), device="cpu").numel() > 0


def test_copied_parameters():
    """A copy has the fields and outlives what it was made from."""
    q = torch.zeros(2, 4, 10, 64, dtype=BF)
    x, w = torch.zeros(2, 1, 10, 64, dtype=BF), torch.zeros(64, 64, dtype=BF)
    for prm in (spr.make_masked(q, q, q, q, softcap=3.0), spr.make_norm_rotate(q, q, q, q),
                spr.make_project(x, w, x)):
        want = bytes(prm)
        copies = [copy.copy(prm), copy.deepcopy(prm), pickle.loads(pickle.dumps(prm))]
        del prm
        for c in copies:
            assert bytes(c) == want and "plan" not in c.__dict__
