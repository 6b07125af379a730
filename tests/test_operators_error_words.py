"""The error words at the start of a workspace: cleared when it is made, then left to the calls."""
import os

import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build
from operators_reference import attend, check, project

BF = torch.bfloat16


def test_words_of_a_new_workspace():
    spr_build.build()
    q = torch.zeros(2, 4, 10, 64, dtype=BF)
    x, w = torch.zeros(2, 1, 10, 64, dtype=BF), torch.zeros(64, 64, dtype=BF)
    for prm in (spr.make_masked(q, q, q, q), spr.make_project(x, w, x)):
        ws = spr.alloc_workspace(prm, device="cpu")
        assert ws.numel() >= 16 and (ws[:16] == 0).all()
        assert spr.sparsepr_workspace_error(ws) == 0
        ws[:4].view(torch.int32)[0] = 4
        assert spr.sparsepr_workspace_error(ws) == 4
        assert spr.sparsepr_workspace_error(ws[:16].view(torch.float32).view(2, 2)) == 4


def test_every_kernel_that_may_give_up_reports_it():
    """Where a wait sets the block's abort flag, the end of the kernel passes it on."""
    csrc = os.path.join(os.path.dirname(spr_build.__file__), "csrc")
    for name in ("k_attend_masked.cu", "k_project.cu"):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        kernels = [k for k in text.split("__global__")[1:] if "abort_s" in k]
        assert kernels
        for k in kernels:
            assert "if (threadIdx.x == 0 && *abort_s) report_timeout(a.status, a.words);" in k


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,Nq,Nk,docs", [(8, 2, 1, 5000, False), (4, 4, 300, 900, True),
                                              (80, 80, 200, 1300, False), (2, 2, 3, 40, False)])
def test_attention_leaves_them_alone(Hq, Hk, Nq, Nk, docs):
    """Partial results and lists are behind them; an earlier error stays."""
    g = torch.Generator("cuda").manual_seed(70)
    q = torch.randn(2, Hq, Nq, 64, generator=g, device="cuda").to(BF)
    k, v = (torch.randn(2, Hk, Nk, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    o = torch.empty_like(q)
    kw = {}
    if docs:
        kw = dict(doc_q=(torch.arange(Nq, device="cuda", dtype=torch.int32) // 70).repeat(2, 1),
                  doc_k=(torch.arange(Nk, device="cuda", dtype=torch.int32) // 200).repeat(2, 1))
    prm = spr.make_masked(q, k, v, o)
    ws = spr.alloc_workspace(prm)
    want, tol, _, _ = attend(q, k, v, **kw)
    for words in ([0, 0, 0, 0], [4, 9, -1, 5]):
        ws[:16].view(torch.int32).copy_(torch.tensor(words, device="cuda", dtype=torch.int32))
        spr.sparsepr_attend_masked(prm, q, k, v, o.zero_(), ws, **kw)
        check(o, want, tol, "O")
        assert ws[:16].view(torch.int32).tolist() == words
        assert spr.sparsepr_workspace_error(ws) == words[0]


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,M", [(4, 512, 512), (64, 4096, 256), (300, 128, 640)])
def test_projection_leaves_them_alone(N, K, M):
    g = torch.Generator("cuda").manual_seed(71)
    x = torch.randn(1, 1, N, K, generator=g, device="cuda").to(BF)
    w = (torch.randn(M, K, generator=g, device="cuda") * K ** -0.5).to(BF)
    y = torch.empty(1, 1, N, M, device="cuda", dtype=BF)
    prm = spr.make_project(x, w, y)
    ws = spr.alloc_workspace(prm)
    want, tol = project(x, w, None, None, None, "none", 1)
    for words in ([0, 0, 0, 0], [4, 9, -1, 5]):
        ws[:16].view(torch.int32).copy_(torch.tensor(words, device="cuda", dtype=torch.int32))
        spr.sparsepr_project(prm, x, w, y.zero_(), ws)
        check(y, want, tol, "Y")
        assert ws[:16].view(torch.int32).tolist() == words
