"""A distance penalty where the queries are far from the keys: all that is far is the lse."""
import pytest
import torch

from operators_reference import U32, attend, check
from test_gpu_attend_masked import run, tensors

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("softcap", [0.0, 4.0])
@pytest.mark.parametrize("Nq,Nk,d,dtype", [(1, 300, 64, BF), (6, 2000, 128, FP), (200, 500, 64, FP),
                                           (260, 130, 128, BF)])
@pytest.mark.parametrize("start", [2 ** 24 + 3, 2 ** 26 + 1, 2 ** 30, -2 ** 26, -2 ** 30])
def test_far_from_the_keys(start, Nq, Nk, d, dtype, softcap):
    """|p - j| is |p - n| + |n - j| for the key place n next to p: O is that of queries at n."""
    B, H = 2, 4
    Q, K, V = tensors(B, H, 2, Nq, Nk, d, dtype, seed=61)
    slopes = torch.tensor([0.0, 0.01, 0.3, -0.02], device="cuda")
    lens = torch.tensor([Nk, Nk - Nk // 3], dtype=torch.int32, device="cuda")
    O, L = run(Q, K, V, slopes=slopes, q_start=start, k_len=lens, softcap=softcap)
    for b in range(B):
        n = int(lens[b])
        place = n - 1 if start > 0 else 0
        # every query as a batch of its own at that place
        q = Q[b].transpose(0, 1).unsqueeze(2)
        k, v = (t[b:b + 1, :, :n].expand(Nq, 2, n, d) for t in (K, V))
        o, tol, lse, ltol = attend(q, k, v, slopes=slopes, q_start=place, softcap=softcap)
        check(O[b], o.squeeze(2).transpose(0, 1), tol.squeeze(2).transpose(0, 1), "O")
        away = (torch.arange(Nq, device="cuda", dtype=torch.float64) + (start - place)).abs()
        part = slopes.double()[:, None] * away
        want = lse.squeeze(2).t() - part
        # the distance and the sum are each rounded once
        check(L[b], want, ltol.squeeze(2).t() + 2 * U32 * part.abs() + U32 * want.abs(), "lse")


@pytest.mark.parametrize("start", [-130, 250])
def test_some_queries_before_or_behind_the_keys(start):
    Q, K, V = tensors(1, 2, 2, 300, 400, 64, BF, seed=62)
    slopes = torch.tensor([0.5, 0.02], device="cuda")
    for kw in ({}, dict(causal=True)):
        O, L = run(Q, K, V, slopes=slopes, q_start=start, **kw)
        o, tol, lse, ltol = attend(Q, K, V, slopes=slopes, q_start=start, **kw)
        check(O, o, tol, "O")
        check(L, lse, ltol, "lse")
