"""Keys that no query of a batch sees may hold anything: the unfilled part of a cache."""
import pytest
import torch

from operators_reference import attend, check
from test_gpu_attend_masked import run, tensors

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("kind", ["causal", "prefix", "lens", "docs", "slopes", "softcap"])
@pytest.mark.parametrize("Hq,Hk,Nq,Nk,d,dtype,start", [
    (4, 1, 1, 300, 64, BF, 100), (4, 2, 1, 2000, 128, FP, 1500), (8, 2, 5, 700, 128, BF, 0),
    (2, 2, 200, 900, 64, BF, 130), (2, 1, 300, 400, 128, FP, -50), (2, 2, 130, 200, 64, BF, -400)])
def test_behind_the_last_query(Hq, Hk, Nq, Nk, d, dtype, start, kind):
    """A causal call at a given position over a cache whose later places were never written."""
    B = 2
    Q, K, V = tensors(B, Hq, Hk, Nq, Nk, d, dtype, seed=60)
    kw = dict(causal=True, q_start=start)
    end = [max(0, min(Nk, start + Nq))] * B
    if kind == "prefix":
        prefix = [Nk // 2 + 3, 0]
        kw["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
        end = [max(e, p) for e, p in zip(end, prefix)]
    if kind == "lens":
        lens = [Nk // 3 + 1, Nk]
        kw["k_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        end = [min(e, n) for e, n in zip(end, lens)]
    if kind == "docs":
        kw["doc_k"] = (torch.arange(Nk, device="cuda", dtype=torch.int32) // 70).repeat(B, 1)
        at = (torch.arange(Nq, device="cuda", dtype=torch.int32) + start).clamp(0, Nk - 1)
        kw["doc_q"] = (at // 70).repeat(B, 1)
    if kind == "slopes":
        kw["slopes"] = torch.full((Hq,), 0.05, device="cuda")
    if kind == "softcap":
        kw["softcap"] = 5.0
    for b in range(B):
        K[b, :, end[b]:], V[b, :, end[b]:] = 0, 0
    o, tol, lse, ltol = attend(Q, K, V, **kw)
    first, _ = run(Q, K, V, **kw)
    for b in range(B):
        K[b, :, end[b]:], V[b, :, end[b]:] = float("inf"), float("nan")
    O, L = run(Q, K, V, **kw)
    check(O, o, tol, "O")
    check(L, lse, ltol, "lse")
    assert torch.equal(O, first)
