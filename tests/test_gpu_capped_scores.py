"""Capped scores: exact relative to each score, under every cap; and the same call gives the same
bits whatever ran before it."""
import math

import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import U32, check, half_step, smallest
from test_gpu_attend_masked import run, tensors

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def reference(Q, K, V, cap, slopes):
    """(O, its tolerance, lse, its tolerance) over every key, the last query on the last key.

    A score is off by its d products (tensor-core steps), by 16 roundings of its own size for the
    cap, and by those of the penalty and the change of base: each key's own, so that one far score
    does not excuse the others.
    """
    Nq, Nk, d = Q.shape[2], K.shape[2], Q.shape[3]
    rep = Q.shape[1] // K.shape[1]
    q, k, v = Q.double(), K.double().repeat_interleave(rep, 1), V.double().repeat_interleave(rep, 1)
    x = q @ k.transpose(-1, -2) * d ** -0.5
    es = (d + 8) * 2 * U32 * (q.abs() @ k.abs().transpose(-1, -2)) * d ** -0.5
    t = torch.tanh(x / cap)
    es = es * (1 - t * t) + es * es / cap  # the cap's slope, and its change over the error
    x = cap * t
    # the cap is bounded, however far the score and its error go
    es = torch.minimum(es, torch.full_like(es, 2 * cap)) + 16 * U32 * x.abs()
    if slopes is not None:
        at = torch.arange(Nq, device=Q.device) + (Nk - Nq)
        bias = slopes.double()[None, :, None, None] * (at[:, None] - torch.arange(Nk, device=Q.device)).abs()
        x = x - bias
        es = es + 4 * U32 * (x.abs() + bias)
    es = es + 4 * U32 * x.abs() + 8 * U32
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    off = torch.expm1(es)
    mean = (p * off).sum(-1)  # how far the sum is off
    u = half_step(Q.dtype)
    o, size = p @ v, p @ v.abs()
    wide = (p * off) @ v.abs() + mean[..., None] * size
    tol = u * o.abs() + (wide + (u + (Nk + 64) * 2 * U32) * size) * (1 + u) + smallest(Q.dtype)
    return o, tol, lse, mean + 4 * U32 * lse.abs() + (Nk / 32 + 64) * U32


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("Nq,d,dtype", [(1, 128, BF), (60, 64, FP), (400, 64, BF), (400, 128, FP)])
@pytest.mark.parametrize("cap", [1e-30, 1e-6, 0.5, 3.0, 50.0, 1e4, 1e6, 1e30, 3e38])
def test_scores_are_exact_relative_to_themselves(cap, Nq, d, dtype, slopes):
    Q, K, V = tensors(1, 4, 2, Nq, 500, d, dtype, seed=51)
    s = torch.tensor([0.0, 1e-3, 0.01, 0.1], device="cuda") if slopes else None
    if dtype == FP:
        K[:, :, 7] = 0  # a score of 0
    for far in (False, True):
        if far:  # one key beyond the near form in one tile, for one query out of three
            K[:, :, 300] *= 40
            Q[:, :, ::3] *= 30
        O, L = run(Q, K, V, softcap=cap, slopes=s)
        o, tol, lse, ltol = reference(Q, K, V, cap, s)
        check(O, o, tol, f"O far={far}")
        check(L, lse, ltol, f"lse far={far}")


def test_a_large_cap_is_no_cap_with_slopes_of_zero_or_without():
    """Scores far below the cap: the same as uncapped ones, to a few roundings of a score."""
    Q, K, V = tensors(1, 2, 2, 300, 700, 128, BF, seed=52)
    _, want = run(Q, K, V)
    zero = torch.zeros(2, device="cuda")
    for cap in (1e5, 1e6, 1e20):
        for kw in ({}, dict(slopes=zero)):
            _, L = run(Q, K, V, softcap=cap, **kw)
            # 24 roundings of a score of at most 16, as many of an lse of at most 16, and what the
            # cap itself takes from such a score, x^3 / 3 c^2
            assert math.isfinite(L.sum().item())
            assert (L - want).abs().max().item() <= 48 * U32 * 16 + 16 ** 3 / (3 * cap ** 2)


@pytest.mark.parametrize("cap", [1e-30, 1e-6, 1.0, 1e30])
@pytest.mark.parametrize("slopes", [False, True])
def test_scores_of_zero_under_any_cap(cap, slopes):
    Q, K, V = tensors(1, 2, 2, 40, 300, 64, BF, seed=53)
    K.zero_()
    s = torch.full((2,), 0.01, device="cuda") if slopes else None
    O, L = run(Q, K, V, softcap=cap, slopes=s)
    o, tol, lse, ltol = reference(Q, K, V, cap, s)
    check(O, o, tol, "O")
    check(L, lse, ltol, "lse")


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


@pytest.mark.parametrize("Nq", [1, 5, 200])
def test_bits_do_not_depend_on_keys_that_do_not_count(Nq):
    """Lengths, negative documents and keys behind a causal query, in tiles that hold others too."""
    Q, K, V = tensors(2, 4, 2, Nq, 500, 64, BF, seed=54)
    lens = torch.tensor([430, 300], dtype=torch.int32, device="cuda")
    doc = torch.zeros(2, 500, dtype=torch.int32, device="cuda")
    doc[:, 100:140] = -1
    kinds = [dict(k_len=lens), dict(k_len=lens, causal=True),
             dict(doc_q=doc[:, :Nq].clamp(min=0).contiguous(), doc_k=doc)]
    for kw in kinds:
        got = []
        for value in (0.0, 1e4, -1e30, float("nan")):
            for b, n in enumerate((430, 300)):
                if "k_len" in kw:
                    K[b, :, n:], V[b, :, n:] = value, value
                else:
                    K[b, :, 100:140], V[b, :, 100:140] = value, value
            got.append(run(Q, K, V, softcap=30.0, **kw))
        for O, L in got[1:]:
            assert torch.equal(O, got[0][0]) and torch.equal(L, got[0][1])
        K[:, :, 100:140], V[:, :, 100:140] = 0.5, 0.5
        K[:, :, 300:], V[:, :, 300:] = 0.5, 0.5
