"""sparsepr_attend_masked against its formula in 64 bits."""
import math

import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import attend, check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def tensors(B, Hq, Hk, Nq, Nk, d, dtype, seed=0, layout="head", size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)

    def one(H, N, s):
        if layout == "token":
            return (torch.randn(B, N, H, d, generator=g, device="cuda") * s).to(dtype).transpose(1, 2)
        if layout == "cut":
            return (torch.randn(B, H + 1, N + 2, d + 8, generator=g, device="cuda") * s).to(
                dtype)[:, 1:, 1:N + 1, 8:]
        return (torch.randn(B, H, N, d, generator=g, device="cuda") * s).to(dtype)
    return one(Hq, Nq, size), one(Hk, Nk, size), one(Hk, Nk, 1.0)


def run(Q, K, V, *, lse=True, layout="head", scale=None, softcap=0.0, causal=False, q_start=None,
        **aux):
    B, H, N, d = Q.shape
    O = torch.full((B, N, H, d) if layout == "token" else (B, H, N, d), 7.0, device="cuda",
                   dtype=Q.dtype)
    O = O.transpose(1, 2) if layout == "token" else O
    L = torch.full((B, H, N), 7.0, device="cuda") if lse else None
    prm = spr.make_masked(Q, K, V, O, scale=scale or 0.0, softcap=softcap, causal=causal,
                          q_start=q_start)
    ws = spr.alloc_workspace(prm)
    status = torch.full((4,), 9, device="cuda", dtype=torch.int32)
    spr.sparsepr_attend_masked(prm, Q, K, V, O, ws, lse=L, status=status, **aux)
    assert status[0].item() == 0
    return O, L


def compare(Q, K, V, layout="head", **kw):
    O, L = run(Q, K, V, layout=layout, **kw)
    o, tol, lse, ltol = attend(Q, K, V, **kw)
    check(O, o, tol, "O")
    check(L, lse, ltol, "lse")
    return O


SHAPES = [  # B, Hq, Hk, Nq, Nk
    (1, 1, 1, 1, 1), (2, 4, 2, 1, 7), (1, 8, 1, 1, 1000), (3, 6, 2, 2, 129), (1, 2, 2, 5, 128),
    (1, 16, 2, 3, 777), (2, 3, 3, 17, 64), (1, 12, 1, 33, 300), (1, 2, 1, 64, 65),
    (2, 2, 2, 127, 127), (1, 3, 3, 128, 128), (1, 2, 1, 129, 257), (1, 2, 2, 255, 511),
    (1, 1, 1, 256, 1), (1, 4, 4, 300, 900), (1, 2, 2, 1000, 130), (2, 2, 1, 513, 640),
    (1, 1, 1, 1, 20000), (1, 1, 1, 2500, 2500),
]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_every_key(shape, d, dtype):
    compare(*tensors(*shape, d, dtype))


@pytest.mark.parametrize("shape", [(2, 4, 2, 1, 333), (1, 4, 1, 40, 200), (2, 2, 2, 300, 300),
                                   (1, 2, 1, 500, 130), (1, 2, 2, 130, 700), (1, 3, 3, 1100, 1100)],
                         ids=str)
@pytest.mark.parametrize("kind", ["causal", "start", "late", "prefix", "lens", "lens_causal",
                                  "softcap", "bias", "all"])
def test_masks(shape, kind):
    B, Hq, Hk, Nq, Nk = shape
    Q, K, V = tensors(*shape, 64 if Hq == 4 else 128, FP if Hk == 1 else BF, seed=3)
    kw = {}
    if kind in ("causal", "prefix", "lens_causal", "all"):
        kw["causal"] = True
    if kind == "start":
        kw.update(causal=True, q_start=5)
    if kind == "late":  # every query before the first key: empty rows
        kw.update(causal=True, q_start=-Nq // 2)
    if kind in ("prefix", "all"):
        kw["prefix"] = torch.tensor([Nk // 3, 0][:B], dtype=torch.int32, device="cuda")
    if kind in ("lens", "lens_causal", "all"):
        kw["k_len"] = torch.tensor([Nk - Nk // 4, 1][:B], dtype=torch.int32, device="cuda")
    if kind in ("softcap", "all"):
        kw["softcap"] = 2.0
    if kind in ("bias", "all"):
        kw["slopes"] = torch.exp2(-torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32))
    compare(Q, K, V, **kw)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kind", ["packed", "one", "each", "scattered", "none_left", "padded"])
def test_documents(kind, causal):
    B, H, N = 2, 2, 700
    Q, K, V = tensors(B, H, H, N, N, 64 if causal else 128, BF, seed=5)
    at = torch.arange(N, device="cuda", dtype=torch.int32).expand(B, N)
    doc = {"packed": at // 150, "one": torch.zeros_like(at), "each": at.clone(),
           "scattered": at * 7919 % 5, "none_left": torch.full_like(at, -1),
           "padded": torch.where(at % 97 < 60, at // 200, -3)}[kind].contiguous()
    compare(Q, K, V, causal=causal, doc_q=doc, doc_k=doc)


def test_documents_across_lengths():
    """Queries of one set of documents over keys of another, some of which have no keys."""
    Q, K, V = tensors(1, 4, 2, 333, 515, 128, FP, seed=6)
    dq = (torch.arange(333, device="cuda", dtype=torch.int32) // 50).view(1, -1).contiguous()
    dk = (torch.arange(515, device="cuda", dtype=torch.int32) // 130).view(1, -1).contiguous()
    compare(Q, K, V, doc_q=dq, doc_k=dk)
    compare(Q[:, :, :3], K, V, doc_q=dq[:, :3].contiguous(), doc_k=dk)


@pytest.mark.parametrize("layout", ["token", "cut"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 1, 300), (2, 4, 2, 300, 300)], ids=str)
def test_layouts(shape, layout):
    compare(*tensors(*shape, 128, BF, seed=7, layout=layout), layout=layout, causal=True)


def test_shared_keys_by_stride():
    """One key and value tensor for both batches and heads, through strides of 0."""
    Q, K, V = tensors(2, 3, 1, 140, 260, 64, BF, seed=8)
    K, V = K[:1].expand(2, 3, 260, 64), V[:1].expand(2, 3, 260, 64)
    compare(Q, K, V)


def test_keys_that_do_not_count_may_hold_anything():
    for Nq in (1, 200):
        Q, K, V = tensors(2, 2, 2, Nq, 300, 128, BF, seed=9)
        lens = torch.tensor([130, 0], dtype=torch.int32, device="cuda")
        for b, n in enumerate((130, 0)):
            K[b, :, n:] = float("nan")
            V[b, :, n:] = float("inf")
        O = compare(Q, K, V, k_len=lens)
        assert (O[1] == 0).all()
        doc = (torch.arange(300, device="cuda", dtype=torch.int32) // 64).repeat(2, 1)
        doc[:, 70:90] = -1
        K[:, :, 70:90] = float("inf")
        V[:, :, 70:90] = float("nan")
        K[1], V[1] = K[0], V[0]
        compare(Q, K, V, k_len=torch.tensor([130, 100], dtype=torch.int32, device="cuda"),
                doc_q=doc[:, :Nq].contiguous(), doc_k=doc)


def test_lengths_past_the_cache_and_below_zero_are_clamped():
    Q, K, V = tensors(2, 2, 2, 3, 50, 64, BF, seed=10)
    lens = torch.tensor([1000, -5], dtype=torch.int32, device="cuda")
    O, L = run(Q, K, V, k_len=lens, causal=True)
    o, tol, lse, ltol = attend(Q, K, V, k_len=lens, causal=True)
    check(O, o, tol, "O")
    check(L, lse, ltol, "lse")


@pytest.mark.parametrize("Nq", [1, 150])
def test_far_scores(Nq):
    """Scores far apart: a late key that outweighs all before it, and rows of equal scores."""
    Q, K, V = tensors(1, 2, 2, Nq, 600, 128, BF, seed=11, size=4.0)
    compare(Q, K, V)
    K[:, :, 590] = Q[:, :, :1].squeeze(2) * 4
    compare(Q, K, V)
    K.zero_()
    compare(Q, K, V)


def test_negative_and_large_scale_of_types():
    Q, K, V = tensors(1, 1, 1, 40, 400, 64, FP, seed=12, size=6.0)
    V *= 100
    compare(Q, K, V, scale=0.5)


def test_rows_do_not_touch_their_surroundings():
    Q, K, V = tensors(1, 2, 2, 130, 200, 64, BF, seed=13)
    big = torch.full((1, 3, 140, 72), 5.0, device="cuda", dtype=BF)
    O = big[:, 1:, 4:134, 8:]
    prm = spr.make_masked(Q, K, V, O)
    spr.sparsepr_attend_masked(prm, Q, K, V, O, spr.alloc_workspace(prm))
    o, tol, _, _ = attend(Q, K, V)
    check(O, o, tol, "O")
    O.fill_(5.0)
    assert (big == 5).all()


def test_repeated_calls_are_equal_bit_for_bit():
    for shape in ((2, 8, 2, 1, 5000), (1, 4, 4, 700, 900)):
        Q, K, V = tensors(*shape, 128, BF, seed=14)
        a, la = run(Q, K, V, causal=True)
        for _ in range(3):
            b, lb = run(Q, K, V, causal=True)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_graphs_that_share_a_workspace():
    runs = []
    sets = [(tensors(2, 8, 2, 1, 3000, 128, BF, seed=15), {}),
            (tensors(1, 4, 4, 400, 400, 128, BF, seed=16), {})]
    prms = [spr.make_masked(*t, torch.empty_like(t[0]), causal=True) for t, _ in sets]
    ws = max((spr.alloc_workspace(p) for p in prms), key=lambda t: t.numel())
    for (t, _), prm in zip(sets, prms):
        O = torch.empty_like(t[0])
        doc = torch.zeros(t[0].shape[0], t[0].shape[2], device="cuda", dtype=torch.int32)
        dk = torch.zeros(t[1].shape[0], t[1].shape[2], device="cuda", dtype=torch.int32)
        call = lambda t=t, O=O, prm=prm, doc=doc, dk=dk, **kw: spr.sparsepr_attend_masked(  # noqa: E731
            prm, *t, O, ws, doc_q=doc, doc_k=dk, **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        want = O.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, O, want))
    for _ in range(3):
        for g, O, _ in runs:
            O.zero_()
            g.replay()
    for _, O, want in runs:
        assert torch.equal(O, want)


def test_lse_joins_two_halves_of_the_keys():
    """Attention over two halves of a cache, joined by their lse, is attention over the whole."""
    Q, K, V = tensors(1, 4, 2, 90, 800, 64, BF, seed=17)
    (o1, l1), (o2, l2) = run(Q, K[:, :, :300], V[:, :, :300]), run(Q, K[:, :, 300:], V[:, :, 300:])
    l = torch.logaddexp(l1, l2)
    O = torch.exp(l1 - l)[..., None] * o1.float() + torch.exp(l2 - l)[..., None] * o2.float()
    o, tol, lse, ltol = attend(Q, K, V)
    # each half rounded its own output once more
    halves = torch.exp(l1 - l)[..., None] * o1.float().abs() + \
        torch.exp(l2 - l)[..., None] * o2.float().abs()
    check(O, o, tol + 2.0 ** -8 * halves.double() + 1e-5, "joined O")
    assert math.isfinite(l.sum().item())
