"""The operators' forms that sizes select, against the formulas in 64 bits: items taken as blocks
come free, capped scores near and far, split sums over boxed batches, broadcast inputs, streams."""
import math

import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import attend, check, norm_rotate, project
from test_gpu_attend_masked import compare, run, tensors
from test_gpu_project import laid_out, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ----------------------------------------------------------- masked attention
@pytest.mark.parametrize("causal", [False, True])
def test_documents_in_more_items_than_blocks(causal):
    """288 pairs of row tiles of very different length."""
    Q, K, V = tensors(2, 48, 48, 600, 600, 64, BF, seed=20)
    at = torch.arange(600, device="cuda", dtype=torch.int32)
    doc = torch.stack([(at > 40).int() + (at > 70).int() + (at > 390).int(),
                       torch.where(at < 511, at // 256, -1)]).int().contiguous()
    a = compare(Q, K, V, causal=causal, doc_q=doc, doc_k=doc)
    b, _ = run(Q, K, V, causal=causal, doc_q=doc, doc_k=doc)
    assert torch.equal(a, b)  # whichever block takes an item


def test_lengths_in_more_items_than_blocks():
    """Single tokens over caches filled to different lengths, keys split, items taken as they come."""
    Q, K, V = tensors(9, 32, 8, 1, 5000, 64, FP, seed=21)
    lens = torch.tensor([5000, 1, 0, 129, 4999, 2048, 77, 3000, 256], dtype=torch.int32, device="cuda")
    for kw in ({}, dict(causal=True), dict(softcap=15.0)):
        O = compare(Q, K, V, k_len=lens, **kw)
        assert (O[2] == 0).all()


@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0), "slopes", "lens", "docs"], ids=str)
def test_last_round_of_tiles_split(kw):
    """160 row tiles: 148 blocks take one whole each, the other 12 are split (not where lengths or
    documents make them differ)."""
    Q, K, V = tensors(2, 80, 80, 200, 1300, 64, BF, seed=28)
    if kw == "slopes":
        kw = dict(slopes=torch.linspace(0, 0.3, 80, device="cuda"))
    elif kw == "lens":
        kw = dict(k_len=torch.tensor([1300, 700], dtype=torch.int32, device="cuda"))
    elif kw == "docs":
        kw = dict(doc_q=(torch.arange(200, device="cuda", dtype=torch.int32) // 70).repeat(2, 1),
                  doc_k=(torch.arange(1300, device="cuda", dtype=torch.int32) // 500).repeat(2, 1))
    a = compare(Q, K, V, **kw)
    b, _ = run(Q, K, V, **kw)
    assert torch.equal(a, b)


def test_causal_heads_in_more_items_than_blocks():
    Q, K, V = tensors(2, 40, 8, 900, 900, 64, BF, seed=22)
    compare(Q, K, V, causal=True)


@pytest.mark.parametrize("Nq", [1, 60, 400])
@pytest.mark.parametrize("cap", [0.5, 3.0, 50.0, 1e6])
def test_capped_scores_near_and_far(Nq, cap):
    """All scores within the polynomial's range, all beyond, and one key beyond in one tile."""
    Q, K, V = tensors(1, 4, 2, Nq, 500, 128, BF, seed=23)
    compare(Q, K, V, softcap=cap)
    K[:, :, 300] *= 40
    compare(Q, K, V, softcap=cap)
    compare(Q, K, V, softcap=cap, slopes=torch.full((4,), 0.01, device="cuda"))


def test_cap_of_infinite_and_nan_scores():
    """An infinite score is capped; a NaN one stays its row's own."""
    for Nq in (3, 200):
        Q, K, V = tensors(1, 2, 2, Nq, 300, 64, BF, seed=24)
        Q[:, :, 0] = 0  # 0 x inf: a row of NaN
        Q[:, :, 1:, 0] = Q[:, :, 1:, 0].abs() + 0.5
        K[:, :, 200, 0] = float("inf")
        O, L = run(Q, K, V, softcap=10.0)
        assert torch.isnan(O[:, :, 0]).all() and torch.isnan(L[:, :, 0]).all()
        assert torch.isfinite(O[:, :, 1:]).all()
        K[:, :, 200, 0] = 3e38  # as good as infinite for the cap
        o, tol, lse, ltol = attend(Q, K, V, softcap=10.0)
        check(O[:, :, 1:], o[:, :, 1:], tol[:, :, 1:], "O")


def test_penalty_with_documents_prefix_and_far_positions():
    Q, K, V = tensors(2, 4, 2, 300, 700, 64, BF, seed=25)
    slopes = torch.tensor([0.0, 0.02, 1.0, -0.01], device="cuda")
    dq = (torch.arange(300, device="cuda", dtype=torch.int32) // 100).repeat(2, 1)
    dk = (torch.arange(700, device="cuda", dtype=torch.int32) // 233).repeat(2, 1)
    compare(Q, K, V, slopes=slopes, doc_q=dq, doc_k=dk)
    compare(Q, K, V, slopes=slopes, causal=True,
            prefix=torch.tensor([400, 20], dtype=torch.int32, device="cuda"))
    for start in (-200, 100000, -100000):
        compare(Q, K, V, slopes=slopes, q_start=start)


def test_attention_on_another_stream():
    """An explicit stream: the call that the extension module leaves to the Python checks."""
    Q, K, V = tensors(1, 2, 2, 130, 200, 64, BF, seed=26)
    O = torch.zeros_like(Q)
    prm = spr.make_masked(Q, K, V, O)
    ws = spr.alloc_workspace(prm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spr.sparsepr_attend_masked(prm, Q, K, V, O, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    o, tol, _, _ = attend(Q, K, V)
    check(O, o, tol, "O")
    with torch.cuda.stream(side):
        spr.sparsepr_attend_masked(prm, Q, K, V, O.zero_(), ws)
    torch.cuda.current_stream().wait_stream(side)
    check(O, o, tol, "O")


def test_parameters_changed_after_they_were_made():
    """A field set by hand is what the next call uses."""
    Q, K, V = tensors(1, 2, 2, 40, 90, 64, BF, seed=27)
    O = torch.empty_like(Q)
    prm = spr.make_masked(Q, K, V, O)
    ws = spr.alloc_workspace(prm)
    prm.causal, prm.softcap = 1, 4.0
    spr.sparsepr_attend_masked(prm, Q, K, V, O, ws)
    o, tol, _, _ = attend(Q, K, V, causal=True, softcap=4.0)
    check(O, o, tol, "O")
    prm.B = 2
    with pytest.raises(ValueError):
        spr.sparsepr_attend_masked(prm, Q, K, V, O, ws)


def test_long_cache_past_32_bit_offsets():
    """Keys whose element offsets pass 2^31."""
    N, d, H = 8_400_000, 64, 2
    K = torch.zeros(1, H, N, d, device="cuda", dtype=BF)
    V = torch.zeros(1, H, N, d, device="cuda", dtype=BF)
    for t, s in ((K, 1), (V, 2)):
        t[:, :, -300:] = randn((1, H, 300, d), BF, s)
    Q = randn((1, H, 1, d), BF, 3)
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    doc = torch.full((1, N), -1, dtype=torch.int32, device="cuda")
    doc[:, -300:] = 4
    O, L = run(Q, K, V, k_len=n, doc_q=torch.full((1, 1), 4, dtype=torch.int32, device="cuda"),
               doc_k=doc)
    o, tol, lse, ltol = attend(Q, K[:, :, -300:], V[:, :, -300:])
    check(O, o, tol, "O")
    check(L, lse, ltol, "lse")


# ----------------------------------------------------------------- projection
CASES = [  # B, N, Hx, dx, Hy, dy, dtype, act, x layout, y layout
    (40, 3, 1, 4096, 1, 256, BF, "none", "head", "head"),   # one batch of 120 rows, K split
    (40, 3, 32, 128, 2, 128, FP, "silu", "head", "head"),   # 42 batches to a box, K split
    (7, 40, 8, 64, 2, 64, BF, "none", "head", "token"),     # three batches to a box
    (2, 90, 16, 128, 1, 264, BF, "gelu", "head", "head"),   # a tile per batch, K split
    (3, 50, 1, 4096, 1, 264, FP, "gelu_tanh", "head", "head"),
    (1, 17, 1, 64, 1, 64, BF, "none", "head", "head"),
    (1, 16, 1, 8, 1, 24, BF, "none", "head", "head"),
    (16, 1, 3, 64, 3, 64, FP, "none", "head", "head"),
    (1, 9, 1, 4104, 1, 4104, BF, "silu", "head", "head"),
    (1, 20000, 1, 64, 1, 320, BF, "none", "head", "head"),  # many tiles of one stage
    (2, 4000, 4, 64, 24, 64, BF, "none", "token", "head"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).split(".")[-1] for x in c))
def test_projection_forms(case):
    B, N, Hx, dx, Hy, dy, dt, act, xl, yl = case
    M, K = Hy * dy, Hx * dx
    x, y = laid_out(B, Hx, N, dx, dt, 31, xl), laid_out(B, Hy, N, dy, dt, 32, yl)
    w, r = randn((M, K), dt, 33, K ** -0.5), randn((B, Hy, N, dy), dt, 34)
    b, g = randn((M,), dt, 35), randn((B, M), dt, 36)
    prm = spr.make_project(x, w, y, residual=r, act=act)
    ws = spr.alloc_workspace(prm)
    spr.sparsepr_project(prm, x, w, y, ws, bias=b, gate=g, residual=r)
    want, tol = project(x, w, b, g, r, act, Hy)
    check(y, want, tol, "Y")


@pytest.mark.parametrize("N", [1, 30, 200])
def test_broadcast_inputs_of_a_projection(N):
    """X and the residual shared by the batches, and the residual by the heads too."""
    B, Hx, Hy, d = 40, 2, 2, 64
    x = randn((1, Hx, N, d), BF, 1).expand(B, Hx, N, d)
    r = randn((1, 1, N, d), BF, 2).expand(B, Hy, N, d)
    w, g = randn((Hy * d, Hx * d), BF, 3, 0.1), randn((B, Hy * d), BF, 4)
    y = torch.empty(B, Hy, N, d, device="cuda", dtype=BF)
    prm = spr.make_project(x, w, y, residual=r)
    spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm), gate=g, residual=r)
    want, tol = project(x, w, None, g, r, "none", Hy)
    check(y, want, tol, "Y")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_over_their_whole_range(act):
    """One product per output, so that the activation sees the values themselves."""
    v = torch.cat([torch.linspace(-30, 30, 3001), torch.tensor([-1e4, -200., 200., 1e4, 0.])])
    for rows in (8, 128):
        x = torch.zeros(1, 1, rows, 8, device="cuda", dtype=BF)
        x[..., 0] = 1
        w = torch.zeros(3008, 8, device="cuda", dtype=BF)
        w[:3006, 0] = v.to(BF).cuda()
        y = torch.empty(1, 1, rows, 3008, device="cuda", dtype=BF)
        prm = spr.make_project(x, w, y, act=act)
        spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm))
        want, tol = project(x, w, None, None, None, act, 1)
        check(y, want, tol, "Y")


# ------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 2), (4, 4), (5, 7), (24, 24)])
def test_queries_and_keys_as_one_list_of_heads(Hq, Hk, pairing):
    """Groups of heads that hold queries, keys and both; other weights for each."""
    for B, N in ((1, 1), (2, 70), (1, 3000)):
        q, k = randn((B, Hq, N, 64), BF, 1), randn((B, Hk, N, 64), BF, 2)
        wq, wk = randn((64,), BF, 3), randn((64,), BF, 4)
        at = torch.arange(N + 9, device="cuda", dtype=torch.float64)[:, None]
        f = 256.0 ** (-torch.arange(16, device="cuda", dtype=torch.float64) / 16)
        cos, sin = (at * f).cos().float(), (at * f).sin().float()
        pos = torch.randint(0, N + 9, (B, N), device="cuda", dtype=torch.int32)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        prm = spr.make_norm_rotate(q, k, qo, ko, rot=32, pairing=pairing)
        spr.sparsepr_norm_rotate(prm, q, k, qo, ko, wq, wk, cos, sin, pos, pos)
        for got, x, w in ((qo, q, wq), (ko, k, wk)):
            want, tol = norm_rotate(x, w, cos, sin, pos, norm=True, eps=1e-6, rot=32,
                                    pairing=pairing, out=BF)
            check(got, want, tol, "y")


def test_nan_in_a_row_stays_there():
    q = randn((1, 2, 40, 64), BF, 1)
    q[0, 1, 7, 3] = float("nan")
    out = torch.empty_like(q)
    prm = spr.make_norm_rotate(q, None, out, None, rot=0)
    spr.sparsepr_norm_rotate(prm, q, None, out, None)
    bad = ~torch.isfinite(out).all(-1)
    assert bad.nonzero().tolist() == [[0, 1, 7]]
    assert math.isfinite(out[0, 0].float().sum().item())


# ------------------------------------------------- streams, together and captured
def all_three(seed):
    """A projection, a norm + rotation and an attention on tensors and workspaces of their own."""
    x, w = randn((1, 1, 700, 512), BF, seed), randn((6 * 64, 512), BF, seed + 1, 0.05)
    qkv = torch.empty(1, 6, 700, 64, device="cuda", dtype=BF)
    q, k, v = qkv[:, :2], qkv[:, 2:4], qkv[:, 4:]
    o = torch.empty(1, 2, 700, 64, device="cuda", dtype=BF)
    cos = torch.ones(700, 32, device="cuda")
    doc = (torch.arange(700, device="cuda", dtype=torch.int32) // 300).view(1, -1)
    pj, nr, am = spr.make_project(x, w, qkv), spr.make_norm_rotate(q, k, q, k), \
        spr.make_masked(q, k, v, o)
    wp, wa = spr.alloc_workspace(pj), spr.alloc_workspace(am)

    def call():
        spr.sparsepr_project(pj, x, w, qkv, wp)
        spr.sparsepr_norm_rotate(nr, q, k, q, k, cos=cos, sin=torch.zeros_like(cos))
        spr.sparsepr_attend_masked(am, q, k, v, o, wa, doc_q=doc, doc_k=doc)
    return call, o


def test_two_streams_at_once():
    calls = [all_three(41), all_three(43)]
    want = []
    for call, o in calls:
        call()
        want.append(o.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for (call, o), s in zip(calls, streams):
            with torch.cuda.stream(s):
                o.zero_()
                call()
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for (_, o), w in zip(calls, want):
        assert torch.equal(o, w)


def test_fork_and_join_in_a_capture():
    """Two branches of one captured graph, joined, then both once more in a row."""
    (a, oa), (b, ob) = all_three(45), all_three(47)
    a(), b()
    want = oa.clone(), ob.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    total = torch.empty_like(oa)
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            b()
        a()
        here.wait_stream(side)
        torch.add(oa, ob, out=total)
        b()
        a()
    for _ in range(3):
        oa.zero_(), ob.zero_(), total.zero_()
        g.replay()
        assert torch.equal(oa, want[0]) and torch.equal(ob, want[1])
        assert torch.equal(total, want[0] + want[1])
