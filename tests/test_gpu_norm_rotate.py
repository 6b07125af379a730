"""sparsepr_norm_rotate against its formula in 64 bits."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import check, norm_rotate

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def make(B, H, N, d, dtype, seed, layout="head"):
    g = torch.Generator("cuda").manual_seed(seed)
    if layout == "head":
        return torch.randn(B, H, N, d, generator=g, device="cuda").to(dtype)
    if layout == "token":  # a view of a token-major projection
        return torch.randn(B, N, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    big = torch.randn(B, H + 2, N + 3, d + 16, generator=g, device="cuda").to(dtype)
    return big[:, 1:H + 1, 2:N + 2, 8:d + 8]


def tables(rows, rot, seed=5):
    g = torch.Generator("cuda").manual_seed(seed)
    ang = torch.rand(rows, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 1000
    return ang.cos().float(), ang.sin().float()


CASES = [  # B, Hq, Hk, Nq, Nk, d, in, out, rot, pairing, norm, weights, positions, layout
    (1, 1, 1, 1, 1, 128, BF, BF, 128, "interleaved", True, True, False, "head"),
    (1, 24, 24, 1, 1, 128, BF, BF, 128, "halves", True, True, True, "head"),
    (2, 3, 1, 257, 19, 64, FP, FP, 32, "halves", True, True, True, "token"),
    (3, 20, 4, 33, 33, 64, FP, BF, 64, "interleaved", True, False, True, "cut"),
    (1, 5, 2, 100, 3, 128, F32, F32, 64, "halves", True, True, False, "token"),
    (1, 2, 2, 65, 65, 128, F32, BF, 128, "interleaved", False, False, True, "cut"),
    (2, 4, 4, 31, 31, 8, BF, BF, 8, "interleaved", True, True, False, "head"),
    (1, 4, 4, 77, 77, 256, BF, BF, 256, "halves", True, True, True, "token"),
    (1, 3, 3, 40, 40, 96, BF, BF, 48, "halves", True, True, False, "cut"),
    (1, 3, 3, 40, 40, 200, FP, FP, 104, "interleaved", True, True, False, "head"),
    (1, 3, 3, 40, 40, 24, F32, F32, 16, "halves", True, True, False, "head"),
    (2, 7, 0, 130, 0, 128, BF, BF, 128, "interleaved", True, True, True, "head"),
    (1, 6, 6, 50, 50, 64, BF, BF, 0, "interleaved", True, True, False, "token"),
    (1, 9, 3, 1025, 2049, 128, BF, BF, 128, "halves", True, True, False, "head"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).split(".")[-1] for x in c))
def test_against_formula(case):
    B, Hq, Hk, Nq, Nk, d, ti, to, rot, pairing, norm, weights, positions, layout = case
    q = make(B, Hq, Nq, d, ti, 1, layout)
    k = make(B, Hk, Nk, d, ti, 2, layout) if Hk else None
    w = [(1 + 0.5 * torch.randn(d, device="cuda")).to(ti) if weights else None for _ in range(2)]
    rows = max(Nq, Nk) + (37 if positions else 0)
    cos, sin = tables(rows, rot) if rot else (None, None)
    pos = [torch.randint(0, rows, (B, n), device="cuda", dtype=torch.int32)
           if positions and n else None for n in (Nq, Nk)]
    qo = torch.full((B, Nq, Hq, d), 7.0, device="cuda", dtype=to).transpose(1, 2)
    ko = torch.full((B, Hk, Nk, d), 7.0, device="cuda", dtype=to) if Hk else None
    prm = spr.make_norm_rotate(q, k, qo, ko, eps=1e-5, norm=norm, rot=rot, pairing=pairing)
    status = torch.full((4,), 9, device="cuda", dtype=torch.int32)
    spr.sparsepr_norm_rotate(prm, q, k, qo, ko, wq=w[0], wk=w[1] if Hk else None, cos=cos, sin=sin,
                             pos_q=pos[0], pos_k=pos[1], status=status)
    for x, y, ww, p, what in ((q, qo, w[0], pos[0], "queries"), (k, ko, w[1], pos[1], "keys")):
        if x is None:
            continue
        want, tol = norm_rotate(x, ww, cos, sin, p, norm=norm, eps=1e-5, rot=rot, pairing=pairing,
                                out=to)
        check(y, want, tol, what)
    assert status[0].item() == 0


def test_in_place_and_repeated():
    q, k = make(2, 4, 70, 128, BF, 1, "token"), make(2, 2, 70, 128, BF, 2)
    cos, sin = tables(70, 128)
    want = []
    for x in (q, k):
        o = torch.empty_like(x)
        prm = spr.make_norm_rotate(x, None, o, None)
        spr.sparsepr_norm_rotate(prm, x, None, o, None, cos=cos, sin=sin)
        want.append(o)
    prm = spr.make_norm_rotate(q, k, q, k)
    spr.sparsepr_norm_rotate(prm, q, k, q, k, cos=cos, sin=sin)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_row_outside_the_tables_is_reported_and_left():
    q = make(2, 3, 5, 64, BF, 1)
    out = torch.full_like(q, 3.0)
    cos, sin = tables(10, 64)
    pos = torch.arange(10, device="cuda", dtype=torch.int32).view(2, 5).clone()
    pos[1, 2] = 10
    status = torch.zeros(4, device="cuda", dtype=torch.int32)
    prm = spr.make_norm_rotate(q, None, out, None)
    spr.sparsepr_norm_rotate(prm, q, None, out, None, cos=cos, sin=sin, pos_q=pos, status=status)
    assert status.tolist() == [1, 1, 2, 10]
    assert (out[1, :, 2] == 3).all()
    pos[1, 2] = 0
    want, tol = norm_rotate(q, None, cos, sin, pos, norm=True, eps=1e-6, rot=64,
                            pairing="interleaved", out=BF)
    keep = torch.ones(2, 5, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    check(out.transpose(1, 2)[keep], want.transpose(1, 2)[keep], tol.transpose(1, 2)[keep], "rest")
    # negative, and no status asked for
    pos[0, 0] = -1
    out.fill_(3.0)
    spr.sparsepr_norm_rotate(prm, q, None, out, None, cos=cos, sin=sin, pos_q=pos)
    assert (out[0, :, 0] == 3).all() and not (out[0, :, 1] == 3).all()


def test_rows_of_zeros_and_extremes():
    q = torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.float32)
    q[0, 0, 1] = 1e18   # the mean square is near the largest fp32
    q[0, 0, 2] = 1e-12  # and below eps
    q[0, 0, 3, 5] = float("nan")
    out = torch.empty_like(q)
    prm = spr.make_norm_rotate(q, None, out, None, rot=0)
    spr.sparsepr_norm_rotate(prm, q, None, out, None)
    assert (out[0, 0, 0] == 0).all()
    assert torch.allclose(out[0, 0, 1], torch.ones(64, device="cuda"), rtol=18 * 2.0 ** -24)
    assert torch.allclose(out[0, 0, 2], torch.full((64,), 1e-9, device="cuda"), rtol=18 * 2.0 ** -24)
    assert torch.isnan(out[0, 0, 3]).all()


def test_graph_and_streams():
    q, k = make(1, 4, 200, 128, BF, 1), make(1, 4, 200, 128, BF, 2)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    cos, sin = tables(200, 128)
    prm = spr.make_norm_rotate(q, k, qo, ko)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spr.sparsepr_norm_rotate(prm, q, k, qo, ko, cos=cos, sin=sin, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = qo.clone(), ko.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spr.sparsepr_norm_rotate(prm, q, k, qo, ko, cos=cos, sin=sin)
    qo.zero_(), ko.zero_()
    g.replay()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
