"""sparsepr_project against its formula in 64 bits."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import check, half_step, project

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def laid_out(B, H, N, d, dtype, seed, layout):
    if layout == "token":
        return randn((B, N, H, d), dtype, seed).transpose(1, 2)
    if layout == "cut":
        return randn((B, H + 1, N + 2, d + 8), dtype, seed)[:, 1:, 1:N + 1, 8:]
    return randn((B, H, N, d), dtype, seed)


CASES = [  # B, N, Hx, dx, Hy, dy, dtype, act, bias, gate, residual, x layout, y layout
    (1, 1, 1, 8, 1, 8, BF, "none", False, False, False, "head", "head"),
    (1, 1, 1, 2048, 1, 512, BF, "none", True, True, True, "head", "head"),
    (4, 1, 5, 128, 1, 640, BF, "none", True, True, True, "head", "head"),
    (3, 1, 1, 264, 2, 64, FP, "silu", True, True, True, "head", "token"),
    (2, 7, 1, 1000, 1, 1000, FP, "gelu", True, False, True, "cut", "cut"),
    (1, 16, 4, 64, 1, 72, BF, "gelu_tanh", True, False, False, "token", "head"),
    (1, 33, 1, 512, 3, 128, BF, "none", False, True, False, "head", "head"),
    (1, 127, 1, 128, 1, 256, BF, "none", True, False, True, "head", "head"),
    (2, 129, 2, 128, 1, 136, BF, "silu", True, True, True, "head", "token"),
    (3, 255, 1, 200, 2, 64, FP, "gelu_tanh", True, True, True, "token", "head"),
    (1, 513, 1, 1160, 1, 1288, BF, "gelu", True, True, True, "head", "head"),
    (2, 300, 3, 64, 3, 128, FP, "none", True, False, False, "cut", "cut"),
    (1, 2100, 8, 128, 1, 1024, BF, "none", True, True, True, "head", "head"),
    (2, 1000, 1, 2048, 12, 128, BF, "none", True, False, False, "head", "head"),
    (1, 2049, 1, 64, 1, 2056, FP, "gelu", False, False, False, "head", "head"),
    (65, 3, 1, 256, 1, 256, BF, "none", True, True, True, "head", "head"),
    (5, 64, 2, 64, 2, 64, BF, "none", False, False, True, "head", "head"),
    (1, 40, 1, 16384, 1, 96, BF, "none", True, False, False, "head", "head"),
]


def inputs(case):
    B, N, Hx, dx, Hy, dy, dt, act, bias, gate, residual, xl, yl = case
    M, K = Hy * dy, Hx * dx
    x = laid_out(B, Hx, N, dx, dt, 1, xl)
    w = randn((M, K + (8 if xl == "cut" else 0)), dt, 2, K ** -0.5)[:, :K]
    y = laid_out(B, Hy, N, dy, dt, 3, yl)
    r = laid_out(B, Hy, N, dy, dt, 4, "head") if residual else None
    return (x, w, y, randn((M,), dt, 5) if bias else None, randn((B, M), dt, 6) if gate else None, r,
            act, Hy)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).split(".")[-1] for x in c))
def test_against_formula(case):
    x, w, y, b, g, r, act, Hy = inputs(case)
    prm = spr.make_project(x, w, y, residual=r, act=act)
    ws = spr.alloc_workspace(prm)
    status = torch.full((4,), 9, device="cuda", dtype=torch.int32)
    spr.sparsepr_project(prm, x, w, y, ws, bias=b, gate=g, residual=r, status=status)
    want, tol = project(x, w, b, g, r, act, Hy)
    check(y, want, tol, "Y")
    # as a whole the roundings of Y are the error: at most half a step each
    if act == "none" and r is None:
        assert (y.double() - want).norm() <= 1.05 * half_step(x.dtype) * want.norm()
    assert status[0].item() == 0
    first = y.clone()
    spr.sparsepr_project(prm, x, w, y, ws, bias=b, gate=g, residual=r)
    assert torch.equal(first, y)  # the same sums in the same order


def test_surroundings_are_left():
    """Rows and columns around a strided Y keep what they held."""
    x, w = randn((2, 1, 70, 96), BF, 1), randn((72, 96), BF, 2, 0.1)
    big = torch.full((2, 1, 75, 104), 5.0, device="cuda", dtype=BF)
    y = big[:, :, 2:72, 16:88]
    prm = spr.make_project(x, w, y)
    spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm))
    want, tol = project(x, w, None, None, None, "none", 1)
    check(y, want, tol, "Y")
    y.fill_(5.0)
    assert (big == 5).all()


def test_residual_in_place():
    for N in (3, 500):
        x, w = randn((2, 4, N, 64), BF, 1), randn((512, 256), BF, 2, 0.06)
        y = randn((2, 1, N, 512), BF, 3)
        want, tol = project(x, w, None, None, y, "none", 1)
        prm = spr.make_project(x, w, y)
        spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm), residual=y)
        check(y, want, tol, "Y")


def test_infinite_and_nan_rows_stay_their_own():
    x, w = randn((1, 1, 300, 256), BF, 1), randn((128, 256), BF, 2, 0.06)
    x[0, 0, 17, 3] = float("nan")
    x[0, 0, 200, 5] = float("inf")
    y = torch.empty(1, 1, 300, 128, device="cuda", dtype=BF)
    prm = spr.make_project(x, w, y)
    spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm))
    bad = ~torch.isfinite(y[0, 0]).all(-1)
    assert bad.nonzero().flatten().tolist() == [17, 200]


def test_graph_streams_and_shared_workspace():
    """Two captured projections that share a workspace, replayed in turn on one stream."""
    a, b = inputs(CASES[1]), inputs(CASES[12])
    runs = []
    pa, pb = (spr.make_project(t[0], t[1], t[2], residual=t[5], act=t[6]) for t in (a, b))
    ws = max(spr.alloc_workspace(pa), spr.alloc_workspace(pb), key=lambda t: t.numel())
    for t, p in ((a, pa), (b, pb)):
        call = lambda t=t, p=p, **kw: spr.sparsepr_project(  # noqa: E731
            p, t[0], t[1], t[2], ws, bias=t[3], gate=t[4], residual=t[5], **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        want = t[2].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, t[2], want))
    for _ in range(3):
        for g, y, _ in runs:
            y.zero_()
            g.replay()
    for g, y, want in runs:
        assert torch.equal(y, want)
