"""Offsets past 2^31 elements in every tensor that the kernels address themselves, and two host
threads on one set of parameters."""
import threading

import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import attend, check, norm_rotate, project

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
FAR = 2 ** 31 + 2 ** 10  # elements from one batch, head or token to the next


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def far(shape, dim, dtype):
    """A tensor of the shape whose dimension `dim` of two entries has the stride FAR."""
    B, H, N, d = shape
    assert shape[dim] == 2 and B * H * N * d <= 2 ** 12
    base = torch.empty(FAR + 2 ** 13, device="cuda", dtype=dtype)
    stride = [H * N * d, N * d, d, 1]
    if dim == 2:
        stride = [H * d, d, FAR, 1]
    else:
        stride[dim] = FAR
    return base.as_strided(shape, stride)


def filled(shape, dim, dtype, seed):
    t = far(shape, dim, dtype)
    t.copy_(randn(shape, dtype, seed))
    return t


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("Nk", [200, 1000])
def test_attention(dim, Nk):
    """Queries, keys, values and outputs; with the keys split (1,000) and not."""
    shape = [1, 1, 1, 64]
    shape[dim] = 2
    B, H, N, d = shape
    q, o = filled(shape, dim, BF, 1), far(shape, dim, BF)
    k, v = randn((B, H, Nk, d), BF, 2), randn((B, H, Nk, d), BF, 3)
    prm = spr.make_masked(q, k, v, o)
    spr.sparsepr_attend_masked(prm, q, k, v, o, spr.alloc_workspace(prm))
    want, tol, _, _ = attend(q, k, v)
    check(o, want, tol, "O")


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_attention_keys(dim):
    shape = [1, 1, 5, 64]
    shape[dim] = 2
    k, v = filled(shape, dim, BF, 4), filled(shape, dim, BF, 5)
    q = randn((shape[0], shape[1], 3, 64), BF, 6)
    o = torch.empty_like(q)
    prm = spr.make_masked(q, k, v, o)
    spr.sparsepr_attend_masked(prm, q, k, v, o, spr.alloc_workspace(prm))
    want, tol, _, _ = attend(q, k, v)
    check(o, want, tol, "O")


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_norm_rotate(dim, dtype):
    shape = [1, 1, 3, 64]
    shape[dim] = 2
    x, y = filled(shape, dim, dtype, 7), far(shape, dim, dtype)
    w = randn((64,), dtype, 8)
    cos, sin = (randn((3, 32), torch.float32, s) for s in (9, 10))
    prm = spr.make_norm_rotate(x, None, y, None)
    spr.sparsepr_norm_rotate(prm, x, None, y, None, wq=w, cos=cos, sin=sin)
    want, tol = norm_rotate(x, w, cos, sin, None, norm=True, eps=1e-6, rot=64,
                            pairing="interleaved", out=dtype)
    check(y, want, tol, "y")


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("where", ["x", "y", "r"])
@pytest.mark.parametrize("rows", ["few", "some"])
def test_projection(rows, where, dim):
    """Few rows (pointers), and more (tensor maps, and pointers where K is split)."""
    d, N = 64, 2 if rows == "few" or dim == 2 else 32
    B, H = (9 if rows == "some" else 1, 1) if dim == 2 else (2, 1) if dim == 0 else (1, 2)
    shape = (B, H, N, d)
    one = lambda name, s: filled(shape, dim, BF, s) if where == name else randn(shape, BF, s)  # noqa: E731
    x, r = one("x", 11), one("r", 12)
    y = far(shape, dim, BF) if where == "y" else torch.empty(shape, device="cuda", dtype=BF)
    w = randn((H * d, H * d), BF, 13, 0.1)
    prm = spr.make_project(x, w, y, residual=r)
    spr.sparsepr_project(prm, x, w, y, spr.alloc_workspace(prm), residual=r)
    want, tol = project(x, w, None, None, r, "none", H)
    check(y, want, tol, "Y")


def test_projection_rows_of_a_split_sum():
    """17 rows of a deep product, whose sums are joined by pointers: Y and R in far batches."""
    B, N, K, d = 2, 16, 4096, 64
    x, w = randn((B, 1, N, K), BF, 14), randn((d, K), BF, 15, K ** -0.5)
    y, r = far((B, 1, N, d), 0, BF), filled((B, 1, N, d), 0, BF, 16)
    prm = spr.make_project(x, w, y, residual=r, act="silu")
    ws = spr.alloc_workspace(prm)
    assert ws.numel() > 256  # split
    spr.sparsepr_project(prm, x, w, y, ws, residual=r)
    want, tol = project(x, w, None, None, r, "silu", 1)
    check(y, want, tol, "Y")


def test_two_threads_on_one_set_of_parameters():
    """Each with its stream, outputs and workspace."""
    q, k, v = randn((2, 4, 150, 64), BF, 17), randn((2, 4, 700, 64), BF, 18), randn((2, 4, 700, 64), BF, 19)
    x, w = randn((1, 1, 300, 256), BF, 20), randn((256, 256), BF, 21, 0.06)
    am, nr = spr.make_masked(q, k, v, torch.empty_like(q)), spr.make_norm_rotate(q, k, q, k, rot=0)
    pj = spr.make_project(x, w, torch.empty_like(x))
    torch.cuda.synchronize()
    outs, failed = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    o, y, qo, ko = (torch.empty_like(t) for t in (q, x, q, k))
                    spr.sparsepr_attend_masked(am, q, k, v, o, spr.alloc_workspace(am))
                    spr.sparsepr_norm_rotate(nr, q, k, qo, ko)
                    spr.sparsepr_project(pj, x, w, y, spr.alloc_workspace(pj))
                torch.cuda.current_stream().synchronize()
                outs[i] = (o, y, qo, ko)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    want, tol, _, _ = attend(q, k, v)
    check(outs[0][0], want, tol, "O")
