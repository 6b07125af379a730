"""AttentionBlock: the operators in a row, each step against its formula in 64 bits on the inputs
that the step got."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import attend, check, norm_rotate, project
from synthetic import workload

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def weights(heads, kv, d, C, dtype):
    return dict(w_qkv=randn(((heads + 2 * kv) * d, C), dtype, 1, C ** -0.5),
                w_out=randn((C, heads * d), dtype, 2, (heads * d) ** -0.5),
                b_qkv=randn(((heads + 2 * kv) * d,), dtype, 3, 0.2), b_out=randn((C,), dtype, 4, 0.2),
                wq=1 + randn((d,), dtype, 5, 0.2), wk=1 + randn((d,), dtype, 6, 0.2))


def tables(rows, rot):
    at = torch.arange(rows, device="cuda", dtype=torch.float64)
    f = 256.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    return (at[:, None] * f).cos().float(), (at[:, None] * f).sin().float()


def projected(x, w, b, heads, d):
    """The product of the block's step, from the operator on its own."""
    B, N, C = x.shape
    y = torch.empty(B, heads, N, d, device="cuda", dtype=x.dtype)
    prm = spr.make_project(x.view(B, 1, N, C), w, y)
    spr.sparsepr_project(prm, x.view(B, 1, N, C), w, y, spr.alloc_workspace(prm), bias=b)
    want, tol = project(x.view(B, 1, N, C), w, b, None, None, "none", heads)
    check(y, want, tol, "projection")
    return y


def check_block(block, W, x, cos, sin, out, *, gate=None, residual=None, at=0, rot, pairing, **mask):
    """Every step of the block's last call."""
    B, N, C = x.shape
    h, kv, d = block.heads, block.kv_heads, block.d
    rows = (h + kv) * d
    if block.cache:
        qk = projected(x, W["w_qkv"][:rows], W["b_qkv"][:rows], h + kv, d)
        v = projected(x, W["w_qkv"][rows:], W["b_qkv"][rows:], kv, d)
        keys, values = block.keys[:, :, :at + N], block.values[:, :, :at + N]
        new_k = keys[:, :, at:]
        assert torch.equal(values[:, :, at:], v)
    else:
        qkv = projected(x, W["w_qkv"], W["b_qkv"], h + 2 * kv, d)
        qk, keys, values = qkv, block.keys, block.values
        new_k = keys
        assert torch.equal(values, qkv[:, h + kv:])
    for name, got, raw, w in (("q", block.q, qk[:, :h], W["wq"]), ("k", new_k, qk[:, h:h + kv], W["wk"])):
        want, tol = norm_rotate(raw, w, cos[at:], sin[at:], None, norm=True, eps=1e-6, rot=rot,
                                pairing=pairing, out=x.dtype)
        check(got, want, tol, name)
    if block.sparse is None:
        o, tol, _, _ = attend(block.q, keys, values, **mask)
        check(block.o, o, tol, "o")
    r = None if residual is None else residual.view(B, 1, N, C)
    want, tol = project(block.o, W["w_out"], W["b_out"], gate, r, "none", 1)
    check(out.view(B, 1, N, C), want, tol, "out")


@pytest.mark.parametrize("case", [
    (1, 1, 128, 2, 2, 64, BF), (2, 300, 256, 4, 2, 64, FP), (3, 130, 264, 6, 1, 128, BF),
    (1, 1025, 512, 4, 4, 128, BF)], ids=str)
@pytest.mark.parametrize("kind", ["all", "causal", "lens", "docs"])
def test_dense(case, kind):
    B, N, C, heads, kv, d, dt = case
    W = weights(heads, kv, d, C, dt)
    x, cos, sin = randn((B, N, C), dt, 7), *tables(N, d // 2)
    gate = randn((B, C), dt, 8)
    pairing = "halves" if kv == 1 else "interleaved"
    kw, mask = {}, {}
    if kind == "causal":
        kw = dict(causal=True, softcap=20.0)
        mask = dict(kw)
    if kind == "lens":
        mask = dict(k_len=torch.tensor([N, N // 2, 1][:B], device="cuda", dtype=torch.int32))
    if kind == "docs":
        doc = (torch.arange(N, device="cuda", dtype=torch.int32) // 90).repeat(B, 1)
        doc[:, N - N // 9:] = -1
        mask = dict(doc=doc)
    block = spr.AttentionBlock((B, N, C), heads, d, kv_heads=kv, rot=d // 2, pairing=pairing, **W,
                               **kw)
    extra = {k: v for k, v in mask.items() if k not in kw}
    out = block(x, cos, sin, gate=gate, residual=x, **extra)
    if "doc" in mask:
        mask = dict(doc_q=mask["doc"], doc_k=mask["doc"])
    check_block(block, W, x, cos, sin, out, gate=gate, residual=x, rot=d // 2, pairing=pairing, **mask)


def test_prompt_frames_and_tokens_over_a_cache():
    """A prompt, two frames and single tokens, each call seeing the keys of all before it; then the
    second prompt over the same cache, whose rows behind the filled part must not matter."""
    B, C, heads, kv, d, dt, cache = 2, 256, 8, 2, 64, BF, 700
    W = weights(heads, kv, d, C, dt)
    cos, sin = tables(cache, d)
    x = randn((B, cache, C), dt, 9)
    first = spr.AttentionBlock((B, 200, C), heads, d, kv_heads=kv, cache=cache, **W)
    blocks = {n: spr.AttentionBlock((B, n, C), heads, d, kv_heads=kv, cache=first, **W)
              for n in (150, 1)}
    blocks[200] = first
    first.keys.fill_(float("nan"))
    first.values.fill_(float("inf"))
    at = 0
    for n in (200, 150, 150, 1, 1, 1):
        part = x[:, at:at + n].contiguous()
        out = blocks[n](part, cos, sin, at=at, residual=part)
        check_block(blocks[n], W, part, cos, sin, out, residual=part, at=at, rot=d,
                    pairing="interleaved", causal=True)
        at += n
    again = x[:, 300:500].contiguous()
    out = first(again, cos, sin)
    check_block(first, W, again, cos, sin, out, rot=d, pairing="interleaved", causal=True)


def test_sparse_call_in_the_block():
    """The sparse call stands where masked attention does; its own result is the call's."""
    wl = workload("tiny")
    C = 256
    kw = dict(Ms=wl.Ms, p=wl.p, Gk=wl.Gk, Gq=wl.Gq, iters=wl.iters, seed=wl.index,
              route_mode=wl.route_mode, tau=wl.tau, M=wl.M, r=wl.r, lam=wl.lam)
    H, N, d = wl.H, wl.N, wl.d
    W = weights(H, H, d, C, BF)
    x, cos, sin = randn((1, N, C), BF, 10), *tables(N, d)
    block = spr.AttentionBlock((1, N, C), H, d, sparse=kw, **W)
    out = block(x, cos, sin, residual=x)
    check_block(block, W, x, cos, sin, out, residual=x, rot=d, pairing="interleaved")
    _, err = spr.sparsepr_get_stats(block._attend, block.ws_sparse)
    assert err == 0
    q, k, v = (t.contiguous() for t in (block.q, block.keys, block.values))
    o = torch.empty_like(q)
    prm = spr.make_params(q, k, v, o, **kw)
    spr.sparsepr_call(prm, q, k, v, o, spr.alloc_workspace(prm))
    assert torch.equal(o, block.o)


def test_captured_block():
    """A captured token step, replayed, gives what the call gives."""
    W = weights(4, 4, 128, 512, BF)
    cos, sin = tables(64, 128)
    block = spr.AttentionBlock((2, 1, 512), 4, 128, cache=64, **W)
    x = randn((2, 1, 512), BF, 11)
    for at in range(5):
        block(x, cos, sin, at=at)
    out = torch.empty_like(x)
    want = block(x, cos, sin, at=5).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(x, cos, sin, at=5, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
