"""Where AttentionBlock's tokens sit: padded batches without a cache, frames over one."""
import pytest
import torch

import free_block_sparse_means_b200 as spr
from operators_reference import attend, check
from test_gpu_attention_block import check_block, randn, tables, weights

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("kind", ["causal", "prefix", "slopes", "causal_slopes"])
@pytest.mark.parametrize("N", [10, 300])
def test_padded_batch(N, kind):
    """Token n of a batch of which k_len tokens are real is at position n, not so many before the
    last real one."""
    B, C, heads, kv, d = 3, 128, 4, 2, 64
    W, (cos, sin) = weights(heads, kv, d, C, BF), tables(N, d)
    x = randn((B, N, C), BF, 7)
    k_len = torch.tensor([N, N // 2, 1], device="cuda", dtype=torch.int32)
    slopes = torch.tensor([0.0, 0.05, 0.3, 1.0], device="cuda") if "slopes" in kind else None
    causal = kind != "slopes"
    prefix = torch.tensor([0, N // 3, 1], device="cuda", dtype=torch.int32) \
        if kind == "prefix" else None
    block = spr.AttentionBlock((B, N, C), heads, d, kv_heads=kv, causal=causal, slopes=slopes, **W)
    out = block(x, cos, sin, k_len=k_len, prefix=prefix)
    check_block(block, W, x, cos, sin, out, rot=d, pairing="interleaved", causal=causal, q_start=0,
                k_len=k_len, prefix=prefix, slopes=slopes)
    # the first tokens do not depend on how many follow
    short = spr.AttentionBlock((B, 5, C), heads, d, kv_heads=kv, causal=True, slopes=slopes, **W)
    if causal and prefix is None:
        short(x[:, :5].contiguous(), cos, sin)
        want, tol, _, _ = attend(short.q[:2], short.keys[:2], short.values[:2], causal=True,
                                 slopes=slopes)
        check(block.o[:2, :, :5], want, tol, "first tokens")


def test_frames_over_a_cache():
    """prefix = at + N: the tokens of a frame see the whole frame and all before it."""
    B, C, heads, kv, d, N, cache = 2, 128, 4, 2, 64, 130, 400
    W, (cos, sin) = weights(heads, kv, d, C, BF), tables(cache, d)
    block = spr.AttentionBlock((B, N, C), heads, d, kv_heads=kv, cache=cache, **W)
    for at in (0, 130, 260):
        x = randn((B, N, C), BF, 8 + at)
        prefix = torch.full((B,), at + N, device="cuda", dtype=torch.int32)
        out = block(x, cos, sin, at=at, prefix=prefix)
        check_block(block, W, x, cos, sin, out, at=at, rot=d, pairing="interleaved")
