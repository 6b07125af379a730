"""The operators around the call in 64 bits, from their formulas, and how far a kernel may be off.

Tolerances count roundings: u = eps / 2 of the output's type for its one rounding, 2^-24 for a
rounding of fp32 arithmetic, 2^-23 for a step of a tensor-core accumulation, which need not round
to nearest.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the spacing of the type's subnormal numbers."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def norm_rotate(x, w, cos, sin, pos, *, norm, eps, rot, pairing, out):
    """(y, tolerance) of one side; x [B, H, N, d]."""
    y = x.double()
    if norm:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
    size = y.abs().clone()
    if rot:
        N = x.shape[2]
        c = cos.double()[:N] if pos is None else cos.double()[pos.long()][:, None]
        s = sin.double()[:N] if pos is None else sin.double()[pos.long()][:, None]
        if pairing == "halves":
            i0, i1 = torch.arange(rot // 2), torch.arange(rot // 2, rot)
        else:
            i0, i1 = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        a, b = y[..., i0], y[..., i1]
        y = y.clone()
        y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
        both = a.abs() * torch.maximum(c.abs(), s.abs()) + b.abs() * torch.maximum(c.abs(), s.abs())
        size[..., i0], size[..., i1] = both, both
    # the sum of squares (13 roundings, halved by the root), the root (4), mean and eps (2), two
    # products (2), the rotation (2): under 18 roundings relative to the terms' size
    tol = half_step(out) * y.abs() + 18 * U32 * size * (1 + half_step(out)) + smallest(out)
    return y, tol


def visible(B, Nq, Nk, device, *, causal, q_start, k_len, doc_q, doc_k, prefix):
    """[B, Nq, Nk] which keys a query sees, and [B, Nq] the queries' positions."""
    j = torch.arange(Nk, device=device)
    n = torch.full((B,), Nk, device=device) if k_len is None else k_len.long().clamp(0, Nk)
    start = n - Nq if q_start is None else torch.full((B,), q_start, device=device)
    p = start[:, None] + torch.arange(Nq, device=device)
    see = (j < n[:, None])[:, None].expand(B, Nq, Nk).clone()
    if doc_q is not None:
        see &= (doc_q[:, :, None] == doc_k[:, None]) & (doc_k >= 0)[:, None]
    if causal:
        ok = j <= p[:, :, None]
        if prefix is not None:
            ok = ok | (j < prefix[:, None])[:, None]
        see &= ok
    return see, p


def attend(Q, K, V, *, scale=None, softcap=0.0, causal=False, q_start=None, k_len=None, doc_q=None,
           doc_k=None, prefix=None, slopes=None):
    """(O, tolerance of O, lse, tolerance of lse)."""
    B, Hq, Nq, d = Q.shape
    Hk, Nk = K.shape[1], K.shape[2]
    scale = d ** -0.5 if scale is None else scale
    see, p = visible(B, Nq, Nk, Q.device, causal=causal, q_start=q_start, k_len=k_len,
                     doc_q=doc_q, doc_k=doc_k, prefix=prefix)
    # a key that no query may see does not count whatever it holds
    n = torch.full((B,), Nk, device=Q.device) if k_len is None else k_len.long().clamp(0, Nk)
    dead = torch.arange(Nk, device=Q.device) >= n[:, None]
    if doc_k is not None:
        dead = dead | (doc_k < 0)
    rep = Hq // Hk
    k = K.double().masked_fill(dead[:, None, :, None], 0.0).repeat_interleave(rep, 1)
    v = V.double().masked_fill(dead[:, None, :, None], 0.0).repeat_interleave(rep, 1)
    q = Q.double()
    x = q @ k.transpose(-1, -2) * scale
    # scores: d products accumulated by the tensor cores and a scale, relative to the terms' size
    es = (d + 8) * 2 * U32 * (q.abs() @ k.abs().transpose(-1, -2)) * scale
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
        es = es + 16 * U32 * softcap  # quotient, exponential, reciprocal and product of the cap
    if slopes is not None:
        bias = slopes.double()[None, :, None, None] * (p[:, None, :, None]
                                                       - torch.arange(Nk, device=Q.device)).abs()
        x = x - bias
        es = es + 4 * U32 * (x.abs() + bias)
    es = es + 4 * U32 * x.abs()
    x = x.masked_fill(~see[:, None], -math.inf)
    es = es.masked_fill(~see[:, None], 0.0).amax(-1) + 8 * U32  # and the exponential's own error
    lse = torch.logsumexp(x, -1)
    pr = torch.nan_to_num(torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]))
    pr = pr.masked_fill(~see[:, None], 0.0)
    o, size = pr @ v, pr @ v.abs()
    u = half_step(Q.dtype)
    # each probability off by its rounding and twice the worst score error (it is in the sum too),
    # Nk accumulation steps, then the output's rounding
    tol = u * o.abs() + (u + 2 * es[..., None] + (Nk + 64) * 2 * U32) * size * (1 + u) \
        + smallest(Q.dtype)
    ltol = torch.where(lse == -math.inf, 0.0, es + 4 * U32 * lse.abs() + (Nk / 32 + 64) * U32)
    return o, tol, lse, ltol


def project(X, W, bias, gate, R, act, Hy):
    """(Y, tolerance) with X [B, Hx, N, dx], Y [B, Hy, N, dy]."""
    B, Hx, N, dx = X.shape
    M, K = W.shape
    x = X.double().transpose(1, 2).reshape(B, N, K)
    t = x @ W.double().t()
    size = x.abs() @ W.double().abs().t()
    if bias is not None:
        t = t + bias.double()
        size = size + bias.double().abs()
    pre = t
    if act == "gelu":
        t = 0.5 * t * (1 + torch.erf(t / math.sqrt(2)))
    elif act == "gelu_tanh":
        t = 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    elif act == "silu":
        t = t * torch.sigmoid(t)
    # K accumulation steps, through an activation of slope at most 1.13, and its own evaluation
    err = 1.13 * (K + 4) * 2 * U32 * size + (16 * U32 * pre.abs() if act != "none" else 0.0)
    if gate is not None:
        g = gate.double()[:, None]
        t, err = t * g, (err + 2 * U32 * t.abs()) * g.abs()
    t = t.view(B, N, Hy, M // Hy).transpose(1, 2)
    err = err.view(B, N, Hy, M // Hy).transpose(1, 2)
    if R is not None:
        err = err + 2 * U32 * (t.abs() + R.double().abs())
        t = t + R.double()
    u = half_step(X.dtype)
    return t, u * t.abs() + err * (1 + u) + smallest(X.dtype)


def check(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite values differ"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]) or torch.isnan(want[~fin]).any(), what
    over = ((got - want).abs() - tol.expand_as(want))[fin]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} past the tolerance " \
                           f"by up to {worst:.3g}"
