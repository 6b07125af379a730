"""The attention half of a transformer block: projections, norm and rotation, attention.

AttentionBlock runs the operators of this package in the order a model uses them, on buffers it
keeps: one product makes queries, keys and values head by head, one pass norms and rotates queries
and keys, the sparse call or masked attention follows, and the output projection adds its gated
result to the residual.  Nothing is transposed or copied in between.

Errors that a call meets on the device (a position outside the tables, a wait that gave up) are
kept until check() is asked.

With a cache, keys and values go to their places behind those of earlier calls and every call
attends to all of them, so that a prompt and the frames or tokens after it take the same path.
"""
from __future__ import annotations

import torch

from . import _binding as spr
from .operators import (make_masked, make_norm_rotate, make_project, sparsepr_attend_masked,
                        sparsepr_norm_rotate, sparsepr_project)


class AttentionBlock:
    """Buffers and parameters of the attention of x [B, N, C] with `heads` query heads of d channels.

    w_qkv: [(heads + 2 kv_heads) d, C], the rows of the query heads, then of the key and the value
    heads; w_out: [C, heads d]; b_qkv, b_out: their biases or None; wq, wk: [d] norm weights or
    None (ones).  All of one 16-bit type; they are used in place, so they may be changed between
    calls.

    sparse: a dict of make_params options selects the sparse call (bf16, as many key heads as query
    heads, no masks); otherwise the attention is dense with softcap, causal and slopes as given.
    cache: number of tokens the keys and values of earlier calls are kept for (dense only, causal by
    position), or another AttentionBlock to share the cache of (blocks for calls of other lengths).
    """

    def __init__(self, shape, heads, d, w_qkv, w_out, *, kv_heads=None, b_qkv=None, b_out=None,
                 wq=None, wk=None, norm=True, eps=1e-6, rot=None, pairing="interleaved",
                 sparse=None, cache=0, softcap=0.0, causal=False, slopes=None):
        B, N, C = shape
        kv = heads if kv_heads is None else int(kv_heads)
        if sparse is not None and (cache or softcap or causal or slopes is not None or kv != heads):
            raise ValueError("the sparse call takes no mask, cap, bias, cache or shared key heads")
        if tuple(w_qkv.shape) != ((heads + 2 * kv) * d, C):
            raise ValueError(f"w_qkv must have shape {((heads + 2 * kv) * d, C)}, got "
                             f"{tuple(w_qkv.shape)}")
        shared = cache if isinstance(cache, AttentionBlock) else None
        if shared is not None:
            cache = shared.cache
            if not cache or (shared.shape[0], shared.kv_heads, shared.d) != (B, kv, d) or \
                    shared.keys.dtype != w_qkv.dtype or shared.keys.device != w_qkv.device:
                raise ValueError("a shared cache must be one of the same batch, key heads, d, type "
                                 "and device")
        if cache and cache < N:
            raise ValueError(f"a cache of {cache} tokens is too short for calls of {N}")
        if sparse is not None and w_qkv.dtype is not torch.bfloat16:
            raise ValueError("the sparse call is bf16")
        self.shape, self.heads, self.kv_heads, self.d = (B, N, C), heads, kv, d
        self.w_qkv, self.w_out, self.b_qkv, self.b_out = w_qkv, w_out, b_qkv, b_out
        self.wq, self.wk, self.slopes = wq, wk, slopes
        self.sparse, self.cache = sparse, int(cache)
        dev, dt = w_qkv.device, w_qkv.dtype

        def empty(*size):
            return torch.empty(size, device=dev, dtype=dt)

        # queries and keys (and, without a cache, the values) of one product
        own = heads + kv + (0 if cache else kv)
        self.qkv = empty(B, own, N, d)
        self.q, self.k = self.qkv[:, :heads], self.qkv[:, heads:heads + kv]
        self.o = empty(B, heads, N, d)
        x = y = empty(B, 1, N, C)
        rows = own * d
        self._w_own, self._w_v = w_qkv[:rows], w_qkv[rows:]
        self._p_in = make_project(x, self._w_own, self.qkv)
        if cache:
            self.keys = shared.keys if shared else empty(B, kv, cache, d)
            self.values = shared.values if shared else empty(B, kv, cache, d)
            self.k_len = torch.zeros(B, device=dev, dtype=torch.int32)
            k_to, v_to = self.keys[:, :, :N], self.values[:, :, :N]
            self._p_v = make_project(x, self._w_v, v_to)
        else:
            k_to, self.keys, self.values = self.k, self.k, self.qkv[:, heads + kv:]
            self.k_len = self._p_v = None
        self._rotate = make_norm_rotate(self.q, self.k, self.q, k_to, norm=norm, eps=eps, rot=rot,
                                        pairing=pairing)
        if sparse is not None:
            self._attend = spr.make_params(self.q, self.keys, self.values, self.o, **sparse)
        else:
            # token n sits at position n, also in a batch of which only k_len tokens are real; with
            # a cache the call's tokens are its last ones
            self._attend = make_masked(self.q, self.keys, self.values, self.o, softcap=softcap,
                                       causal=causal or bool(cache), q_start=None if cache else 0)
        self._p_out = make_project(self.o, w_out, y, residual=x)
        # the steps of a call follow one another, so one workspace serves them all but the sparse
        # call, which may keep centroids in its own for the next call
        made = [self._p_in, self._p_out] + [p for p in (self._p_v,) if p is not None]
        if sparse is None:
            made.append(self._attend)
        self.ws = max((spr.alloc_workspace(p, device=dev) for p in made), key=lambda t: t.numel())
        self.ws_sparse = None if sparse is None else spr.alloc_workspace(self._attend, device=dev)
        # the status of norm + rotation's last call with positions, and the first error of all of them
        self._rotated = torch.zeros(4, device=dev, dtype=torch.int32)
        self.status = torch.zeros(4, device=dev, dtype=torch.int32)
        self._called = False

    def __call__(self, x, cos=None, sin=None, *, at=0, positions=None, gate=None, residual=None,
                 k_len=None, doc=None, prefix=None, out=None):
        """out = residual + gate * (attention(x) w_out^T + b_out); [B, N, C].

        cos, sin: tables of the rotation; positions: [B, N] table rows (default: token n takes row
        n, with a cache row at + n; a row outside the tables is an error that check() raises); at: number of tokens already in the cache; gate: [B, C];
        k_len, prefix: [B] and doc: [B, N], the masks of sparsepr_attend_masked (k_len and doc not
        with a cache).  Token n is at position n, with a cache at + n, for the causal mask and the
        slopes.  The tokens of a frame see one another and all before them with prefix = at + N.
        """
        B, N, C = self.shape
        if tuple(x.shape) != self.shape or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous {self.shape} tensor")
        if self.sparse is not None and (k_len is not None or doc is not None or prefix is not None):
            raise ValueError("the sparse call takes no mask")
        if self.cache and (k_len is not None or doc is not None):
            raise ValueError("with a cache, the keys of a call are those of its tokens so far")
        if self.cache and not 0 <= at <= self.cache - N:
            raise ValueError(f"at must leave room for {N} of {self.cache} tokens, got {at}")
        if not self.cache and at:
            raise ValueError("at needs a cache")
        if self._rotate.rot:
            if cos is None or sin is None:
                raise ValueError("rotation needs cos and sin")
            if positions is None and min(cos.shape[0], sin.shape[0]) < at + N:
                raise ValueError(f"the tables must have {at + N} rows or more")
        for name, t in (("residual", residual), ("out", out)):
            if t is not None and (tuple(t.shape) != self.shape or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {self.shape} tensor")
        if out is None:
            out = torch.empty_like(x)
        x4, y4 = x.view(B, 1, N, C), out.view(B, 1, N, C)
        b_own = b_v = None
        if self.b_qkv is not None:
            rows = self._w_own.shape[0]
            b_own, b_v = self.b_qkv[:rows], self.b_qkv[rows:]
        sparsepr_project(self._p_in, x4, self._w_own, self.qkv, self.ws, bias=b_own)
        k_to = self.k
        if self.cache:
            k_to, v_to = self.keys[:, :, at:at + N], self.values[:, :, at:at + N]
            sparsepr_project(self._p_v, x4, self._w_v, v_to, self.ws, bias=b_v)
            k_len = self.k_len.fill_(at + N)
            if positions is None and self._rotate.rot and at:
                cos, sin = cos[at:], sin[at:]
        # (rows that are not given are inside the tables, as checked above)
        given = positions is not None and bool(self._rotate.rot)
        sparsepr_norm_rotate(self._rotate, self.q, self.k, self.q, k_to, wq=self.wq, wk=self.wk,
                             cos=cos, sin=sin, pos_q=positions, pos_k=positions,
                             status=self._rotated if given else None)
        if given:
            torch.where(self.status[:1] != 0, self.status, self._rotated, out=self.status)
        self._called = True
        if self.sparse is not None:
            with torch.cuda.device(x.device):  # the call itself takes the current one
                spr.sparsepr_call(self._attend, self.q, self.keys, self.values, self.o,
                                  self.ws_sparse)
        else:
            sparsepr_attend_masked(self._attend, self.q, self.keys, self.values, self.o, self.ws,
                                   k_len=k_len, doc_q=doc, doc_k=doc, prefix=prefix,
                                   slopes=self.slopes)
        sparsepr_project(self._p_out, self.o, self.w_out, y4, self.ws, bias=self.b_out, gate=gate,
                         residual=None if residual is None else residual.view(B, 1, N, C))
        return out

    def check(self):
        """Wait for the block's calls so far and raise SparsePRError if one of them met an error on the
        device; the error is then forgotten.

        A token whose position is outside the tables has a query without norm and rotation and, in
        the cache, whatever key was there: results that see it are not valid, nor are those of other
        blocks on the same cache.  After a wait that gave up the output of that call is not whole.
        """
        code, b, n, row = self.status.tolist()
        waited = spr.sparsepr_workspace_error(self.ws)
        self.status.zero_()
        self.ws[:16].zero_()
        met = [f"position {row} of token {n}, batch {b}, is not a row of the tables"] * bool(code) \
            + ["a wait gave up"] * bool(waited)
        if met:
            raise spr.SparsePRError("AttentionBlock: " + "; ".join(met), spr.SPR_EDEVICE)
        if self.sparse is not None and self._called:
            with torch.cuda.device(self.ws_sparse.device):
                spr.sparsepr_get_stats(self._attend, self.ws_sparse)
