"""The operators around the call: norm + rotation, masked attention, projection.

Argument checks and marshalling only; the contract of each is in
include/sparsepr.h.  Every function takes its output tensors from the caller,
enqueues on `stream` (default: the current stream of the tensors' device) and
returns without waiting.  They are forward only: a call whose inputs require a
gradient while gradients are enabled, or carry a forward-mode tangent, is refused.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from ._binding import (SprMaskedParams, SprNormRotateParams, SprProjectParams, _check,
                       load_library, load_marshal)

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
PAIRINGS = {"interleaved": 0, "halves": 1}
ACTS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}
ALIGN_END = -2 ** 31
INT32_MAX = 2 ** 31 - 1


def _dims(name, t):
    """(shape, strides) of a [B, H, N, d] tensor; a dimension of one entry gets the stride of a
    contiguous tensor, so that whatever torch keeps there does not matter."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be a 4-dimensional tensor, got {tuple(t.shape)}")
    if max(t.shape) > INT32_MAX:
        raise ValueError(f"{name} has more than 2^31 - 1 entries in a dimension: {tuple(t.shape)}")
    B, H, N, d = t.shape
    if d > 1 and t.stride(3) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    sn = t.stride(2) if N > 1 else d
    sh = t.stride(1) if H > 1 else N * sn
    sb = t.stride(0) if B > 1 else H * sh
    return (B, H, N, d), (sb, sh, sn)


def _dtype(name, t, allowed=DTYPES):
    if t.dtype not in allowed:
        raise ValueError(f"{name} must be one of {[str(a) for a in allowed]}, got {t.dtype}")
    return DTYPES[t.dtype]


def _option(name, value, table):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, not {value!r}")
    return table[value]


def _single(name, value):
    """A number for a field whose 0 has a meaning of its own: one that fp32 rounds to 0 is refused."""
    value = float(value)
    if value and not ctypes.c_float(value).value:
        raise ValueError(f"{name} = {value} is 0 in fp32")
    return value


def _made(prm, kind, where, *tensors):
    """Keep with the parameters a plan of their calls: what the tensors they were made for look
    like.  A call with such tensors is checked and made by the extension module in one step; any
    other call, also one whose parameters were changed since, goes through the checks below."""
    entry = ctypes.cast(getattr(load_library(), where), ctypes.c_void_p).value
    prm.plan = load_marshal().plan(kind, ctypes.addressof(prm), ctypes.sizeof(prm), entry, tensors)
    return prm


def _planned(where, prm, *args):
    """Make the call by its plan; False where the checks have to decide."""
    plan = prm.__dict__.get("plan")
    status = -1 if plan is None else _call(plan, ctypes.addressof(prm), *args)
    if status > 0:
        _check(where, status)
    return status == 0


def _call(*args):
    global _call
    _call = load_marshal().call
    return _call(*args)


def _same(name, t, prm, shape_fields, stride_field, dtype):
    """Check that a tensor is the one its parameters were made for."""
    shape, strides = _dims(name, t)
    want = tuple(getattr(prm, f) for f in shape_fields)
    if shape != want:
        raise ValueError(f"{name} must have shape {want}, got {shape}")
    if strides != tuple(getattr(prm, stride_field)):
        raise ValueError(f"{name} must have the strides its parameters were made with")
    if DTYPES.get(t.dtype) != dtype:
        raise ValueError(f"{name} has type {t.dtype}, not the one its parameters were made with")


def _aux(name, t, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(ws):
    """A workspace is as large as its elements say only where they lie one after the other."""
    if not isinstance(ws, torch.Tensor):
        raise ValueError("ws must be a torch tensor")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run(where, tensors, names, stream, call, *args):
    """Check where the tensors live (the first one decides) and make the call there."""
    index = tensors[0].get_device()
    grad = torch.is_grad_enabled()
    dual = getattr(forward_ad, "_current_level", 0) >= 0  # 0.8 us a tensor to look, so only then
    astray = None
    for i, t in enumerate(tensors):
        if t is not None:
            if grad and t.requires_grad:
                raise ValueError(f"{where} has no backward pass; {names.split()[i]} requires a "
                                 "gradient (call it under torch.no_grad())")
            if dual and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{where} has no derivative; {names.split()[i]} carries a tangent")
            if t.get_device() != index:
                astray = i
    if index < 0 or astray is not None:
        name = names.split()[astray or 0]
        raise ValueError(f"{name} must be on {tensors[0].device}" if index >= 0 else
                         f"{names.split()[0]} must be on a CUDA device")
    if stream is None:
        stream = torch.cuda.current_stream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream must be one of {tensors[0].device}")
    if index == torch.cuda.current_device():
        _check(where, call(*args, stream.cuda_stream))
    else:
        with torch.cuda.device(index):
            _check(where, call(*args, stream.cuda_stream))


# ------------------------------------------------------------ norm + rotation
def make_norm_rotate(Q, K, Qo, Ko, *, eps=1e-6, norm=True, rot=None,
                     pairing="interleaved") -> SprNormRotateParams:
    """spr_norm_rotate_params for queries [B, Hq, Nq, d] and keys [B, Hk, Nk, d] (None: queries
    only) and their outputs; rot: rotated channels (default all d, 0 none)."""
    prm = SprNormRotateParams()
    (B, Hq, Nq, d), prm.q_strides[:] = _dims("Q", Q)
    shape, prm.qo_strides[:] = _dims("Qo", Qo)
    if shape != (B, Hq, Nq, d):
        raise ValueError(f"Qo must have shape {(B, Hq, Nq, d)}, got {shape}")
    prm.B, prm.Hq, prm.Nq, prm.d = B, Hq, Nq, d
    prm.dtype_in, prm.dtype_out = _dtype("Q", Q), _dtype("Qo", Qo)
    if (K is None) != (Ko is None):
        raise ValueError("K and Ko go together")
    if K is not None:
        shape, prm.k_strides[:] = _dims("K", K)
        if shape[0] != B or shape[3] != d:
            raise ValueError(f"K must have shape [{B}, Hk, Nk, {d}], got {shape}")
        out, prm.ko_strides[:] = _dims("Ko", Ko)
        if out != shape:
            raise ValueError(f"Ko must have shape {shape}, got {out}")
        if K.dtype != Q.dtype or Ko.dtype != Qo.dtype:
            raise ValueError("keys must have the queries' types")
        prm.Hk, prm.Nk = shape[1], shape[2]
    prm.norm, prm.eps = int(bool(norm)), float(eps)
    prm.rot = d if rot is None else int(rot)
    if rot is not None and not 0 <= int(rot) <= d:
        raise ValueError(f"rot must be 0..{d}, got {rot}")
    prm.pairing = _option("pairing", pairing, PAIRINGS)
    return _made(prm, 0, "sparsepr_norm_rotate", Q, K, Qo, Ko)


def sparsepr_norm_rotate(prm, Q, K, Qo, Ko, wq=None, wk=None, cos=None, sin=None, pos_q=None,
                         pos_k=None, status=None, stream=None):
    """RMS norm of each head's queries and keys and the rotary embedding, one pass.

    wq, wk: [d] weights of the inputs' type (None: ones); cos, sin: [rows, rot / 2] fp32 tables;
    pos_q, pos_k: [B, N] int32 table row of each token (None: token n takes row n); status:
    optional int32[4] device tensor.  Qo may be Q and Ko may be K.
    """
    if _planned("sparsepr_norm_rotate", prm, Q, K, Qo, Ko, wq, wk, cos, sin, pos_q, pos_k, status,
                stream):
        return
    _same("Q", Q, prm, ("B", "Hq", "Nq", "d"), "q_strides", prm.dtype_in)
    _same("Qo", Qo, prm, ("B", "Hq", "Nq", "d"), "qo_strides", prm.dtype_out)
    if prm.Hk:
        _same("K", K, prm, ("B", "Hk", "Nk", "d"), "k_strides", prm.dtype_in)
        _same("Ko", Ko, prm, ("B", "Hk", "Nk", "d"), "ko_strides", prm.dtype_out)
    elif K is not None or Ko is not None or wk is not None or pos_k is not None:
        raise ValueError("the parameters were made without keys")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _aux(name, w, Q.dtype, (prm.d,))
    rows = 0
    if prm.rot:
        if cos is None or sin is None:
            raise ValueError("rotation needs cos and sin")
        rows = cos.shape[0] if isinstance(cos, torch.Tensor) and cos.dim() == 2 else -1
        _aux("cos", cos, torch.float32, (rows, prm.rot // 2))
        _aux("sin", sin, torch.float32, (rows, prm.rot // 2))
    for name, p, n in (("pos_q", pos_q, prm.Nq), ("pos_k", pos_k, prm.Nk)):
        if p is not None:
            _aux(name, p, torch.int32, (prm.B, n))
    if status is not None:
        _aux("status", status, torch.int32, (4,))
    _run("sparsepr_norm_rotate", (Q, K, Qo, Ko, wq, wk, cos, sin, pos_q, pos_k, status),
         "Q K Qo Ko wq wk cos sin pos_q pos_k status", stream,
         load_library().sparsepr_norm_rotate, ctypes.byref(prm), Q.data_ptr(), _ptr(K), _ptr(wq),
         _ptr(wk), _ptr(cos), _ptr(sin), rows, _ptr(pos_q), _ptr(pos_k), Qo.data_ptr(), _ptr(Ko),
         _ptr(status))


# ----------------------------------------------------------- masked attention
def make_masked(Q, K, V, O, *, scale=0.0, softcap=0.0, causal=False,
                q_start=None) -> SprMaskedParams:
    """spr_masked_params for Q, O [B, Hq, Nq, d] and K, V [B, Hk, Nk, d]; q_start: position of
    the first query (default: the last query sits on each batch's last key)."""
    prm = SprMaskedParams()
    (B, Hq, Nq, d), prm.q_strides[:] = _dims("Q", Q)
    shape, prm.k_strides[:] = _dims("K", K)
    if shape[0] != B or shape[3] != d:
        raise ValueError(f"K must have shape [{B}, Hk, Nk, {d}], got {shape}")
    vshape, prm.v_strides[:] = _dims("V", V)
    if vshape != shape:
        raise ValueError(f"V must have shape {shape}, got {vshape}")
    oshape, prm.o_strides[:] = _dims("O", O)
    if oshape != (B, Hq, Nq, d):
        raise ValueError(f"O must have shape {(B, Hq, Nq, d)}, got {oshape}")
    prm.B, prm.Hq, prm.Hk, prm.Nq, prm.Nk, prm.d = B, Hq, shape[1], Nq, shape[2], d
    prm.dtype = _dtype("Q", Q, (torch.bfloat16, torch.float16))
    for name, t in (("K", K), ("V", V), ("O", O)):
        if t.dtype != Q.dtype:
            raise ValueError(f"{name} must be {Q.dtype}, got {t.dtype}")
    prm.scale, prm.softcap = _single("scale", scale), _single("softcap", softcap)
    prm.causal = int(bool(causal))
    if q_start is not None and abs(int(q_start)) > 1 << 30:
        raise ValueError(f"q_start must be -2^30..2^30, got {q_start}")
    prm.q_start = ALIGN_END if q_start is None else int(q_start)
    return _made(prm, 1, "sparsepr_attend_masked", Q, K, V, O)


def sparsepr_attend_masked(prm, Q, K, V, O, ws, k_len=None, doc_q=None, doc_k=None, prefix=None,
                           slopes=None, lse=None, status=None, stream=None):
    """Exact attention under a length, document, causal or prefix mask, with capped scores or a
    bias by distance.

    k_len, prefix: [B] int32; doc_q, doc_k: [B, Nq], [B, Nk] int32 (negative: padding); slopes:
    [Hq] fp32; lse: [B, Hq, Nq] fp32 output; status: optional int32[4].  Rows that see no key are
    zero (lse -inf).
    """
    if _planned("sparsepr_attend_masked", prm, Q, K, V, O, ws, k_len, doc_q, doc_k, prefix, slopes,
                lse, status, stream):
        return
    _same("Q", Q, prm, ("B", "Hq", "Nq", "d"), "q_strides", prm.dtype)
    _same("K", K, prm, ("B", "Hk", "Nk", "d"), "k_strides", prm.dtype)
    _same("V", V, prm, ("B", "Hk", "Nk", "d"), "v_strides", prm.dtype)
    _same("O", O, prm, ("B", "Hq", "Nq", "d"), "o_strides", prm.dtype)
    i32 = torch.int32
    for name, t in (("k_len", k_len), ("prefix", prefix)):
        if t is not None:
            _aux(name, t, i32, (prm.B,))
    if doc_q is not None:
        _aux("doc_q", doc_q, i32, (prm.B, prm.Nq))
    if doc_k is not None:
        _aux("doc_k", doc_k, i32, (prm.B, prm.Nk))
    if slopes is not None:
        _aux("slopes", slopes, torch.float32, (prm.Hq,))
    if lse is not None:
        _aux("lse", lse, torch.float32, (prm.B, prm.Hq, prm.Nq))
    if status is not None:
        _aux("status", status, i32, (4,))
    _workspace(ws)
    if (doc_q is None) != (doc_k is None):
        raise ValueError("doc_q and doc_k go together")
    if prefix is not None and not prm.causal:
        raise ValueError("a prefix needs causal=True")
    _run("sparsepr_attend_masked", (Q, K, V, k_len, doc_q, doc_k, prefix, slopes, O, lse, ws, status),
         "Q K V k_len doc_q doc_k prefix slopes O lse ws status", stream,
         load_library().sparsepr_attend_masked, ctypes.byref(prm), Q.data_ptr(), K.data_ptr(),
         V.data_ptr(), _ptr(k_len), _ptr(doc_q), _ptr(doc_k), _ptr(prefix), _ptr(slopes),
         O.data_ptr(), _ptr(lse), ws.data_ptr(), ws.nbytes, _ptr(status))


# ----------------------------------------------------------------- projection
def make_project(X, W, Y, *, residual=None, act="none") -> SprProjectParams:
    """spr_project_params for X [B, Hx, N, dx], W [Hy * dy, Hx * dx] and Y [B, Hy, N, dy]
    (one head: plain rows); residual: a tensor of Y's shape whose strides the call will use."""
    prm = SprProjectParams()
    (B, Hx, N, dx), prm.x_strides[:] = _dims("X", X)
    (By, Hy, Ny, dy), prm.y_strides[:] = _dims("Y", Y)
    if (By, Ny) != (B, N):
        raise ValueError(f"Y must have shape [{B}, Hy, {N}, dy], got {tuple(Y.shape)}")
    if not isinstance(W, torch.Tensor) or tuple(W.shape) != (Hy * dy, Hx * dx):
        raise ValueError(f"W must be a [{Hy * dy}, {Hx * dx}] tensor")
    if Hx * dx > 1 and W.stride(1) != 1:
        raise ValueError("W must have a contiguous last dimension")
    r = Y if residual is None else residual
    shape, prm.r_strides[:] = _dims("residual", r)
    if shape != (B, Hy, N, dy):
        raise ValueError(f"residual must have shape {(B, Hy, N, dy)}, got {shape}")
    prm.B, prm.N, prm.Hx, prm.dx, prm.Hy, prm.dy = B, N, Hx, dx, Hy, dy
    prm.w_stride = W.stride(0) if W.shape[0] > 1 else Hx * dx
    prm.dtype = _dtype("X", X, (torch.bfloat16, torch.float16))
    for name, t in (("W", W), ("Y", Y), ("residual", r)):
        if t.dtype != X.dtype:
            raise ValueError(f"{name} must be {X.dtype}, got {t.dtype}")
    prm.act = _option("act", act, ACTS)
    return _made(prm, 2, "sparsepr_project", X, W, Y, residual)


def sparsepr_project(prm, X, W, Y, ws, bias=None, gate=None, residual=None, status=None,
                     stream=None):
    """Y = residual + gate * act(X W^T + bias), either side row-major or head-major.

    bias: [M]; gate: [B, M]; residual: Y's shape (may be Y itself); all of X's type.  status:
    optional int32[4].
    """
    if _planned("sparsepr_project", prm, X, W, Y, ws, bias, gate, residual, status, stream):
        return
    _same("X", X, prm, ("B", "Hx", "N", "dx"), "x_strides", prm.dtype)
    _same("Y", Y, prm, ("B", "Hy", "N", "dy"), "y_strides", prm.dtype)
    M, K = prm.Hy * prm.dy, prm.Hx * prm.dx
    if not isinstance(W, torch.Tensor) or W.dtype != X.dtype or tuple(W.shape) != (M, K) or \
            (K > 1 and W.stride(1) != 1) or (M > 1 and W.stride(0) != prm.w_stride):
        raise ValueError("W must be the tensor its parameters were made with")
    if residual is not None:
        _same("residual", residual, prm, ("B", "Hy", "N", "dy"), "r_strides", prm.dtype)
    _workspace(ws)
    for name, t, shape in (("bias", bias, (M,)), ("gate", gate, (prm.B, M))):
        if t is not None:
            _aux(name, t, X.dtype, shape)
    if status is not None:
        _aux("status", status, torch.int32, (4,))
    _run("sparsepr_project", (X, W, bias, gate, residual, Y, ws, status),
         "X W bias gate residual Y ws status", stream,
         load_library().sparsepr_project, ctypes.byref(prm), X.data_ptr(), W.data_ptr(), _ptr(bias),
         _ptr(gate), _ptr(residual), Y.data_ptr(), ws.data_ptr(), ws.nbytes, _ptr(status))
