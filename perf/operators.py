"""The operators around the sparse attention call, as they are measured.

Three operators of the attention block that a SparsePR call stands in:

* ``norm_rotate``: RMS norm of the queries and keys of each head and the rotary
  position embedding, in one pass over both tensors (what makes the call's Q
  and K out of the projections).
* ``attend_masked``: exact attention under a length, document, causal or prefix
  mask, with capped scores or a bias by distance (the layers and steps that stay
  dense, padded and packed batches, single query tokens over a long cache).
* ``project``: the projections in front of and behind the call, with bias,
  activation, gate and residual in the product's epilogue and either side in
  the call's head-major layout.

``run`` computes an operator in plain torch, or (``own``) through the public
entry points of ``free_block_sparse_means_b200``.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of a 24-head layer: the launch itself is the cost
        {"name": "nr_step", "op": "norm_rotate", "B": 1, "Hq": 24, "Hk": 24, "N": 1, "d": 128,
         "dtype": "bf16", "out": "bf16", "rot": 128, "pairing": "interleaved", "norm": True,
         "positions": True, "token_major": False},
        # the HunyuanVideo-shaped call's queries and keys, all 118,800 tokens of the latent grid
        {"name": "nr_hunyuan", "op": "norm_rotate", "B": 1, "Hq": 24, "Hk": 24, "N": 118800,
         "d": 128, "dtype": "bf16", "out": "bf16", "rot": 128, "pairing": "interleaved",
         "norm": True, "positions": False, "token_major": False},
        # a batch of ragged length with shared key heads, read as views of a token-major
        # projection, half of each head rotated in split halves
        {"name": "nr_ragged", "op": "norm_rotate", "B": 3, "Hq": 20, "Hk": 4, "N": 2049, "d": 64,
         "dtype": "fp16", "out": "fp16", "rot": 32, "pairing": "halves", "norm": True,
         "positions": True, "token_major": True},
        # one query token per sequence over a cache of 32,768 keys filled to different lengths
        {"name": "at_token", "op": "attend_masked", "B": 8, "Hq": 32, "Hk": 8, "Nq": 1,
         "Nk": 32768, "d": 128, "dtype": "bf16", "mask": "causal", "lens": True, "docs": 0,
         "softcap": 0.0, "bias": False, "lse": True},
        # a dense layer at half the sweep workload's length: every query against every key
        {"name": "at_dense", "op": "attend_masked", "B": 1, "Hq": 16, "Hk": 16, "Nq": 16384,
         "Nk": 16384, "d": 128, "dtype": "bf16", "mask": "none", "lens": False, "docs": 0,
         "softcap": 0.0, "bias": False, "lse": False},
        # clips of different lengths packed into two padded rows, no attention across clips
        {"name": "at_docs", "op": "attend_masked", "B": 2, "Hq": 24, "Hk": 24, "Nq": 5003,
         "Nk": 5003, "d": 128, "dtype": "bf16", "mask": "none", "lens": False, "docs": 6,
         "softcap": 0.0, "bias": False, "lse": True},
        # frame-by-frame generation after a bidirectional prompt, capped scores, shared key heads
        {"name": "at_prefix", "op": "attend_masked", "B": 2, "Hq": 16, "Hk": 4, "Nq": 4097,
         "Nk": 4097, "d": 64, "dtype": "fp16", "mask": "prefix", "lens": False, "docs": 0,
         "softcap": 30.0, "bias": False, "lse": False},
        # the mid workload's call with a penalty on the distance along the token order
        {"name": "at_distance", "op": "attend_masked", "B": 1, "Hq": 24, "Hk": 24, "Nq": 8192,
         "Nk": 8192, "d": 128, "dtype": "bf16", "mask": "none", "lens": False, "docs": 0,
         "softcap": 0.0, "bias": True, "lse": False},
        # the output projection of four single tokens of a 40-head layer: the weights are the cost
        {"name": "pj_step", "op": "project", "B": 4, "N": 1, "Hx": 40, "dx": 128, "Hy": 1,
         "dy": 5120, "dtype": "bf16", "act": "none", "bias": True, "gate": True, "residual": True},
        # the output projection behind the Wan-shaped call: 40 heads x 75,600 tokens, read head-major
        {"name": "pj_out", "op": "project", "B": 1, "N": 75600, "Hx": 40, "dx": 128, "Hy": 1,
         "dy": 5120, "dtype": "bf16", "act": "none", "bias": True, "gate": True, "residual": True},
        # queries, keys and values of 16 heads from one product, written head-major
        {"name": "pj_qkv", "op": "project", "B": 2, "N": 4095, "Hx": 1, "dx": 2048, "Hy": 48,
         "dy": 128, "dtype": "bf16", "act": "none", "bias": True, "gate": False,
         "residual": False},
        # the widening product of the block's feed-forward half
        {"name": "pj_ffn", "op": "project", "B": 1, "N": 2500, "Hx": 1, "dx": 2048, "Hy": 1,
         "dy": 8192, "dtype": "fp16", "act": "gelu_tanh", "bias": True, "gate": False,
         "residual": False},
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rotate", "attend_masked", "attend_masked", "project"])
    if op == "norm_rotate":
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 1, 2, 5])
        B = rng.choice([1, 1, 2, 3])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return {"op": op, "B": B, "Hq": Hq, "Hk": Hk,
                "N": _span(rng, 1, 118800 * 24 // (B * Hq) // 4), "d": d, "dtype": dtype,
                "out": rng.choice([dtype, "bf16"]), "rot": rng.choice([d, d, d // 2, 0]),
                "pairing": rng.choice(["interleaved", "halves"]), "norm": rng.random() < 0.85,
                "positions": rng.random() < 0.5, "token_major": rng.random() < 0.4}
    if op == "attend_masked":
        B = rng.choice([1, 2, 3, 5])
        Hk = rng.choice([1, 2, 4, 6])
        Hq = Hk * rng.choice([1, 1, 3, 4])
        kind = rng.choice(["few", "cross", "self", "self"])
        if kind == "few":
            Nq, Nk = _span(rng, 1, 40), _span(rng, 1, 60000)
        elif kind == "cross":
            Nq, Nk = _span(rng, 1, 6000), _span(rng, 1, 6000)
        else:
            Nq = Nk = _span(rng, 16, 7000)
        docs = rng.choice([0, 0, 1, 5, 17]) if kind == "self" else 0
        return {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "Nq": Nq, "Nk": Nk,
                "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "bf16", "fp16"]),
                "mask": rng.choice(["none", "causal", "prefix"]),
                "lens": kind != "self" and rng.random() < 0.6, "docs": docs,
                "softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "bias": rng.random() < 0.3,
                "lse": rng.random() < 0.5}
    d = rng.choice([64, 128])
    heads = rng.choice([2, 5, 12, 16, 24])
    side = rng.choice(["in", "out", "none"])
    wide, other = heads * d, 8 * _span(rng, 8, 900)
    B = rng.choice([1, 1, 2, 4])
    most = int(75600 * 5120 * 5120 / 8 / (wide * other * B))
    return {"op": op, "B": B, "N": _span(rng, 1, max(1, min(40000, most))),
            "Hx": heads if side == "in" else 1, "dx": d if side == "in" else other,
            "Hy": heads if side == "out" else 1,
            "dy": d if side == "out" else (other if side == "in" else 8 * _span(rng, 8, 900)),
            "dtype": rng.choice(["bf16", "bf16", "fp16"]), "act": rng.choice(ACTS),
            "bias": rng.random() < 0.7, "gate": rng.random() < 0.4,
            "residual": rng.random() < 0.5}


# --------------------------------------------------- masks a case describes
def _key_lengths(case):
    """[B] number of filled keys: the cache's whole length, then less for each sequence."""
    b = torch.arange(case["B"], dtype=torch.float64)
    part = 1.0 - 0.61 * b / max(1, case["B"])
    return (part * case["Nk"]).floor().clamp(min=1).to(torch.int32)


def _prefixes(case):
    """[B] length of the part that every query sees."""
    b = torch.arange(case["B"], dtype=torch.float64)
    return ((0.31 + 0.13 * b) % 1.0 * case["Nk"]).floor().to(torch.int32)


def _documents(case):
    """[B, N] document of each token; the last tokens of a row are padding (-1)."""
    B, N, n = case["B"], case["Nk"], case["docs"]
    valid = (N - (torch.arange(B, dtype=torch.float64) * 0.07 * N).floor() - N // 50)
    cuts = (valid[:, None] * (torch.arange(1, n + 1, dtype=torch.float64) / n) ** 1.4).floor()
    cuts[:, -1] = valid
    at = torch.arange(N, dtype=torch.float64).expand(B, N).contiguous()
    doc = torch.searchsorted(cuts.contiguous(), at, right=True)
    return torch.where(doc < n, doc, -1).to(torch.int32)


def _pairs(case):
    """Query-key pairs that the mask leaves, summed over the batch (one head)."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    klen = _key_lengths(case).double() if case["lens"] else torch.full((B,), Nk).double()
    i = torch.arange(Nq).double()
    hi = klen[:, None].expand(B, Nq)
    if case["mask"] != "none":
        hi = (klen[:, None] - Nq + i + 1).clamp(min=0)
        if case["mask"] == "prefix":
            hi = torch.maximum(hi, torch.minimum(_prefixes(case).double(), klen)[:, None])
    if not case["docs"]:
        return int(hi.sum())
    doc = _documents(case).long()
    n = case["docs"]
    size = torch.zeros(B, n + 1).double().scatter_add_(1, doc + 1, torch.ones(B, Nk).double())
    first = size[:, 1:].cumsum(1) - size[:, 1:]
    inside = doc.clamp(min=0)
    seen = torch.minimum(hi, (first + size[:, 1:]).gather(1, inside)) - first.gather(1, inside)
    return int((seen.clamp(min=0) * (doc >= 0)).sum())


# ------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _tokens(gen, B, H, N, d, dtype, token_major=False):
    """Rows around a few centres, as the tokens of a video have them, of unit size."""
    shape = (B, N, H, d) if token_major else (B, H, N, d)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    x += torch.randn((16, d), generator=gen, device=DEV)[torch.randint(
        0, 16, shape[:3], generator=gen, device=DEV)]
    x = x.mul_(0.7071).to(dtype)
    return x.transpose(1, 2) if token_major else x


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm_rotate":
        B, Hq, Hk, N, d, rot = (case[k] for k in ("B", "Hq", "Hk", "N", "d", "rot"))
        # trained queries and keys: uneven sizes from channel to channel
        s["q"] = _tokens(gen, B, Hq, N, d, dt, case["token_major"])
        s["k"] = _tokens(gen, B, Hk, N, d, dt, case["token_major"])
        s["wq"] = (1 + 0.3 * _normal(gen, (d,), torch.float32)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.3 * _normal(gen, (d,), torch.float32)).to(dt) if case["norm"] else None
        s["cos"] = s["sin"] = s["pos"] = None
        if rot:
            rows = N + 57 if case["positions"] else N
            at = torch.arange(rows, device=DEV, dtype=torch.float64)
            freq = 256.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
            s["cos"] = (at[:, None] * freq).cos().float()
            s["sin"] = (at[:, None] * freq).sin().float()
            if case["positions"]:
                s["pos"] = torch.randint(0, rows, (B, N), generator=gen, device=DEV,
                                         dtype=torch.int32)
        odt = TYPES[case["out"]]
        s["qo"] = torch.empty((B, Hq, N, d), device=DEV, dtype=odt)
        s["ko"] = torch.empty((B, Hk, N, d), device=DEV, dtype=odt)
        if own:
            import free_block_sparse_means_b200 as spr
            s["plan"] = spr.make_norm_rotate(s["q"], s["k"], s["qo"], s["ko"], norm=case["norm"],
                                             rot=rot, pairing=case["pairing"])
        return s
    if case["op"] == "attend_masked":
        B, Hq, Hk, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hk", "Nq", "Nk", "d"))
        s["q"] = _tokens(gen, B, Hq, Nq, d, dt)
        s["k"] = _tokens(gen, B, Hk, Nk, d, dt)
        s["v"] = _tokens(gen, B, Hk, Nk, d, dt)
        s["k_len"] = _key_lengths(case).to(DEV) if case["lens"] else None
        s["prefix"] = _prefixes(case).to(DEV) if case["mask"] == "prefix" else None
        s["doc"] = _documents(case).to(DEV) if case["docs"] else None
        s["slopes"] = None
        if case["bias"]:
            h = torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32)
            s["slopes"] = torch.exp2(-8.0 * h / Hq)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, Hq, Nq), device=DEV) if case["lse"] else None
        if own:
            import free_block_sparse_means_b200 as spr
            s["plan"] = spr.make_masked(s["q"], s["k"], s["v"], s["o"], softcap=case["softcap"],
                                        causal=case["mask"] != "none")
            s["ws"] = spr.alloc_workspace(s["plan"], device=DEV)
        return s
    B, N, Hx, dx, Hy, dy = (case[k] for k in ("B", "N", "Hx", "dx", "Hy", "dy"))
    K, M = Hx * dx, Hy * dy
    s["x"] = _tokens(gen, B, Hx, N, dx, dt)
    s["w"] = _normal(gen, (M, K), dt, K ** -0.5)
    s["bias"] = _normal(gen, (M,), dt, 0.2) if case["bias"] else None
    s["gate"] = _normal(gen, (B, M), dt, 0.5) if case["gate"] else None
    s["r"] = _normal(gen, (B, Hy, N, dy), dt) if case["residual"] else None
    s["y"] = torch.empty((B, Hy, N, dy), device=DEV, dtype=dt)
    if own:
        import free_block_sparse_means_b200 as spr
        s["plan"] = spr.make_project(s["x"], s["w"], s["y"], residual=s["r"], act=case["act"])
        s["ws"] = spr.alloc_workspace(s["plan"], device=DEV)
    return s


# --------------------------------------------------------------- plain forms
def _plain_norm_rotate(x, w, s, out):
    case = s["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot = case["rot"]
    if rot:
        cos, sin = s["cos"], s["sin"]
        if s["pos"] is not None:
            at = s["pos"].long()
            cos, sin = cos[at][:, None], sin[at][:, None]
        if case["pairing"] == "halves":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        x = torch.cat([turned, x[..., rot:]], -1)
    return x.to(TYPES[out])


def _plain_attend(s):
    case = s["case"]
    B, Hq, Hk, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hk", "Nq", "Nk", "d"))
    dev = s["q"].device
    q = (s["q"].float() * d ** -0.5).reshape(B, Hk, Hq // Hk * Nq, d)
    z = torch.matmul(q, s["k"].float().transpose(-1, -2)).view(B, Hq, Nq, Nk)
    if case["softcap"] > 0:
        z.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    klen = s["k_len"] if s["k_len"] is not None else torch.full((B,), Nk, device=dev)
    at = klen[:, None].long() - Nq + torch.arange(Nq, device=dev)  # position of each query
    j = torch.arange(Nk, device=dev)
    if s["slopes"] is not None:
        z.addcmul_(-s["slopes"].view(1, Hq, 1, 1),
                   (at[:, None, :, None] - j).abs().float())
    seen = (j < klen[:, None])[:, None, :]
    if case["mask"] != "none":
        past = j <= at[:, :, None]
        if s["prefix"] is not None:
            past = past | (j < s["prefix"][:, None])[:, None, :]
        seen = seen & past
    if s["doc"] is not None:
        seen = seen & (s["doc"][:, :, None] == s["doc"][:, None, :]) & (s["doc"] >= 0)[:, None, :]
    z.masked_fill_(~seen[:, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hk, Hq // Hk * Nq, Nk), s["v"].float()).view(B, Hq, Nq, d)
    o = torch.where(total > 0, o / total, 0.0).to(s["q"].dtype)
    lse = (top + total.log()).squeeze(-1) if case["lse"] else None
    return o, lse


def _plain_project(s):
    case = s["case"]
    B, N, Hx, dx, Hy, dy = (case[k] for k in ("B", "N", "Hx", "dx", "Hy", "dy"))
    x = s["x"].transpose(1, 2).reshape(B, N, Hx * dx).float()
    y = torch.matmul(x, s["w"].float().t())
    if s["bias"] is not None:
        y += s["bias"].float()
    if case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    elif case["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if s["gate"] is not None:
        y = y * s["gate"].float()[:, None]
    y = y.view(B, N, Hy, dy).transpose(1, 2)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["x"].dtype).contiguous()


def run(s):
    case = s["case"]
    if own:
        import free_block_sparse_means_b200 as spr
        if case["op"] == "norm_rotate":
            spr.sparsepr_norm_rotate(s["plan"], s["q"], s["k"], s["qo"], s["ko"], wq=s["wq"],
                                     wk=s["wk"], cos=s["cos"], sin=s["sin"], pos_q=s["pos"],
                                     pos_k=s["pos"])
            return s["qo"], s["ko"]
        if case["op"] == "attend_masked":
            spr.sparsepr_attend_masked(s["plan"], s["q"], s["k"], s["v"], s["o"], s["ws"],
                                       k_len=s["k_len"], prefix=s["prefix"], doc_q=s["doc"],
                                       doc_k=s["doc"], slopes=s["slopes"], lse=s["lse"])
            return s["o"], s["lse"]
        spr.sparsepr_project(s["plan"], s["x"], s["w"], s["y"], s["ws"], bias=s["bias"],
                             gate=s["gate"], residual=s["r"])
        return s["y"]
    if case["op"] == "norm_rotate":
        return (_plain_norm_rotate(s["q"], s["wq"], s, case["out"]),
                _plain_norm_rotate(s["k"], s["wk"], s, case["out"]))
    if case["op"] == "attend_masked":
        return _plain_attend(s)
    return _plain_project(s)


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm_rotate":
        B, Hq, Hk, N, d, rot = (case[k] for k in ("B", "Hq", "Hk", "N", "d", "rot"))
        size = 4 if case["dtype"] == "fp32" else 2
        size_out = 4 if case["out"] == "fp32" else 2
        n = B * (Hq + Hk) * N * d
        table = 4 * rot * N + (4 * B * N if case["positions"] and rot else 0)
        return {"bytes": n * (size + size_out) + table + (2 * d * size if case["norm"] else 0),
                "flops": n * (4 if case["norm"] else 0) + 3 * n * rot // d}
    if case["op"] == "attend_masked":
        B, Hq, Hk, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hk", "Nq", "Nk", "d"))
        keys = int(_key_lengths(case).sum()) if case["lens"] else B * Nk
        size = 2 * 2 * B * Hq * Nq * d + 2 * 2 * Hk * keys * d
        size += 4 * B * Hq * Nq if case["lse"] else 0
        size += 4 * B * Nk if case["docs"] else 0
        return {"bytes": size, "flops": 4 * d * Hq * _pairs(case)}
    rows, K, M = case["B"] * case["N"], case["Hx"] * case["dx"], case["Hy"] * case["dy"]
    size = rows * K + M * K + rows * M * (2 if case["residual"] else 1)
    size += (M if case["bias"] else 0) + (case["B"] * M if case["gate"] else 0)
    return {"bytes": 2 * size, "flops": 2 * rows * K * M}


# -------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm_rotate":
        return _exact_turn(s, "q", "wq"), _exact_turn(s, "k", "wk")
    return _exact_attend(s) if case["op"] == "attend_masked" else _exact_project(s)


def _exact_turn(s, x, w):
    """Pairs as complex numbers, turned by e^(i angle)."""
    case = s["case"]
    out = torch.empty(s[x].shape, device=DEV, dtype=torch.float64)
    at = torch.arange(case["N"], device=DEV) if s["pos"] is None else s["pos"].long()
    rot = case["rot"]
    for b in range(case["B"]):
        for h in range(out.shape[1]):
            y = s[x][b, h].double()
            if case["norm"]:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["d"] + 1e-6)
                y = y * s[w].double()
            if rot:
                row = at[b] if at.dim() == 2 else at
                turn = torch.complex(s["cos"].double()[row], s["sin"].double()[row])
                if case["pairing"] == "halves":
                    z = torch.complex(y[:, :rot // 2].contiguous(), y[:, rot // 2:rot].contiguous())
                    z = z * turn
                    y[:, :rot // 2], y[:, rot // 2:rot] = z.real, z.imag
                else:
                    z = torch.view_as_complex(y[:, :rot].reshape(-1, rot // 2, 2).contiguous())
                    y[:, :rot] = torch.view_as_real(z * turn).reshape(-1, rot)
            out[b, h] = y
    return out


def _exact_attend(s):
    case = s["case"]
    B, Hq, Hk, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hk", "Nq", "Nk", "d"))
    o = torch.zeros((B, Hq, Nq, d), device=DEV, dtype=torch.float64)
    lse = torch.full((B, Hq, Nq), -math.inf, device=DEV, dtype=torch.float64)
    j = torch.arange(Nk, device=DEV)
    for b in range(B):
        n = int(s["k_len"][b]) if s["k_len"] is not None else Nk
        for h in range(Hq):
            k, v = s["k"][b, h // (Hq // Hk)].double(), s["v"][b, h // (Hq // Hk)].double()
            for i0 in range(0, Nq, 4096):
                i1 = min(Nq, i0 + 4096)
                pos = torch.arange(i0, i1, device=DEV)[:, None] + (n - Nq)
                x = s["q"][b, h, i0:i1].double() @ k.t() / math.sqrt(d)
                if case["softcap"] > 0:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (pos - j).abs()
                hide = (j >= n).expand(i1 - i0, Nk)
                if case["mask"] == "causal":
                    hide = hide | (j > pos)
                if case["mask"] == "prefix":
                    hide = hide | ((j > pos) & (j >= s["prefix"][b]))
                if s["doc"] is not None:
                    doc = s["doc"][b]
                    hide = hide | (doc[i0:i1, None] != doc[None]) | (doc[None] < 0)
                x = torch.where(hide, -math.inf, x)
                lse[b, h, i0:i1] = torch.logsumexp(x, -1)
                o[b, h, i0:i1] = torch.nan_to_num(torch.softmax(x, -1), nan=0.0) @ v
    return o, (lse if case["lse"] else None)


def _exact_project(s):
    case = s["case"]
    B, N, Hx, dx, Hy, dy = (case[k] for k in ("B", "N", "Hx", "dx", "Hy", "dy"))
    y = torch.empty((B, Hy, N, dy), device=DEV, dtype=torch.float64)
    w = s["w"].double().view(Hy * dy, Hx, dx)
    for b in range(B):
        for n0 in range(0, N, 8192):
            n1 = min(N, n0 + 8192)
            t = torch.einsum("hnd,mhd->nm", s["x"][b, :, n0:n1].double(), w)
            if s["bias"] is not None:
                t = t + s["bias"].double()
            if case["act"] == "gelu":
                t = t * torch.special.ndtr(t)
            elif case["act"] == "gelu_tanh":
                t = t * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
            elif case["act"] == "silu":
                t = t * torch.sigmoid(t)
            if s["gate"] is not None:
                t = t * s["gate"][b].double()
            t = t.view(n1 - n0, Hy, dy).transpose(0, 1)
            y[b, :, n0:n1] = t if s["r"] is None else t + s["r"][b, :, n0:n1].double()
    return y
