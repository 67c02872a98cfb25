"""Cases of the operators around the row operators: embedding lookup, head norms with the position
rotation, and activation checkpoints in 8 bits with the backward passes that read them.

With u(r, c) = uniform of word start + r cols + c of the key's stream, q = 1 - p and
drop(v) = u >= p ? v / q : 0:

    embedding         y[r] = drop(scale table[ids[r]]), zeros where the id is no row of the table
      backward        dtable[v] = scale (sum of drop(dy[r]) over the rows r whose id is v)
    head_norm_rotate  each head x of a token's queries and keys: n = x gamma / sqrt(mean(x^2) + eps), and
                      its pairs (a, b) turned by the token's angles: (a cos - b sin, b cos + a sin);
                      a position that is no row of the tables turns nothing
      backward        g = the gradient turned back, h = x rstd: dgamma = sums of g h over tokens and
                      heads, dx = rstd (g gamma - h mean(g gamma h))
    checkpoint        blocks of 128 columns, m = max |x|: scale = m / 127 and inverse = 127 / m as floats,
                      t = |x| inverse as a float, code = sign(x) min(127, floor(t) + (u < t - floor(t)))
      restore         code scale
      backward        layer norm's and dropout-add-layer-norm's gradients at the sum code scale

`run` computes these in elementary torch operations, or with the library's calls where
`own` is set; `exact` computes them in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
BLOCK = 128  # columns of a checkpoint's scale

# Just under the bytes of the largest listed case.
MOST = 6.1e8


def _lookup(name, way, type, rows, cols, vocab, ids="zipf", p=0.0, scale=1.0, res32=False, params32=False, ids64=True,
            padded=0.0, pad=0):
    """res32: the rows (y, dy) are float; params32: the table and its gradient are; ids: how the
    tokens are spread over the vocabulary; padded: the share of rows without a token; pad:
    elements between the rows."""
    c = {"op": "embedding", "way": way, "type": type, "rows": rows, "cols": cols, "vocab": vocab, "ids": ids, "p": p,
         "scale": scale, "res32": res32, "params32": params32, "ids64": ids64, "padded": padded, "pad": pad}
    return {"name": name, **c} if name else c


def _heads(name, way, type, rows, hq, hk, dim, rotary, length, interleaved=False, params32=False, gamma=True, packed=True,
           given=True, ids64=True, padded=0.0):
    """length: rows of the angles' tables (the longest sequence); packed: queries and keys are slices
    of one projection's output; given: positions are given (else a row's position is its index);
    padded: the share of rows without a position."""
    c = {"op": "heads", "way": way, "type": type, "rows": rows, "hq": hq, "hk": hk, "dim": dim, "rotary": rotary,
         "length": length, "interleaved": interleaved, "params32": params32, "gamma": gamma, "packed": packed, "given": given,
         "ids64": ids64, "padded": padded}
    return {"name": name, **c} if name else c


def _kept(name, way, type, rows, cols, p=0.0, res32=False, params32=False, bias=False, dsum=False, pad=0):
    """way: "pack", "restore", "norm" or "addnorm" (the backward passes from codes)."""
    c = {"op": "checkpoint", "way": way, "type": type, "rows": rows, "cols": cols, "p": p, "res32": res32,
         "params32": params32, "bias": bias, "dsum": dsum, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a training batch's tokens with the dropout that follows, and the table's gradient
        _lookup("lookup fwd bf16 16384x4096", "fwd", "bf16", 16384, 4096, 131072, "uniform", 0.1, 64.0),
        _lookup("lookup bwd bf16 16384x4096", "bwd", "bf16", 16384, 4096, 32768, "zipf", 0.1, 64.0),
        # one token of a serving loop: the smallest call
        _lookup("lookup fwd bf16 1x4096", "fwd", "bf16", 1, 4096, 32768),
        # a ragged, padded batch of an odd width into a float table's gradient
        _lookup("lookup bwd f16 res32 2047x1001", "bwd", "f16", 2047, 1001, 50001, "zipf", 0.1, 1.0, res32=True, params32=True,
                ids64=False, padded=0.2, pad=7),
        # grouped queries and keys of a training batch, slices of one projection, both directions
        _heads("heads fwd bf16 16384x(32+8)x128", "fwd", "bf16", 16384, 32, 8, 128, 128, 8192),
        _heads("heads bwd bf16 8192x(32+8)x128", "bwd", "bf16", 8192, 32, 8, 128, 128, 8192),
        # a decoding step of eight sequences at positions far apart
        _heads("heads fwd bf16 8x(32+8)x128", "fwd", "bf16", 8, 32, 8, 128, 128, 32768),
        # a small float model with half of each head turned, neighbours paired, a padded batch
        _heads("heads bwd f32 333x(6+2)x80", "bwd", "f32", 333, 6, 2, 80, 40, 1024, interleaved=True, packed=False,
               ids64=False, padded=0.1),
        # the residual stream of a training batch put away, and a short batch of an odd width brought back
        _kept("pack bf16 16384x8192", "pack", "bf16", 16384, 8192),
        _kept("restore f16 333x2049", "restore", "f16", 333, 2049, pad=7),
        # a pre-norm block's junction in the backward pass, and a small model's norm
        _kept("addnorm bwd bf16 8192x8192", "addnorm", "bf16", 8192, 8192, 0.1, bias=True, dsum=True),
        _kept("norm bwd f32 4096x1024", "norm", "f32", 4096, 1024),
    ]


def draw(rng):
    while True:
        op = rng.choice(("embedding", "heads", "checkpoint"))
        kind = rng.choice(("bf16", "bf16", "f16", "f32"))
        half = kind != "f32"
        rows = int(2 ** rng.uniform(0, 15))
        cols = int(2 ** rng.uniform(4, 13.5))
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        pad = rng.choice((0, 0, 0, 8, 5))
        if op == "embedding":
            c = _lookup(None, rng.choice(("fwd", "bwd")), kind, rows, cols, int(2 ** rng.uniform(4, 17)),
                        rng.choice(("zipf", "zipf", "uniform", "one")), rng.choice((0.0, 0.0, 0.1, 0.25)),
                        rng.choice((1.0, round(math.sqrt(cols), 3))), half and rng.random() < 0.4, half and rng.random() < 0.4,
                        rng.random() < 0.5, rng.choice((0.0, 0.0, 0.3)), pad)
        elif op == "heads":
            dim = rng.choice((32, 64, 64, 128, 128, 128, 256, 80, 96, 72, 65))
            rotary = rng.choice((dim // 2 * 2, dim // 2 * 2, dim // 4 * 2, max(2, dim // 8 * 2)))
            hk = int(2 ** rng.uniform(0, 5.1))
            given = rng.random() < 0.7
            c = _heads(None, rng.choice(("fwd", "bwd")), kind, rows, hk * rng.choice((1, 1, 3, 4, 8)), hk, dim, rotary,
                       int(2 ** rng.uniform(9, 15)) if given else rows, rng.random() < 0.4, half and rng.random() < 0.4,
                       rng.random() < 0.8, rng.random() < 0.6, given, rng.random() < 0.5,
                       rng.choice((0.0, 0.0, 0.2)) if given else 0.0)
        else:
            way = rng.choice(("pack", "restore", "norm", "addnorm"))
            both = way == "addnorm"
            c = _kept(None, way, kind, rows, cols, rng.choice((0.0, 0.1, 0.25)) if both else 0.0, half and rng.random() < 0.4,
                      half and "norm" in way and rng.random() < 0.4, both and rng.random() < 0.6, both and rng.random() < 0.6,
                      pad)
        if work(c)["bytes"] <= MOST and _elements(c) <= 1 << 27:
            return c


def _elements(case):
    if case["op"] == "heads":
        return case["rows"] * (case["hq"] + case["hk"]) * case["dim"]
    if case["op"] == "embedding" and case["way"] == "bwd":
        return (case["rows"] + case["vocab"]) * case["cols"]
    return case["rows"] * case["cols"]


def _distinct(n, values, spread):
    """How many of `values` equally likely (or, "zipf", log-uniform) numbers n draws are expected to hit."""
    if spread == "one":
        return min(n, 1)
    if spread == "uniform":
        return values * -math.expm1(n * math.log1p(-1 / values)) if values > 1 else min(n, 1)
    v = torch.arange(values, dtype=torch.float64)
    share = torch.log1p(1 / (v + 1)) / math.log(values + 1)
    return float(-torch.expm1(-n * share).sum())


def work(case):
    op, way = case["op"], case["way"]
    t = 4 if case["type"] == "f32" else 2
    w = 4 if case["params32"] else t
    rows = case["rows"]
    draw_ops = 12 if case.get("p") or way == "pack" else 0  # the hash of one element's counter, its compare and its quotient
    if op == "heads":
        n, turned = _elements(case), rows
        angles = min(turned, case["length"]) if not case["given"] else _distinct(turned, case["length"], "uniform")
        b = n * t * (2 if way == "fwd" else 3) + angles * case["rotary"] * 4
        b += (8 if case["ids64"] else 4) * rows if case["given"] else 0
        b += 2 * case["dim"] * w * (way == "bwd") + 2 * case["dim"] * w * case["gamma"]
        return {"bytes": b, "flops": n * (7 if way == "fwd" else 15)}
    cols, n = case["cols"], rows * case["cols"]
    r = 4 if case["res32"] else t
    if op == "embedding":
        there = n * (1 - case["padded"])
        b = rows * (8 if case["ids64"] else 4)
        if way == "fwd":  # the distinct rows of the table -> y
            b += _distinct(rows * (1 - case["padded"]), case["vocab"], case["ids"]) * cols * w + n * r
        else:  # dy -> the whole gradient
            b += there * r + case["vocab"] * cols * w
        return {"bytes": b, "flops": there * (2 + draw_ops)}
    codes = n + 4 * rows * -(-cols // BLOCK)
    if way in ("pack", "restore"):
        return {"bytes": codes + n * r, "flops": n * (8 + draw_ops if way == "pack" else 1)}
    if way == "norm":
        return {"bytes": codes + n * (t + r) + 3 * cols * w + 8 * rows, "flops": n * 15}
    return {"bytes": codes + n * (2 * t + r * (1 + case["dsum"])) + (3 + case["bias"]) * cols * w + 8 * rows,
            "flops": n * (17 + draw_ops)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    T = TYPES[case["type"]]
    W = torch.float32 if case["params32"] else T
    key = (seed * 2654435761 + 97) % (1 << 32)
    s = {"case": case, "key": key, "start": (key * 40503) % (1 << 24), "T": T, "W": W}
    return (_prepare_lookup if case["op"] == "embedding" else _prepare_heads if case["op"] == "heads" else _prepare_kept)(s, g)


def _normal(g, rows, cols, pad, kind, scale):
    return torch.empty(rows, cols + pad, dtype=kind, device=DEV).normal_(0.0, scale, generator=g)[:, :cols]


def _vector(g, cols, kind, around, scale):
    return (around + scale * torch.randn(cols, generator=g, device=DEV)).to(kind)


def _prepare_lookup(s, g):
    c = s["case"]
    R = torch.float32 if c["res32"] else s["T"]
    s["R"] = R
    u = torch.rand(c["rows"], generator=g, device=DEV, dtype=torch.float64)
    if c["ids"] == "zipf":
        ids = ((c["vocab"] + 1.0) ** u).long() - 1  # token v with a chance of about 1 / (v + 1)
    elif c["ids"] == "uniform":
        ids = (u * c["vocab"]).long()
    else:
        ids = torch.full((c["rows"],), (s["key"] >> 3) % c["vocab"], device=DEV)
    ids.clamp_(max=c["vocab"] - 1)
    if c["padded"]:
        ids = torch.where(torch.rand(c["rows"], generator=g, device=DEV) < c["padded"], -1, ids)
    s["ids"] = ids.to(torch.int64 if c["ids64"] else torch.int32)
    if c["way"] == "fwd":
        s["table"] = _normal(g, c["vocab"], c["cols"], 0, s["W"], 0.02)
        s["y"] = torch.empty(c["rows"], c["cols"] + c["pad"], dtype=R, device=DEV)[:, :c["cols"]]
    else:
        s["dy"] = _normal(g, c["rows"], c["cols"], c["pad"], R, 0.01)
        s["dtable"] = torch.empty(c["vocab"], c["cols"], dtype=s["W"], device=DEV)
        s["workspace"] = None
    return s


def _prepare_heads(s, g):
    c = s["case"]
    T, W, rows, dim, half = s["T"], s["W"], c["rows"], c["dim"], c["rotary"] // 2
    nq, nk = c["hq"] * dim, c["hk"] * dim

    def pair(scale):
        """Queries and keys, in a projection's output with the values behind them or alone."""
        if c["packed"]:
            m = _normal(g, rows, nq + 2 * nk, 0, T, scale)
            return m[:, :nq], m[:, nq:nq + nk]
        return _normal(g, rows, nq, 0, T, scale), _normal(g, rows, nk, 0, T, scale)

    s["q"], s["k"] = pair(1.5)
    s["gamma_q"], s["gamma_k"] = (_vector(g, dim, W, 1.0, 0.1) if c["gamma"] else None for _ in range(2))
    angle = torch.arange(c["length"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
        torch.arange(half, device=DEV, dtype=torch.float64) / -max(half, 1))
    s["cosines"], s["sines"] = angle.cos().float(), angle.sin().float()
    s["positions"] = None
    if c["given"]:
        at = torch.randint(0, c["length"], (rows,), generator=g, device=DEV)
        if c["padded"]:
            at = torch.where(torch.rand(rows, generator=g, device=DEV) < c["padded"], -1, at)
        s["positions"] = at.to(torch.int64 if c["ids64"] else torch.int32)
    if c["way"] == "fwd":
        s["yq"], s["yk"] = (torch.empty(rows, n, dtype=T, device=DEV) for n in (nq, nk))
    else:
        s["dyq"], s["dyk"] = pair(0.01)
        d = torch.empty(rows, nq + nk, dtype=T, device=DEV)
        s["dq"], s["dk"] = d[:, :nq], d[:, nq:]
        s["dgamma_q"], s["dgamma_k"] = (torch.empty(dim, dtype=W, device=DEV) for _ in range(2))
    return s


def _prepare_kept(s, g):
    c = s["case"]
    T, W, rows, cols, pad = s["T"], s["W"], c["rows"], c["cols"], c["pad"]
    R = torch.float32 if c["res32"] else T
    s["R"] = R
    # a residual stream: some columns much larger than the rest
    x = _normal(g, rows, cols, pad, torch.float32, 2.0)
    x.mul_(torch.exp(0.8 * torch.randn(cols, generator=g, device=DEV)))
    s["x"] = x if R is torch.float32 else torch.empty(rows, cols + pad, dtype=R, device=DEV)[:, :cols].copy_(x)
    if c["way"] == "pack":
        s["codes"] = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(rows, -(-cols // BLOCK), device=DEV)
        return s
    s["codes"], s["scales"] = _pack(s)
    if c["way"] == "restore":
        del s["x"]
        s["y"] = torch.empty(rows, cols + pad, dtype=R, device=DEV)[:, :cols]
        return s
    v = s.pop("x").float()  # the statistics that the forward pass left
    s["mean"] = v.mean(1)
    s["rstd"] = torch.rsqrt((v - s["mean"][:, None]).square().mean(1) + EPS)
    s["gamma"] = _vector(g, cols, W, 1.0, 0.1)
    s["dy"] = _normal(g, rows, cols, pad, T, 0.01)
    s["dsum"] = _normal(g, rows, cols, pad, R, 0.01) if c["dsum"] else None
    s["dgamma"], s["dbeta"] = (torch.empty(cols, dtype=W, device=DEV) for _ in range(2))
    s["dbias"] = torch.empty(cols, dtype=W, device=DEV) if c["bias"] else None
    s["dresidual"] = torch.empty(rows, cols, dtype=R, device=DEV)
    s["dx"] = torch.empty(rows, cols, dtype=T, device=DEV) if c["way"] == "addnorm" else s["dresidual"]
    return s


# ---- the plain form ----

def _uniform(s, rows, cols):
    """The uniforms of the elements' counters: the low 23 bits of each word, lowbias32."""
    def shift(x, k):  # a logical shift of 32-bit patterns
        return (x >> k) & ((1 << (32 - k)) - 1)

    def mix(x):
        x = (x ^ shift(x, 16)) * 0x7FEB352D
        x = (x ^ shift(x, 15)) * (0x846CA68B - (1 << 32))
        return x ^ shift(x, 16)

    key = torch.full((), s["key"], dtype=torch.int64, device=DEV).to(torch.int32)
    c = torch.arange(s["start"], s["start"] + rows * cols, device=DEV).to(torch.int32)
    return ((mix(c ^ mix(key)) & 0x7FFFFF).to(torch.float32) * 2.0 ** -23).view(rows, cols)


def _drop(s, v):
    if s["case"]["p"] == 0:
        return v
    p = torch.full((), s["case"]["p"], dtype=torch.float32, device=DEV)
    return torch.where(_uniform(s, *v.shape) >= p, v / (1 - p), 0.0)


def _plain_lookup(s):
    c = s["case"]
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < c["vocab"])
    if c["way"] == "fwd":
        z = s["table"][torch.where(there, ids, 0)].float() * c["scale"]
        return {"y": _drop(s, torch.where(there[:, None], z, 0.0)).to(s["R"])}
    v = _drop(s, s["dy"].float())
    total = torch.zeros(c["vocab"] + 1, c["cols"], device=DEV)  # the last row: rows without a token
    total.index_add_(0, torch.where(there, ids, c["vocab"]), v)
    return {"dtable": (total[:-1] * c["scale"]).to(s["W"])}


def _angles(s):
    """Every row's cosines and sines; 1 and 0 where its position is none of the tables'."""
    c = s["case"]
    at = s["positions"].long() if c["given"] else torch.arange(c["rows"], device=DEV)
    there = ((at >= 0) & (at < c["length"]))[:, None]
    at = at.clamp(0, c["length"] - 1)
    return torch.where(there, s["cosines"][at], 1.0)[:, None], torch.where(there, s["sines"][at], 0.0)[:, None]


def _turn(c, x, cosines, sines):
    """x [rows, heads, dim] with its pairs turned."""
    rot = c["rotary"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        pairs = torch.stack((a * cosines - b * sines, b * cosines + a * sines), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        pairs = torch.cat((a * cosines - b * sines, b * cosines + a * sines), -1)
    return torch.cat((pairs, x[..., rot:]), -1)


def _normed_heads(c, x, gamma, cosines, sines):
    v = x.float().view(c["rows"], -1, c["dim"])
    n = v * torch.rsqrt(v.square().mean(-1, True) + EPS)
    if gamma is not None:
        n = n * gamma.float()
    return _turn(c, n, cosines, sines).view(c["rows"], -1).to(x.dtype)


def _heads_back(s, x, dy, gamma, cosines, sines):
    c = s["case"]
    v = x.float().view(c["rows"], -1, c["dim"])
    rstd = torch.rsqrt(v.square().mean(-1, True) + EPS)
    h = v * rstd
    g = _turn(c, dy.float().view(v.shape), cosines, -sines)
    dgamma = (g * h).sum((0, 1)).to(s["W"])
    if gamma is not None:
        g = g * gamma.float()
    dx = rstd * (g - h * (g * h).mean(-1, True))
    return dx.view(c["rows"], -1).to(x.dtype), dgamma


def _plain_heads(s):
    c = s["case"]
    cosines, sines = _angles(s)
    if c["way"] == "fwd":
        return {"yq": _normed_heads(c, s["q"], s["gamma_q"], cosines, sines),
                "yk": _normed_heads(c, s["k"], s["gamma_k"], cosines, sines)}
    dq, dgamma_q = _heads_back(s, s["q"], s["dyq"], s["gamma_q"], cosines, sines)
    dk, dgamma_k = _heads_back(s, s["k"], s["dyk"], s["gamma_k"], cosines, sines)
    return {"dq": dq, "dk": dk, "dgamma_q": dgamma_q, "dgamma_k": dgamma_k}


def _blocks(x):
    """x [rows, cols] as [rows, blocks, 128], zeros behind the last column."""
    rows, cols = x.shape
    n = -(-cols // BLOCK)
    return torch.nn.functional.pad(x, (0, n * BLOCK - cols)).view(rows, n, BLOCK)


def _pack(s):
    c = s["case"]
    x = _blocks(s["x"].float())
    most = x.abs().amax(-1, True)
    held = most >= 2.0 ** -100
    # quotients in 64 bits and rounded once, which is the float quotient
    scale = torch.where(held, (most.double() / 127).float(), 0.0)
    inverse = torch.where(held, (127 / most.double()).float(), 0.0)
    t = x.abs() * inverse
    down = t.floor()
    up = _blocks(_uniform(s, c["rows"], c["cols"])) < t - down
    code = (down + up).clamp(max=127) * x.sign()
    return code.to(torch.int8).view(c["rows"], -1)[:, :c["cols"]].contiguous(), scale[..., 0]


def _restored(s):
    c = s["case"]
    return (_blocks(s["codes"]).float() * s["scales"][..., None]).view(c["rows"], -1)[:, :c["cols"]]


def _plain_kept(s):
    c = s["case"]
    if c["way"] == "pack":
        codes, scales = _pack(s)
        return {"codes": codes, "scales": scales}
    v = _restored(s)
    if c["way"] == "restore":
        return {"y": v.to(s["R"])}
    dy = s["dy"].float()
    h = (v - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    d = s["rstd"][:, None] * (g - g.mean(1, True) - h * (g * h).mean(1, True))
    out = {"dgamma": (dy * h).sum(0).to(s["W"]), "dbeta": dy.sum(0).to(s["W"])}
    if c["way"] == "norm":
        return {"dx": d.to(s["R"]), **out}
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    dx = _drop(s, d)
    if s["dbias"] is not None:
        out["dbias"] = dx.sum(0).to(s["W"])
    return {"dresidual": d.to(s["R"]), "dx": dx.to(s["T"]), **out}


def run(s):
    c = s["case"]
    if own:
        return (_own_lookup if c["op"] == "embedding" else _own_heads if c["op"] == "heads" else _own_kept)(s)
    return (_plain_lookup if c["op"] == "embedding" else _plain_heads if c["op"] == "heads" else _plain_kept)(s)


# ---- the library's calls ----

def _own_lookup(s):
    import bulk_fills_amd as tk
    c = s["case"]
    t, rows, cols = c["type"], c["rows"], c["cols"]
    flags = (tk.TK_RESIDUAL_F32 if c["res32"] else 0) | (tk.TK_PARAMS_F32 if c["params32"] else 0)
    flags |= tk.TK_INDEX_I64 if c["ids64"] else 0
    if c["way"] == "fwd":
        f = {"f32": tk.tk_embedding_f32, "f16": tk.tk_embedding_f16, "bf16": tk.tk_embedding_bf16}[t]
        f(s["key"], s["start"], rows, cols, c["p"], c["scale"], flags, c["vocab"], s["ids"], s["table"], None, s["y"], None)
        return {"y": s["y"]}
    f = {"f32": tk.tk_embedding_backward_f32, "f16": tk.tk_embedding_backward_f16, "bf16": tk.tk_embedding_backward_bf16}[t]
    if s["workspace"] is None:  # kept between steps, as a training loop does
        s["workspace"] = torch.empty(tk.tk_embedding_workspace_bytes(rows, cols, c["vocab"]), dtype=torch.uint8, device=DEV)
    f(s["key"], s["start"], rows, cols, c["p"], c["scale"], flags, c["vocab"], s["ids"], s["dy"], None, s["dtable"], None,
      s["workspace"])
    return {"dtable": s["dtable"]}


def _own_heads(s):
    import bulk_fills_amd as tk
    c = s["case"]
    t, rows = c["type"], c["rows"]
    flags = (tk.TK_PARAMS_F32 if c["params32"] else 0) | (tk.TK_INDEX_I64 if c["ids64"] else 0)
    flags |= tk.TK_INTERLEAVED if c["interleaved"] else 0
    shape = (rows, c["hq"], c["hk"], c["dim"], c["rotary"], EPS, flags)
    if c["way"] == "fwd":
        f = {"f32": tk.tk_head_norm_rotate_f32, "f16": tk.tk_head_norm_rotate_f16, "bf16": tk.tk_head_norm_rotate_bf16}[t]
        f(*shape, s["q"], None, s["k"], None, s["gamma_q"], s["gamma_k"], s["positions"], c["length"], s["cosines"],
          s["sines"], s["yq"], None, s["yk"], None)
        return {k: s[k] for k in ("yq", "yk")}
    f = {"f32": tk.tk_head_norm_rotate_backward_f32, "f16": tk.tk_head_norm_rotate_backward_f16,
         "bf16": tk.tk_head_norm_rotate_backward_bf16}[t]
    f(*shape, s["dyq"], None, s["dyk"], None, s["q"], None, s["k"], None, s["gamma_q"], s["gamma_k"], s["positions"],
      c["length"], s["cosines"], s["sines"], s["dq"], None, s["dk"], None, s["dgamma_q"], s["dgamma_k"])
    return {k: s[k] for k in ("dq", "dk", "dgamma_q", "dgamma_k")}


def _own_kept(s):
    import bulk_fills_amd as tk
    c = s["case"]
    way, t, rows, cols = c["way"], c["type"], c["rows"], c["cols"]
    flags = (tk.TK_RESIDUAL_F32 if c["res32"] else 0) | (tk.TK_PARAMS_F32 if c["params32"] else 0)
    if way == "pack":
        f = {"f32": tk.tk_checkpoint_f32, "f16": tk.tk_checkpoint_f16, "bf16": tk.tk_checkpoint_bf16}[t]
        f(s["key"], s["start"], rows, cols, flags, s["x"], None, s["codes"], None, s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if way == "restore":
        f = {"f32": tk.tk_checkpoint_restore_f32, "f16": tk.tk_checkpoint_restore_f16,
             "bf16": tk.tk_checkpoint_restore_bf16}[t]
        f(rows, cols, flags, s["codes"], None, s["scales"], s["y"], None)
        return {"y": s["y"]}
    if way == "norm":
        f = {"f32": tk.tk_layer_norm_backward_checkpoint_f32, "f16": tk.tk_layer_norm_backward_checkpoint_f16,
             "bf16": tk.tk_layer_norm_backward_checkpoint_bf16}[t]
        f(rows, cols, flags, s["dy"], None, s["codes"], None, s["scales"], s["gamma"], s["mean"], s["rstd"], s["dx"], None,
          s["dgamma"], s["dbeta"])
        return {k: s[k] for k in ("dx", "dgamma", "dbeta")}
    f = {"f32": tk.tk_dropout_add_layer_norm_backward_checkpoint_f32,
         "f16": tk.tk_dropout_add_layer_norm_backward_checkpoint_f16,
         "bf16": tk.tk_dropout_add_layer_norm_backward_checkpoint_bf16}[t]
    f(s["key"], s["start"], rows, cols, c["p"], flags, s["dy"], None, s["dsum"], None, s["codes"], None, s["scales"],
      s["gamma"], s["mean"], s["rstd"], s["dx"], None, s["dresidual"], None, s["dgamma"], s["dbeta"], s["dbias"])
    return {k: s[k] for k in ("dresidual", "dx", "dgamma", "dbeta", "dbias") if s[k] is not None}


# ---- the definition in 64 bits ----

def _low32(a, b):
    """The low 32 bits of a product of 32-bit numbers held in 64: its 16-bit halves one by one."""
    return (a * (b & 0xFFFF) + ((a * (b >> 16) & 0xFFFF) << 16)) & 0xFFFFFFFF


def _uniform64(s, rows, cols):
    def lowbias(v):
        v = _low32(v ^ (v >> 16), 0x7FEB352D)
        v = _low32(v ^ (v >> 15), 0x846CA68B)
        return v ^ (v >> 16)
    w = lowbias((torch.arange(rows * cols, device=DEV) + s["start"]) ^ lowbias(torch.tensor(s["key"], device=DEV)))
    return ((w % (1 << 23)).double() / (1 << 23)).view(rows, cols)


def _scale64(s, rows, cols):
    """What dropout multiplies each element with: 0, or 1 / (1 - p)."""
    p = float(torch.tensor(s["case"]["p"], dtype=torch.float32))
    return 1.0 if p == 0 else (_uniform64(s, rows, cols) >= p).double() / (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    return (_exact_lookup if case["op"] == "embedding" else _exact_heads if case["op"] == "heads" else _exact_kept)(case, s, d)


def _exact_lookup(case, s, d):
    ids, rows, cols = s["ids"].long(), case["rows"], case["cols"]
    there = ids >= 0
    scale = float(torch.tensor(case["scale"], dtype=torch.float32))
    k = _scale64(s, rows, cols)
    if case["way"] == "fwd":
        y = torch.zeros(rows, cols, dtype=torch.float64, device=DEV)
        y[there] = d["table"][ids[there]] * scale
        return {"y": y * k}
    v = (d["dy"] * k)[there] * scale
    order = torch.argsort(ids[there])
    which, ends = torch.unique_consecutive(ids[there][order], return_counts=True)
    sums = torch.zeros(case["vocab"], cols, dtype=torch.float64, device=DEV)
    if len(which):
        sums[which] = torch.segment_reduce(v[order], "sum", lengths=ends, axis=0)
    return {"dtable": sums}


def _exact_heads(case, s, d):
    rows, dim, rot, half = case["rows"], case["dim"], case["rotary"], case["rotary"] // 2
    at = torch.arange(rows, device=DEV) if s["positions"] is None else s["positions"].long()
    z = torch.complex(d["cosines"], d["sines"])
    z = torch.cat((z, torch.ones(1, half, dtype=z.dtype, device=DEV)))  # the last row: no position
    z = z[torch.where((at < 0) | (at >= case["length"]), case["length"], at)].view(rows, 1, half)

    def turn(x, by):
        x = x.view(rows, -1, dim)
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        w = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = w.real, w.imag
        return y

    def one(n):
        x = d[n].reshape(rows, -1, dim)
        gamma = d.get("gamma_" + n, torch.ones(dim, dtype=torch.float64, device=DEV))
        rstd = ((x * x).sum(-1, keepdim=True) / dim + EPS) ** -0.5
        if case["way"] == "fwd":
            return {"y" + n: turn(x * rstd * gamma, z).reshape(rows, -1)}
        g = turn(d["dy" + n].reshape(rows, -1), z.conj())
        dgamma, g = (g * x * rstd).sum((0, 1)), g * gamma
        dx = rstd * g - rstd ** 3 * x * ((g * x).sum(-1, keepdim=True) / dim)
        return {"d" + n: dx.reshape(rows, -1), "dgamma_" + n: dgamma}

    return {**one("q"), **one("k")}


def _exact_kept(case, s, d):
    rows, cols, way = case["rows"], case["cols"], case["way"]
    block = torch.arange(cols, device=DEV) // BLOCK
    if way == "pack":
        x = d["x"].abs()
        most = torch.zeros(rows, s["scales"].shape[1], dtype=torch.float64, device=DEV).index_reduce_(1, block, x, "amax")
        zero = most < 2.0 ** -100

        def as_float(v):  # the definition's own roundings
            return torch.where(zero, 0.0, v).float().double()
        t = (x * as_float(127 / most)[:, block]).float().double()
        n = torch.minimum(t.floor() + (_uniform64(s, rows, cols) < t % 1).double(), torch.tensor(127.0, device=DEV))
        return {"codes": (n * d["x"].sign()).to(torch.int8), "scales": most / 127 * ~zero}
    v = s["codes"].double() * d["scales"][:, block]
    if way == "restore":
        return {"y": v}
    rstd, dy = d["rstd"].view(rows, 1), d["dy"]
    h = (v - d["mean"].view(rows, 1)) * rstd
    out = {"dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}
    g = dy * d["gamma"]
    v = rstd * (g - (g.sum(1, True) + h * (g * h).sum(1, True)) / cols)
    if way == "norm":
        return {"dx": v, **out}
    v = v + d.get("dsum", 0.0)
    out["dresidual"], out["dx"] = v, v * _scale64(s, rows, cols)
    if "dbias" in d:
        out["dbias"] = out["dx"].sum(0)
    return out
