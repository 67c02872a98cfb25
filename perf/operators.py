"""Cases of the row operators: dropout-add, layer norm, and the two fused, each direction.

Every operator works on a rows x cols matrix whose rows may lie `pad` elements apart.
With z = x + bias, u(r, c) = uniform of word start + r cols + c of the key's stream and
q = 1 - p:

    drop(v) = u >= p ? v / q : 0
    dropout_add             y = residual + drop(z)
      backward              dx = drop(dy);  dbias = column sums of dx
    layer_norm              y = (x - mean) rstd gamma + beta, with the row's mean and
                            rstd = (variance + eps)^(-1/2)
      backward              g = dy gamma, h = (x - mean) rstd:
                            dx = rstd (g - mean(g) - h mean(g h)),
                            dgamma = column sums of dy h, dbeta = column sums of dy
    dropout_add_layer_norm  sum = residual + drop(z), y = layer norm of sum
      backward              dresidual = dsum + layer norm's dx, dx = drop(dresidual),
                            dbias = column sums of dx, and dgamma, dbeta

`run` computes these in elementary torch operations, or with the library's calls where
`own` is set; `exact` computes them in 64 bits.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5

# Just under the bytes of the largest listed case.
MOST = 1.07e9


def _case(name, op, way, type, rows, cols, p=0.0, res32=False, params32=False, bias=False, residual=False, dsum=False,
          pad=0):
    """op: "add", "norm" or "addnorm"; way: "fwd" or "bwd"; res32: the residual stream (residual,
    sum, and their gradients; layer norm's x and dx) is float; params32: bias, gamma, beta and
    their gradients are float; dsum: the sum has a gradient of its own; pad: elements between
    the rows of the inputs."""
    c = {"op": op, "way": way, "type": type, "rows": rows, "cols": cols, "p": p, "res32": res32, "params32": params32,
         "bias": bias, "residual": residual, "dsum": dsum, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the projection's epilogue of a training step: bias, dropout, residual; and its gradient
        _case("add fwd bf16 8192x4096", "add", "fwd", "bf16", 8192, 4096, 0.1, bias=True, residual=True),
        _case("add bwd bf16 8192x4096", "add", "bwd", "bf16", 8192, 4096, 0.1, bias=True),
        # a short ragged batch of an odd width, rows cut from a wider buffer
        _case("add fwd f16 333x2049 pad", "add", "fwd", "f16", 333, 2049, 0.2, bias=True, residual=True, pad=7),
        # one token's norm in a serving loop: the smallest call
        _case("norm fwd bf16 1x4096", "norm", "fwd", "bf16", 1, 4096),
        # the norm that opens a block, reading a float residual stream
        _case("norm fwd bf16 res32 16384x8192", "norm", "fwd", "bf16", 16384, 8192, res32=True, params32=True),
        # a small model's norm in float, and a per-head norm: many short rows
        _case("norm bwd f32 4096x1024", "norm", "bwd", "f32", 4096, 1024),
        _case("norm bwd bf16 65536x128", "norm", "bwd", "bf16", 65536, 128),
        # a pre-norm block's junction in a training step, forward and backward
        _case("addnorm fwd bf16 16384x8192", "addnorm", "fwd", "bf16", 16384, 8192, 0.1, bias=True, residual=True),
        _case("addnorm bwd bf16 8192x8192", "addnorm", "bwd", "bf16", 8192, 8192, 0.1, bias=True, residual=True,
              dsum=True),
        # an odd width with a float residual stream and float parameters
        _case("addnorm bwd f16 res32 2047x5001", "addnorm", "bwd", "f16", 2047, 5001, 0.1, res32=True, params32=True,
              bias=True, residual=True, dsum=True),
        # a post-norm junction without a bias, a short batch
        _case("addnorm fwd f32 64x768", "addnorm", "fwd", "f32", 64, 768, 0.1, residual=True),
        # very wide rows
        _case("addnorm bwd bf16 512x24576", "addnorm", "bwd", "bf16", 512, 24576, 0.1, params32=True, bias=True,
              residual=True),
    ]


def draw(rng):
    while True:
        op, way = rng.choice(("add", "norm", "addnorm")), rng.choice(("fwd", "bwd"))
        kind = rng.choice(("bf16", "bf16", "f16", "f32"))
        rows = int(2 ** rng.uniform(0, 16))
        cols = int(2 ** rng.uniform(4, 15))
        if rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        drop = op != "norm"
        c = _case(None, op, way, kind, rows, cols, rng.choice((0.0, 0.1, 0.25, 0.5)) if drop else 0.0,
                  kind != "f32" and rng.random() < 0.4, kind != "f32" and rng.random() < 0.4, drop and rng.random() < 0.6,
                  drop and (op == "addnorm" or rng.random() < 0.7), op == "addnorm" and way == "bwd" and rng.random() < 0.6,
                  rng.choice((0, 0, 0, 8, 5)))
        if work(c)["bytes"] <= MOST and rows * cols <= 1 << 27:
            return c


def _sizes(case):
    t = 4 if case["type"] == "f32" else 2
    return t, 4 if case["res32"] else t, 4 if case["params32"] else t


def work(case):
    t, r, w = _sizes(case)
    n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
    op, fwd, bias = case["op"], case["way"] == "fwd", case["bias"]
    draw_ops = 12 if case["p"] else 0  # the hash of one element's counter, its compare and its quotient
    if op == "add":
        # forward: x, residual -> y;  backward: dy -> dx, dbias
        b = n * (t + r + (r if case["residual"] else 0)) + bias * cols * w if fwd else n * (r + t) + bias * cols * w
        f = n * (2 + draw_ops) if fwd else n * (1 + draw_ops)
    elif op == "norm":
        # forward: x -> y, mean, rstd;  backward: dy, x, mean, rstd -> dx, dgamma, dbeta
        b = n * (r + t) + 2 * cols * w + 8 * rows if fwd else n * (t + 2 * r) + 3 * cols * w + 8 * rows
        f = n * 8 if fwd else n * 14
    elif fwd:  # x, residual -> sum, y, mean, rstd
        b = n * (t + r * (2 if case["residual"] else 1) + t) + (2 + bias) * cols * w + 8 * rows
        f = n * (10 + draw_ops)
    else:  # dy, dsum, sum, mean, rstd -> dresidual, dx, dgamma, dbeta, dbias
        b = n * (2 * t + r * (2 + case["dsum"])) + (3 + bias) * cols * w + 8 * rows
        f = n * (16 + draw_ops)
    return {"bytes": b, "flops": f}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows, cols, op, fwd = case["rows"], case["cols"], case["op"], case["way"] == "fwd"
    T = TYPES[case["type"]]
    R = torch.float32 if case["res32"] else T
    W = torch.float32 if case["params32"] else T

    def matrix(kind, scale):
        m = torch.empty(rows, cols + case["pad"], dtype=kind, device=DEV)
        m.normal_(0.0, scale, generator=g)
        return m[:, :cols]

    def vector(around, scale):
        return (around + scale * torch.randn(cols, generator=g, device=DEV)).to(W)

    def out(kind):
        return torch.empty(rows, cols, dtype=kind, device=DEV)

    def stat():
        return torch.empty(rows, dtype=torch.float32, device=DEV)

    key = (seed * 2654435761 + 97) % (1 << 32)
    s = {"case": case, "key": key, "start": (key * 40503) % (1 << 24), "T": T, "R": R, "W": W}
    if fwd:
        if op != "norm":
            s["x"] = matrix(T, 1.0)
            s["bias"] = vector(0.0, 0.1) if case["bias"] else None
            s["residual"] = matrix(R, 2.0) if case["residual"] else None
        else:
            s["x"] = matrix(R, 2.0)
        if op != "add":
            s.update(gamma=vector(1.0, 0.1), beta=vector(0.0, 0.1), mean=stat(), rstd=stat())
        s["y"] = out(R if op == "add" else T)
        if op == "addnorm":
            s["sum"] = out(R)
    else:
        s["dy"] = matrix(R if op == "add" else T, 0.01)
        s["dx"] = out(R if op == "norm" else T)
        if op != "norm":
            s["dbias"] = torch.empty(cols, dtype=W, device=DEV) if case["bias"] else None
        if op != "add":
            v = matrix(R, 2.0)  # the norm's input, and the statistics that the forward pass left
            s.update(sum=v, mean=v.float().mean(1), gamma=vector(1.0, 0.1))
            s["rstd"] = torch.rsqrt((v.float() - s["mean"][:, None]).square().mean(1) + EPS)
            s.update(dgamma=torch.empty(cols, dtype=W, device=DEV), dbeta=torch.empty(cols, dtype=W, device=DEV))
        if op == "addnorm":
            s["dsum"] = matrix(R, 0.01) if case["dsum"] else None
            s["dresidual"] = out(R)
    return s


# ---- the plain form ----

def _keep(s, rows, cols):
    """Whether dropout keeps each element: the word of its counter, lowbias32, against p."""
    def shift(x, k):  # a logical shift of 32-bit patterns
        return (x >> k) & ((1 << (32 - k)) - 1)

    def mix(x):
        x = (x ^ shift(x, 16)) * 0x7FEB352D
        x = (x ^ shift(x, 15)) * (0x846CA68B - (1 << 32))
        return x ^ shift(x, 16)

    key = torch.full((), s["key"], dtype=torch.int64, device=DEV).to(torch.int32)
    c = torch.arange(s["start"], s["start"] + rows * cols, device=DEV).to(torch.int32)
    u = (mix(c ^ mix(key)) & 0x7FFFFF).to(torch.float32) * 2.0 ** -23
    return (u >= _p(s)).view(rows, cols)


def _p(s):
    return torch.full((), s["case"]["p"], dtype=torch.float32, device=DEV)


def _drop(s, v):
    if s["case"]["p"] == 0:
        return v
    return torch.where(_keep(s, *v.shape), v / (1 - _p(s)), 0.0)


def _dropped_sum(s):
    z = s["x"].float()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    v = _drop(s, z)
    return v if s["residual"] is None else s["residual"].float() + v


def _norm(s, v):
    mean = v.mean(1)
    d = v - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["T"]), "mean": mean, "rstd": rstd}


def _norm_back(s):
    dy = s["dy"].float()
    h = (s["sum"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dv = s["rstd"][:, None] * (g - g.mean(1, True) - h * (g * h).mean(1, True))
    return dv, {"dgamma": (dy * h).sum(0).to(s["W"]), "dbeta": dy.sum(0).to(s["W"])}


def _plain(s):
    op, fwd = s["case"]["op"], s["case"]["way"] == "fwd"
    if fwd:
        if op == "add":
            return {"y": _dropped_sum(s).to(s["R"])}
        if op == "norm":
            return _norm(s, s["x"].float())
        v = _dropped_sum(s)
        return {"sum": v.to(s["R"]), **_norm(s, v)}
    if op == "norm":
        dv, more = _norm_back(s)
        return {"dx": dv.to(s["R"]), **more}
    dv, more = (s["dy"].float(), {}) if op == "add" else _norm_back(s)
    if op == "addnorm":
        if s["dsum"] is not None:
            dv = dv + s["dsum"].float()
        more["dresidual"] = dv.to(s["R"])
    dx = _drop(s, dv)
    if s["dbias"] is not None:
        more["dbias"] = dx.sum(0).to(s["W"])
    return {"dx": dx.to(s["T"]), **more}


def run(s):
    if not own:
        return _plain(s)
    import bulk_fills_amd as tk
    c = s["case"]
    op, fwd, t, rows, cols, p = c["op"], c["way"] == "fwd", c["type"], c["rows"], c["cols"], c["p"]
    flags = (tk.TK_RESIDUAL_F32 if c["res32"] else 0) | (tk.TK_PARAMS_F32 if c["params32"] else 0)
    if op == "add" and fwd:
        f = {"f32": tk.tk_dropout_add_f32, "f16": tk.tk_dropout_add_f16, "bf16": tk.tk_dropout_add_bf16}[t]
        f(s["key"], s["start"], rows, cols, p, flags, s["x"], None, s["bias"], s["residual"], None, s["y"], None)
        return {"y": s["y"]}
    if op == "add":
        f = {"f32": tk.tk_dropout_add_backward_f32, "f16": tk.tk_dropout_add_backward_f16,
             "bf16": tk.tk_dropout_add_backward_bf16}[t]
        f(s["key"], s["start"], rows, cols, p, flags, s["dy"], None, s["dx"], None, s["dbias"])
        return {k: s[k] for k in ("dx", "dbias") if s[k] is not None}
    if op == "norm" and fwd:
        f = {"f32": tk.tk_layer_norm_f32, "f16": tk.tk_layer_norm_f16, "bf16": tk.tk_layer_norm_bf16}[t]
        f(rows, cols, EPS, flags, s["x"], None, s["gamma"], s["beta"], s["y"], None, s["mean"], s["rstd"])
        return {k: s[k] for k in ("y", "mean", "rstd")}
    if op == "norm":
        f = {"f32": tk.tk_layer_norm_backward_f32, "f16": tk.tk_layer_norm_backward_f16,
             "bf16": tk.tk_layer_norm_backward_bf16}[t]
        f(rows, cols, flags, s["dy"], None, s["sum"], None, s["gamma"], s["mean"], s["rstd"], s["dx"], None, s["dgamma"],
          s["dbeta"])
        return {k: s[k] for k in ("dx", "dgamma", "dbeta")}
    if fwd:
        f = {"f32": tk.tk_dropout_add_layer_norm_f32, "f16": tk.tk_dropout_add_layer_norm_f16,
             "bf16": tk.tk_dropout_add_layer_norm_bf16}[t]
        f(s["key"], s["start"], rows, cols, p, EPS, flags, s["x"], None, s["bias"], s["residual"], None, s["gamma"],
          s["beta"], s["sum"], None, s["y"], None, s["mean"], s["rstd"])
        return {k: s[k] for k in ("sum", "y", "mean", "rstd")}
    f = {"f32": tk.tk_dropout_add_layer_norm_backward_f32, "f16": tk.tk_dropout_add_layer_norm_backward_f16,
         "bf16": tk.tk_dropout_add_layer_norm_backward_bf16}[t]
    f(s["key"], s["start"], rows, cols, p, flags, s["dy"], None, s["dsum"], None, s["sum"], None, s["gamma"], s["mean"],
      s["rstd"], s["dx"], None, s["dresidual"], None, s["dgamma"], s["dbeta"], s["dbias"])
    return {k: s[k] for k in ("dx", "dresidual", "dgamma", "dbeta", "dbias") if s[k] is not None}


# ---- the definition in 64 bits ----

def _low32(a, b):
    """The low 32 bits of a product of 32-bit numbers held in 64: its 16-bit halves one by one."""
    return (a * (b & 0xFFFF) + ((a * (b >> 16) & 0xFFFF) << 16)) & 0xFFFFFFFF


def _word64(key, counter):
    def lowbias(v):
        v = _low32(v ^ (v >> 16), 0x7FEB352D)
        v = _low32(v ^ (v >> 15), 0x846CA68B)
        return v ^ (v >> 16)
    return lowbias(counter ^ lowbias(torch.tensor(key, device=DEV)))


def exact(case, seed):
    s = prepare(case, seed)
    rows, cols, n = case["rows"], case["cols"], case["rows"] * case["cols"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def scale():
        """What dropout multiplies each element with: 0, or 1 / (1 - p)."""
        p = float(torch.tensor(case["p"], dtype=torch.float32))
        if p == 0:
            return 1.0
        w = _word64(s["key"], torch.arange(n, device=DEV) + s["start"])
        return ((w % (1 << 23)).double() / (1 << 23) >= p).double().view(rows, cols) / (1 - p)

    out = {}
    if case["way"] == "fwd":
        v = d["x"]
        if case["op"] != "norm":
            if "bias" in d:
                v = v + d["bias"]
            v = v * scale() + d.get("residual", 0.0)
            out["y" if case["op"] == "add" else "sum"] = v
        if case["op"] != "add":
            mean = v.sum(1, True) / cols
            rstd = ((v - mean) ** 2).sum(1, True).div(cols).add(EPS).pow(-0.5)
            out.update(y=(v - mean) * rstd * d["gamma"] + d["beta"], mean=mean[:, 0], rstd=rstd[:, 0])
        return out
    v = d["dy"]
    if case["op"] != "add":
        rstd = d["rstd"].view(rows, 1)
        h = (d["sum"] - d["mean"].view(rows, 1)) * rstd
        out["dgamma"], out["dbeta"] = (v * h).sum(0), v.sum(0)
        g = v * d["gamma"]
        v = rstd * (g - (g.sum(1, True) + h * (g * h).sum(1, True)) / cols)
    if case["op"] == "norm":
        return {"dx": v, **out}
    if case["op"] == "addnorm":
        v = v + d.get("dsum", 0.0)
        out["dresidual"] = v
    out["dx"] = v * scale()
    if "dbias" in d:
        out["dbias"] = out["dx"].sum(0)
    return out
