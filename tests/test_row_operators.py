"""The row operators on the GPU against their 64-bit reference: dropout-add, layer norm and
both fused, forward and backward, at the sizes where a shape of kernel begins or ends, for
every pair of types; rows cut from wider buffers at odd addresses, whose neighbours must stay
as they were; in place; cut calls; captured calls; two streams; and a block's run of them."""
import contextlib

import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref
from gpu_harness import log

pytestmark = pytest.mark.gpu

# element type, residual stream float, parameters float
KINDS = [("f32", False, False), ("f16", False, False), ("f16", True, True), ("bf16", False, False), ("bf16", True, False),
         ("bf16", False, True)]
IDS = ["f32", "f16", "f16-r32-p32", "bf16", "bf16-r32", "bf16-p32"]
# rows, cols: both sides of every change of kernel shape, odd widths, single rows and columns
SIZES = [(1, 1), (3, 1), (5, 2), (1, 7), (33, 8), (9, 9), (2, 64), (17, 127), (50, 128), (7, 129), (6, 511), (70, 512),
         (3, 513), (5, 1000), (8, 1024), (5, 1025), (3, 2047), (2, 2048), (4, 2049), (33, 4096), (3, 4097), (5, 5001),
         (2, 8192), (3, 8193), (2, 16384), (3, 16385), (2, 24577), (1, 32768), (2, 32769), (1, 70001), (2500, 40),
         (1300, 136), (1201, 1032),
         # backward: 3, 60, 75, 256 lines of partial sums; 100 and 160 of more than the caches are to hold
         (40, 300), (300, 1500), (600, 520), (4200, 600), (200, 8000), (640, 4096)]
FILL = -77.0


def fn(name, kind):
    return getattr(tk, f"tk_{name}_{kind[0]}")


def flags(kind):
    return (tk.TK_RESIDUAL_F32 if kind[1] else 0) | (tk.TK_PARAMS_F32 if kind[2] else 0)


def types(kind):
    t = ref.DTYPES[kind[0]]
    return t, torch.float32 if kind[1] else t, torch.float32 if kind[2] else t


class Maker:
    """Matrices cut from wider buffers at an odd offset (pad > 0) or dense, and a check that
    nothing around the outputs was written."""

    def __init__(self, rows, cols, pad, seed):
        self.rows, self.cols, self.pad, self.outs = rows, cols, pad, []
        self.g = torch.Generator().manual_seed(seed)

    def place(self, dtype):
        ld = self.cols + self.pad
        lead = self.pad and 1 + self.pad % 3
        buf = torch.full((lead + self.rows * ld + 5,), FILL, dtype=dtype, device="cuda")
        return buf, buf[lead:lead + self.rows * ld].view(self.rows, ld)[:, :self.cols]

    def mat(self, dtype, scale=1.0, shift=0.0):
        v = (torch.randn(self.rows, self.cols, generator=self.g) * scale + shift).to(dtype)
        at = self.place(dtype)[1]
        at.copy_(v)
        return at, v.double()

    def vec(self, dtype, around=0.0, scale=0.3):
        v = (torch.randn(self.cols, generator=self.g) * scale + around).to(dtype)
        at = torch.empty(self.cols + 1, dtype=dtype, device="cuda")[self.pad % 2:][:self.cols]  # element-aligned only
        at.copy_(v)
        return at, v.double()

    def out(self, dtype):
        buf, at = self.place(dtype)
        self.outs.append((buf, at))
        return at

    def flat(self, n, dtype):
        buf = torch.full((n + 6,), FILL, dtype=dtype, device="cuda")
        self.outs.append((buf, buf[3:3 + n]))
        return buf[3:3 + n]

    def untouched(self, what):
        for buf, at in self.outs:
            rest = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(rest, at.shape, at.stride(), at.storage_offset()).fill_(False)
            assert bool((buf[rest] == FILL).all()), f"{what}: bytes around an output were written"


def cases(kind):
    for i, (rows, cols) in enumerate(SIZES):
        yield rows, cols, (0, 3, 8)[i % 3], i


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_dropout_add(kind):
    T, R, W = types(kind)
    for rows, cols, pad, i in cases(kind):
        for p, with_bias, with_res in ((0.0, True, True), (0.1, True, True), (0.5, False, True), (0.25, True, False),
                                       (0.7, False, False)):
            what = f"dropout_add {kind} {rows}x{cols} pad {pad} p {p} bias {with_bias} residual {with_res}"
            log(what)
            m = Maker(rows, cols, pad, i)
            x, xr = m.mat(T)
            b, br = m.vec(W) if with_bias else (None, None)
            r, rr = m.mat(R, 2.0) if with_res else (None, None)
            y = m.out(R)
            fn("dropout_add", kind)(8, 5 + i, rows, cols, p, flags(kind), x, None, b, r, None, y, None)
            keep = ref.keep_mask(8, 5 + i, rows, cols, p)
            ref.check(y, ref.dropout_add(xr, br, rr, keep, p), what)
            m.untouched(what)

            what = what.replace("add", "add_backward")
            m = Maker(rows, cols, pad, i + 1000)
            dy, dyr = m.mat(R)
            dx, db = m.out(T), m.flat(cols, W) if with_bias else None
            fn("dropout_add_backward", kind)(8, 5 + i, rows, cols, p, flags(kind), dy, None, dx, None, db)
            v, e = ref._dropped(dyr, torch.zeros_like(dyr), keep, p)
            ref.check(dx, (v, e), what)
            if with_bias:
                ref.check(db, ref.column_sum(v, e), what + " dbias")
            m.untouched(what)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_layer_norm(kind):
    T, R, W = types(kind)
    for rows, cols, pad, i in cases(kind):
        for affine, stats, eps, shift in ((True, True, 1e-5, 0.5), (False, False, 1e-2, 30.0)):
            what = f"layer_norm {kind} {rows}x{cols} pad {pad} affine {affine}"
            log(what)
            m = Maker(rows, cols, pad, i)
            x, xr = m.mat(R, 2.0, shift)
            g, gr = m.vec(W, 1.0) if affine else (None, None)
            b, br = m.vec(W) if affine else (None, None)
            y = m.out(T)
            mean, rstd = (m.flat(rows, torch.float32), m.flat(rows, torch.float32)) if stats else (None, None)
            fn("layer_norm", kind)(rows, cols, eps, flags(kind), x, None, g, b, y, None, mean, rstd)
            want = ref.layer_norm(xr, torch.zeros_like(xr), gr, br, eps)
            ref.check(y, want["y"], what + " y")
            if stats:
                ref.check(mean, want["mean"], what + " mean")
                ref.check(rstd, want["rstd"], what + " rstd")
            m.untouched(what)

            what = what.replace("norm", "norm_backward")
            m = Maker(rows, cols, pad, i + 1000)
            dy, dyr = m.mat(T)
            x, xr = m.mat(R, 2.0, shift)
            mu, rs = xr.mean(1).float(), (xr.var(1, unbiased=False) + eps).rsqrt().float()
            dx = m.out(R)
            dg, db = (m.flat(cols, W), m.flat(cols, W)) if affine else (None, None)
            fn("layer_norm_backward", kind)(rows, cols, flags(kind), dy, None, x, None, g, mu.cuda(), rs.cuda(), dx, None,
                                            dg, db)
            v, e, sums = ref.layer_norm_backward(dyr, xr, gr, mu.double(), rs.double())
            ref.check(dx, (v, e), what + " dx")
            if affine:
                ref.check(dg, sums["dgamma"], what + " dgamma")
                ref.check(db, sums["dbeta"], what + " dbeta")
            m.untouched(what)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_dropout_add_layer_norm(kind):
    T, R, W = types(kind)
    for rows, cols, pad, i in cases(kind):
        for p, with_bias, with_res, with_sum in ((0.1, True, True, True), (0.0, False, True, False), (0.4, True, False, True)):
            what = f"dropout_add_layer_norm {kind} {rows}x{cols} pad {pad} p {p} bias {with_bias} residual {with_res}"
            log(what)
            m = Maker(rows, cols, pad, i)
            x, xr = m.mat(T)
            b, br = m.vec(W) if with_bias else (None, None)
            r, rr = m.mat(R, 2.0) if with_res else (None, None)
            g, gr = m.vec(W, 1.0)
            t, tr = m.vec(W)
            s = m.out(R) if with_sum else None
            y, mean, rstd = m.out(T), m.flat(rows, torch.float32), m.flat(rows, torch.float32)
            fn("dropout_add_layer_norm", kind)(8, 9 + i, rows, cols, p, 1e-5, flags(kind), x, None, b, r, None, g, t, s,
                                               None, y, None, mean, rstd)
            keep = ref.keep_mask(8, 9 + i, rows, cols, p)
            v, e = ref.dropout_add(xr, br, rr, keep, p)
            want = ref.layer_norm(v, e, gr, tr, 1e-5)
            if with_sum:
                ref.check(s, (v, e), what + " sum")
            ref.check(y, want["y"], what + " y")
            ref.check(mean, want["mean"], what + " mean")
            ref.check(rstd, want["rstd"], what + " rstd")
            m.untouched(what)

            what = what.replace("norm", "norm_backward")
            m = Maker(rows, cols, pad, i + 1000)
            dy, dyr = m.mat(T)
            ds, dsr = m.mat(R) if with_sum else (None, None)
            v, vr = m.mat(R, 2.0)
            mu, rs = vr.mean(1).float(), (vr.var(1, unbiased=False) + 1e-5).rsqrt().float()
            dx, dr = m.out(T), m.out(R) if with_res else None
            dg, dt, db = m.flat(cols, W), m.flat(cols, W), m.flat(cols, W) if with_bias else None
            fn("dropout_add_layer_norm_backward", kind)(8, 9 + i, rows, cols, p, flags(kind), dy, None, ds, None, v, None, g,
                                                        mu.cuda(), rs.cuda(), dx, None, dr, None, dg, dt, db)
            want = ref.dropout_add_layer_norm_backward(dyr, dsr, vr, gr, mu.double(), rs.double(), keep, p)
            for name, got in (("dx", dx), ("dresidual", dr), ("dgamma", dg), ("dbeta", dt), ("dbias", db)):
                if got is not None:
                    ref.check(got, want[name], what + " " + name)
            m.untouched(what)


# ---- further properties ----

def run_block(kind, n, cols, m, p=0.1):
    """Inputs and outputs of one fused forward and backward, for the tests below."""
    T, R, W = types(kind)
    g = torch.Generator().manual_seed(m)
    rnd = lambda *s, k=1.0: torch.randn(*s, generator=g) * k  # noqa: E731
    d = {"x": rnd(n, cols).to(T), "r": rnd(n, cols, k=2.0).to(R), "bias": rnd(cols).to(W), "gamma": rnd(cols).to(W),
         "beta": rnd(cols).to(W), "dy": rnd(n, cols).to(T), "dsum": rnd(n, cols).to(R)}
    d = {k: v.cuda() for k, v in d.items()}
    for k, (shape, t) in {"sum": ((n, cols), R), "y": ((n, cols), T), "mean": ((n,), torch.float32),
                          "rstd": ((n,), torch.float32), "dx": ((n, cols), T), "dr": ((n, cols), R), "dg": ((cols,), W),
                          "db": ((cols,), W), "dbias": ((cols,), W)}.items():
        d[k] = torch.full(shape, FILL, dtype=t, device="cuda")
    d["ws"] = torch.empty(max(4, tk.tk_backward_workspace_bytes(n, cols)), dtype=torch.uint8, device="cuda")

    def go(stream=None):
        fn("dropout_add_layer_norm", kind)(8, 64, n, cols, p, 1e-5, flags(kind), d["x"], None, d["bias"], d["r"], None,
                                           d["gamma"], d["beta"], d["sum"], None, d["y"], None, d["mean"], d["rstd"],
                                           stream)
        fn("dropout_add_layer_norm_backward", kind)(8, 64, n, cols, p, flags(kind), d["dy"], None, d["dsum"], None, d["sum"],
                                                    None, d["gamma"], d["mean"], d["rstd"], d["dx"], None, d["dr"], None,
                                                    d["dg"], d["db"], d["dbias"], d["ws"], stream)
    return d, go


OUTS = ("sum", "y", "mean", "rstd", "dx", "dr", "dg", "db", "dbias")


def assert_same(a, b, what):
    for k in OUTS:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), f"{what}: {k}"


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_f32_dropout_add_is_dropout(kind):
    """Without bias and residual the float operator is tk_dropout_f32, bit for bit; the others
    keep the same elements."""
    T, R, _ = types(kind)
    n, cols = 301, 1003
    x = torch.randn(n, cols, device="cuda").to(T)
    x[x == 0] = 1
    last = (1 << 32) - n * cols  # the last counters there are
    for start, p in ((0, 0.1), (5, 0.5), (64, 0.999), (3, 1.0 - 2.0 ** -24), (0, 2.0 ** -25), (last, 0.3), (last - 5, 0.3),
                     ((1 << 16) - 3, 0.5)):
        y, want = torch.empty(n, cols, dtype=R, device="cuda"), torch.empty(n, cols, device="cuda")
        fn("dropout_add", kind)(9, start, n, cols, p, flags(kind), x, None, None, None, None, y, None)
        tk.tk_dropout_f32(9, start, n * cols, p, x.float(), want)
        if kind[0] == "f32":
            assert torch.equal(y.view(torch.int32), want.view(torch.int32))
        assert torch.equal(y == 0, want == 0), (start, p)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [5, 100, 1024, 4097, 16384, 33000])
def test_cut_calls_equal_the_whole(kind, cols):
    """Rows do not depend on each other: a call cut at any row, with the counters that belong to
    it, gives the whole call's rows, bit for bit (its column sums add up otherwise)."""
    T, R, W = types(kind)
    n, cut = 37, 11
    log(f"cut {kind} {cols}")
    whole, go = run_block(kind, n, cols, 3)
    go()
    for lo, hi in ((0, cut), (cut, n)):
        sub, _ = run_block(kind, n, cols, 3)
        f = {k: v[lo:hi] if v.dim() == 2 or k in ("mean", "rstd") else v for k, v in sub.items() if k != "ws"}
        fn("dropout_add_layer_norm", kind)(8, 64 + lo * cols, hi - lo, cols, 0.1, 1e-5, flags(kind), f["x"], None, f["bias"],
                                           f["r"], None, f["gamma"], f["beta"], f["sum"], None, f["y"], None, f["mean"],
                                           f["rstd"])
        fn("dropout_add_layer_norm_backward", kind)(8, 64 + lo * cols, hi - lo, cols, 0.1, flags(kind), f["dy"], None,
                                                    f["dsum"], None, f["sum"], None, f["gamma"], f["mean"], f["rstd"],
                                                    f["dx"], None, f["dr"], None, f["dg"], f["db"], f["dbias"])
        for k in ("sum", "y", "mean", "rstd", "dx", "dr"):
            assert torch.equal(f[k], whole[k][lo:hi]), (k, lo, hi)
            outside = torch.cat([sub[k][:lo], sub[k][hi:]])
            assert bool((outside == FILL).all()), f"{k}: rows of the other part were written"


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [3, 200, 1001, 4096, 9000, 33001])
def test_in_place(kind, cols):
    """Outputs in the place of inputs of the same type give the same bits."""
    T, R, _ = types(kind)
    n = 19
    log(f"in place {kind} {cols}")
    d, go = run_block(kind, n, cols, 4)
    go()
    same = T == R
    for sum_at, y_at in (("r", "x"), ("x" if same else "r", "r" if same else "x")):
        e, _ = run_block(kind, n, cols, 4)
        fn("dropout_add_layer_norm", kind)(8, 64, n, cols, 0.1, 1e-5, flags(kind), e["x"], None, e["bias"], e["r"], None,
                                           e["gamma"], e["beta"], e[sum_at], None, e[y_at], None, e["mean"], e["rstd"])
        assert torch.equal(e[sum_at], d["sum"]) and torch.equal(e[y_at], d["y"])
    for dr_at, dx_at in (("dsum", "dy"), ("sum", "dy")):
        e, _ = run_block(kind, n, cols, 4)
        for k in ("sum", "mean", "rstd"):
            e[k].copy_(d[k])
        fn("dropout_add_layer_norm_backward", kind)(8, 64, n, cols, 0.1, flags(kind), e["dy"], None, e["dsum"], None,
                                                    e["sum"], None, e["gamma"], e["mean"], e["rstd"], e[dx_at], None,
                                                    e[dr_at], None, e["dg"], e["db"], e["dbias"])
        assert torch.equal(e[dr_at], d["dr"]) and torch.equal(e[dx_at], d["dx"]) and torch.equal(e["dg"], d["dg"])
    y = torch.empty(n, cols, dtype=R, device="cuda")
    fn("dropout_add", kind)(2, 7, n, cols, 0.3, flags(kind), d["x"], None, d["bias"], d["r"], None, y, None)
    e, _ = run_block(kind, n, cols, 4)
    fn("dropout_add", kind)(2, 7, n, cols, 0.3, flags(kind), e["x"], None, e["bias"], e["r"], None, e["r"], None)
    assert torch.equal(e["r"], y)
    x2, y2 = torch.empty_like(y), torch.empty(n, cols, dtype=T, device="cuda")
    x2.copy_(d["r"])
    fn("layer_norm", kind)(n, cols, 1e-5, flags(kind), x2, None, d["gamma"], d["beta"], y2, None)
    if same:
        fn("layer_norm", kind)(n, cols, 1e-5, flags(kind), x2, None, d["gamma"], d["beta"], x2, None)
        assert torch.equal(x2, y2)


@pytest.mark.parametrize("kind", [k for k in KINDS if not k[1]], ids=[i for i, k in zip(IDS, KINDS) if not k[1]])
def test_slices_of_one_buffer(kind):
    """x and y as column slices of one buffer, read and written side by side."""
    T, R, W = types(kind)
    n, cols = 23, 1000
    d, go = run_block(kind, n, cols, 5)
    packed = torch.full((n, 3 * cols + 7), FILL, dtype=T, device="cuda")
    packed[:, 2:2 + cols] = d["x"]
    x, y = packed[:, 2:2 + cols], packed[:, 2 * cols + 5:3 * cols + 5]
    want = torch.empty(n, cols, dtype=T, device="cuda")
    fn("dropout_add", kind)(2, 7, n, cols, 0.3, flags(kind), d["x"], None, d["bias"], d["r"], None, want, None)
    fn("dropout_add", kind)(2, 7, n, cols, 0.3, flags(kind), x, None, d["bias"], d["r"], None, y, None)
    assert torch.equal(y, want) and torch.equal(x, d["x"])
    left = torch.cat([packed[:, :2], packed[:, 2 + cols:2 * cols + 5], packed[:, 3 * cols + 5:]], 1)
    assert bool((left == FILL).all())


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [64, 3000, 12000])
def test_special_values(kind, cols):
    """Constant rows, infinities and NaN follow the formulas; a dropped element is 0 whatever it was."""
    T, R, W = types(kind)
    n = 8
    g = torch.Generator().manual_seed(1)
    x = torch.randn(n, cols, generator=g).to(T)
    r = torch.randn(n, cols, generator=g).to(R)
    keep = ref.keep_mask(8, 0, n, cols, 0.5)
    kept, dropped = [[int(i) for i in (keep[k] == v).nonzero()[:, 0]] for k, v in ((1, 1), (1, 0))]
    x[0], r[0] = 0, 3.0              # a constant row: y = beta
    x[1, dropped[0]] = float("nan")  # dropped: no NaN anywhere
    x[1, dropped[1]] = float("inf")
    x[2, int((keep[2] == 1).nonzero()[0, 0])] = float("nan")
    r[3, 5] = float("inf")
    assert kept
    gm, bt = torch.randn(cols, generator=g).to(W), torch.randn(cols, generator=g).to(W)
    s, y = torch.empty(n, cols, dtype=R, device="cuda"), torch.empty(n, cols, dtype=T, device="cuda")
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    fn("dropout_add_layer_norm", kind)(8, 0, n, cols, 0.5, 1e-5, flags(kind), x.cuda(), None, None, r.cuda(), None,
                                       gm.cuda(), bt.cuda(), s, None, y, None, mean, rstd)
    v, e = ref.dropout_add(x.double(), None, r.double(), keep, 0.5)
    want = ref.layer_norm(v, e, gm.double(), bt.double(), 1e-5)
    for k in (0, 1, 4, 5, 6, 7):
        ref.check(s[k:k + 1], (v[k:k + 1], e[k:k + 1]), f"sum row {k}")
        ref.check(y[k:k + 1], (want["y"][0][k:k + 1], want["y"][1][k:k + 1]), f"y row {k}")
    assert torch.equal(y[0].cpu(), bt.to(T)), "a constant row gives beta"
    for k in (2, 3):
        assert bool(torch.isnan(y[k]).all()) and not bool(torch.isfinite(rstd[k]))
    # eps = 0: tiny variances keep their reciprocal root; a constant row has none
    x = (torch.randn(2, cols, generator=g, dtype=torch.float64) * 2.0 ** -55).float()
    x[1] = 1.0
    xr, yr = x.to(R), torch.empty(2, cols, dtype=T, device="cuda")
    fn("layer_norm", kind)(2, cols, 0.0, flags(kind), xr.cuda(), None, None, None, yr, None)
    if R != torch.float16:  # 2^-55 is no f16
        z = xr.double()[:1]
        w = ref.layer_norm(z, torch.zeros_like(z), None, None, 0.0)
        ref.check(yr[:1], w["y"], "tiny variance")
    assert bool(torch.isnan(yr[1]).all())


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_no_rows(kind):
    """Over no rows the forward calls write nothing and the gradients are zeros."""
    T, R, W = types(kind)
    cols = 100
    e = lambda t: torch.empty(0, cols, dtype=t, device="cuda")  # noqa: E731
    st = torch.empty(0, device="cuda")
    g, b, c = (torch.full((cols,), FILL, dtype=W, device="cuda") for _ in range(3))
    fn("layer_norm", kind)(0, cols, 1e-5, flags(kind), e(R), None, None, None, e(T), None)
    fn("dropout_add_layer_norm_backward", kind)(1, 0, 0, cols, 0.1, flags(kind), e(T), None, None, None, e(R), None, None, st,
                                                st, e(T), None, e(R), None, g, b, c)
    assert not g.any() and not b.any() and not c.any()
    c.fill_(FILL)
    fn("dropout_add_backward", kind)(1, 0, 0, cols, 0.1, flags(kind), e(R), None, e(T), None, c)
    assert not c.any()


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("shape", [(300, 768), (40, 9000)])
def test_captured_calls_replay_to_the_eager_result(kind, shape):
    """Forward and backward captured into two graphs with a workspace each; replayed in turn with
    eager work between, new inputs in place, and the outputs cleared."""
    want, go = run_block(kind, *shape, 6)
    go()
    want = {k: v.clone() for k, v in want.items()}
    other, go_other = run_block(kind, *shape, 7)
    go_other()
    want2 = {k: v.clone() for k, v in other.items()}
    runs = [run_block(kind, *shape, s) for s in (6, 7)]
    graphs = []
    for d, go in runs:
        go()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        graphs.append(g)
    for r in range(4):
        source = (want, want2)[r % 2]  # the first graph gets either's inputs
        for k in ("x", "r", "bias", "gamma", "beta", "dy", "dsum"):
            runs[0][0][k].copy_(source[k])
        for d, _ in runs:
            for k in OUTS:
                d[k].fill_(FILL)
        log(f"graph {kind} {shape} replay {r}")
        for g in graphs:
            g.replay()
        go_other()  # eager calls beside them
        torch.cuda.synchronize()
        assert_same(runs[0][0], source, f"replay {r}")
        assert_same(runs[1][0], want2, f"replay {r}, second graph")
    del graphs


def test_captured_calls_with_an_allocated_workspace():
    """A workspace of None inside a capture comes from the graph's own pool."""
    d, go = run_block(KINDS[3], 200, 1024, 8)
    go()
    want = {k: v.clone() for k, v in d.items()}
    back = tk.tk_dropout_add_layer_norm_backward_bf16
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        back(8, 64, 200, 1024, 0.1, 0, d["dy"], None, d["dsum"], None, d["sum"], None, d["gamma"], d["mean"], d["rstd"],
             d["dx"], None, d["dr"], None, d["dg"], d["db"], d["dbias"])
    for r in range(3):
        for k in ("dx", "dr", "dg", "db", "dbias"):
            d[k].fill_(FILL)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # would land in a freed workspace
        g.replay()
        torch.cuda.synchronize()
        assert_same(d, want, f"replay {r}")
        del junk


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[4]], ids=["f32", "bf16-r32"])
def test_two_streams(kind):
    """Two calls at once on two streams, each with its own workspace, and the same call again."""
    a, go_a = run_block(kind, 2000, 1000, 9)
    b, go_b = run_block(kind, 700, 9001, 10)
    go_a()
    go_b()
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in d.items()} for d in (a, b)]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for r in range(3):
        for d in (a, b):
            for k in OUTS:
                d[k].fill_(FILL)
        torch.cuda.synchronize()
        for _ in range(3):
            go_a(s)
            go_b(t)
        torch.cuda.synchronize()
        assert_same(a, want[0], f"stream a, round {r}")
        assert_same(b, want[1], f"stream b, round {r}")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [3, 40, 100, 200, 1000, 5001, 7000, 20000, 40000])
def test_large_calls(kind, cols):
    """Calls whose reads pass the caches (over 96 MB of them) against calls on quarters of their
    rows, most of which read through them: bit for bit by rows; and their column sums
    against float64 sums, which may be off by a half step of each term and of the sum."""
    T, R, W = types(kind)
    n, p = -(-52_000_000 // cols), 0.25
    log(f"large {kind} {n}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    mat = lambda t: torch.empty(n, cols, dtype=t, device="cuda").normal_(generator=g)  # noqa: E731
    vec = lambda: torch.randn(cols, generator=g, device="cuda").to(W)  # noqa: E731
    out = lambda t: torch.full((n, cols), FILL, dtype=t, device="cuda")  # noqa: E731
    x, r, dy, ds, bias, gamma, beta = mat(T), mat(R), mat(T), mat(R), vec(), vec(), vec()

    def go(lo, hi, o):
        m, sl, fl = hi - lo, slice(lo, hi), flags(kind)
        start = 40 + lo * cols
        fn("dropout_add", kind)(8, start, m, cols, p, fl, x[sl], None, bias, r[sl], None, o["add"][sl], None)
        fn("dropout_add", kind)(8, start, m, cols, p, fl, x[sl], None, None, None, None, o["drop"][sl], None)
        fn("dropout_add_backward", kind)(8, start, m, cols, p, fl, ds[sl], None, o["dx0"][sl], None, o["dbias0"])
        fn("dropout_add_layer_norm", kind)(8, start, m, cols, p, 1e-5, fl, x[sl], None, bias, r[sl], None, gamma, beta,
                                           o["sum"][sl], None, o["y"][sl], None, o["mean"][sl], o["rstd"][sl])
        fn("layer_norm", kind)(m, cols, 1e-5, fl, r[sl], None, gamma, beta, o["y1"][sl], None)
        fn("dropout_add_layer_norm_backward", kind)(8, start, m, cols, p, fl, dy[sl], None, ds[sl], None, o["sum"][sl], None,
                                                    gamma, o["mean"][sl], o["rstd"][sl], o["dx"][sl], None, o["dr"][sl],
                                                    None, o["dg"], o["db"], o["dbias"])

    def outs():
        o = {k: out(t) for k, t in (("add", R), ("drop", R), ("dx0", T), ("sum", R), ("y", T), ("y1", T), ("dx", T), ("dr", R))}
        o.update({k: torch.full((n,), FILL, device="cuda") for k in ("mean", "rstd")})
        o.update({k: torch.full((cols,), FILL, dtype=W, device="cuda") for k in ("dg", "db", "dbias", "dbias0")})
        return o

    whole, cut = outs(), outs()
    go(0, n, whole)
    for k in range(4):
        go(n * k // 4, n * (k + 1) // 4, cut)
    for k in ("add", "drop", "dx0", "sum", "y", "y1", "mean", "rstd", "dx", "dr"):
        assert torch.equal(whole[k], cut[k]), k
    h = (whole["sum"].double() - whole["mean"].double()[:, None]) * whole["rstd"].double()[:, None]
    for k, terms, half in (("dg", dy.double() * h, 4 * ref.U), ("db", dy.double(), 0.0),
                           ("dbias", whole["dx"].double(), torch.finfo(T).eps / 2),
                           ("dbias0", whole["dx0"].double(), torch.finfo(T).eps / 2)):
        size = terms.abs().sum(0)
        limit = size * (half + (n + 16) * ref.U)
        want = terms.sum(0)
        limit = limit + (want.abs() + limit) * torch.finfo(W).eps / 2 + n * ref.TINY[T]
        far = (whole[k].double() - want).abs() > limit
        assert not bool(far.any()), (k, int(far.sum()))


def test_very_long_rows():
    """More columns than one launch of the strips and of their sums covers (2^28 and 2^26): over one
    row the bias's gradient is dx, and each is dy over 1 - p or 0; over none it is 0."""
    cols = (1 << 28) + 777
    log("very long rows")
    dy = torch.full((1, cols), 0.75, device="cuda")
    dx, db = torch.full((1, cols), FILL, device="cuda"), torch.full((cols,), FILL, device="cuda")
    tk.tk_dropout_add_backward_f32(3, 9, 1, cols, 0.25, 0, dy, None, dx, None, db)
    assert torch.equal(dx[0], db)
    tk.tk_dropout_add_backward_f32(3, 9, 0, cols, 0.25, 0, dy[:0], None, dx[:0], None, db)
    assert not bool(db.any())
    kept = dx == 1.0
    assert bool((kept | (dx == 0)).all())
    tail = ref.keep_mask(3, 9 + cols - 5000, 1, 5000, 0.25)
    assert torch.equal(kept[:, -5000:].cpu().double(), tail)
    y = torch.empty_like(dx)
    tk.tk_dropout_add_f32(3, 9, 1, cols, 0.25, 0, dy, None, None, None, None, y, None)
    assert torch.equal(y, dx)


def test_binding_checks_on_the_device():
    """What the binding refuses of device tensors, before any launch."""
    x, y = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    call = tk.tk_layer_norm_f32
    with pytest.raises(ValueError, match="matrix"):
        call(4, 9, 1e-5, 0, x, None, None, None, y, None)
    with pytest.raises(ValueError, match="matrix"):
        call(4, 8, 1e-5, 0, x.t().contiguous().t(), None, None, None, y, None)
    with pytest.raises(ValueError, match="matrix"):
        call(4, 8, 1e-5, 0, torch.zeros(1, 8, device="cuda").expand(4, 8), None, None, None, y, None)
    with pytest.raises(ValueError, match="matrix"):
        call(4, 8, 1e-5, 0, x, 16, None, None, y, None)
    with pytest.raises(ValueError, match="vector"):
        call(4, 8, 1e-5, 0, x, None, torch.zeros(7, device="cuda"), None, y, None)
    with pytest.raises(ValueError, match="type"):
        tk.tk_layer_norm_bf16(4, 8, 1e-5, tk.TK_RESIDUAL_F32, x, None, None, None, y, None)
    with pytest.raises(tk.TkError):
        call(4, 8, -1.0, 0, x, None, None, None, y, None)
    mu = torch.zeros(4, device="cuda")
    many, stats, sums = torch.zeros(4000, 8, device="cuda"), torch.zeros(4000, device="cuda"), torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        tk.tk_layer_norm_backward_f32(4000, 8, 0, many, None, many, None, None, stats, stats, torch.empty_like(many), None,
                                      sums, None, None, torch.cuda.Stream())
    # one work-group's sums need none
    assert tk.tk_backward_workspace_bytes(4, 8) == 0
    torch.cuda.synchronize()
    tk.tk_layer_norm_backward_f32(4, 8, 0, x, None, x, None, None, mu, mu, y, None, sums, None, None, torch.cuda.Stream())
    tk.tk_layer_norm_backward_f32(4, 8, 0, x, None, x, None, None, mu, mu, y, None, sums, None, (0, 0))
    # a call that needs none takes none
    tk.tk_layer_norm_backward_f32(4, 8, 0, x, None, x, None, None, mu, mu, y, None, None, None, None, torch.cuda.Stream())
    torch.cuda.synchronize()
    # up to 8192 columns the gradients of the rows alone need none, beyond they do
    for cols, refused in ((8192, False), (8193, True)):
        z = torch.zeros(2, cols, device="cuda")
        args = (2, cols, 0, z, None, z, None, None, mu[:2], mu[:2], torch.empty_like(z), None, None, None)
        with pytest.raises(tk.TkError) if refused else contextlib.nullcontext():
            tk.tk_layer_norm_backward_f32(*args, (0, 0))
        tk.tk_layer_norm_backward_f32(*args)
    call(4, 8, 1e-5, 0, x.view(2, 2, 8), None, None, None, y, 8)  # any shape that flattens
    call(1, 8, 1e-5, 0, x[1:2], 100, None, None, y[:1], None)     # one row has no distance to a next
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_a_blocks_run(kind):
    """A transformer block's run of them, pre-norm: norm, a product, dropout-add with the next
    norm fused, a product, dropout-add; and back.  Against float64 autograd of the same block,
    on the values that the operators exchange in their own types."""
    T, R, W = types(kind)
    n, cols, p = 61, 520, 0.2
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s, k=1.0: torch.randn(*s, generator=g) * k  # noqa: E731
    x0 = rnd(n, cols, k=1.5).to(R)
    w1, w2 = (rnd(cols, cols, k=cols ** -0.5).to(T) for _ in range(2))
    prm = {k: (rnd(cols, k=0.3) + (1 if k[0] == "g" else 0)).to(W) for k in ("g1", "b1", "bias1", "g2", "b2", "bias2")}
    dout = rnd(n, cols).to(R)
    cu = {k: v.cuda() for k, v in prm.items()}
    fl, e = flags(kind), lambda t: torch.empty(n, cols, dtype=t, device="cuda")  # noqa: E731
    st = lambda: torch.empty(n, device="cuda")  # noqa: E731
    mm = lambda a, b: (a.float() @ b.float().cuda()).to(T)  # noqa: E731
    # forward
    x = x0.cuda()
    h1, m1, r1 = e(T), st(), st()
    fn("layer_norm", kind)(n, cols, 1e-5, fl, x, None, cu["g1"], cu["b1"], h1, None, m1, r1)
    a1 = mm(h1, w1)
    s, h2, m2, r2 = e(R), e(T), st(), st()
    fn("dropout_add_layer_norm", kind)(11, 0, n, cols, p, 1e-5, fl, a1, None, cu["bias1"], x, None, cu["g2"], cu["b2"], s,
                                       None, h2, None, m2, r2)
    a2 = mm(h2, w2)
    out = e(R)
    fn("dropout_add", kind)(12, 0, n, cols, p, fl, a2, None, cu["bias2"], s, None, out, None)
    # backward
    da2, gb2 = e(T), torch.empty(cols, dtype=W, device="cuda")
    fn("dropout_add_backward", kind)(12, 0, n, cols, p, fl, dout.cuda(), None, da2, None, gb2)
    dh2 = mm(da2, w2.t().contiguous())
    da1, dx = e(T), e(R)
    gg2, gt2, gb1 = (torch.empty(cols, dtype=W, device="cuda") for _ in range(3))
    fn("dropout_add_layer_norm_backward", kind)(11, 0, n, cols, p, fl, dh2, None, dout.cuda(), None, s, None, cu["g2"], m2,
                                                r2, da1, None, dx, None, gg2, gt2, gb1)
    dh1 = mm(da1, w1.t().contiguous())
    dx1 = e(R)
    gg1, gt1 = (torch.empty(cols, dtype=W, device="cuda") for _ in range(2))
    fn("layer_norm_backward", kind)(n, cols, fl, dh1, None, x, None, cu["g1"], m1, r1, dx1, None, gg1, gt1)
    got = {"x": (dx.double() + dx1.double()).cpu(), "g1": gg1, "b1": gt1, "bias1": gb1, "g2": gg2, "b2": gt2, "bias2": gb2}

    def block(x, g1, b1, bias1, g2, b2, bias2):
        ln = lambda v, a, b: torch.nn.functional.layer_norm(v, (cols,), a, b, 1e-5)  # noqa: E731
        k1, k2 = (ref.keep_mask(k, 0, n, cols, p) / ref.quotient(p) for k in (11, 12))
        v = x + k1 * (ln(x, g1, b1) @ w1.double() + bias1)
        return v + k2 * (ln(v, g2, b2) @ w2.double() + bias2)

    leaves = {k: v.double().requires_grad_() for k, v in {"x": x0, **prm}.items()}
    want = block(**leaves)
    want.backward(dout.double())
    # every value passes at most eight roundings to T or R between the inputs and a gradient, each
    # off by up to half a step, relative to values of the same size: 16 half steps of the coarsest
    # type, and twice that because a gradient is itself a difference of terms of its size
    half = torch.finfo(T).eps / 2
    rel = lambda a, b: float((a.detach().cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, want.detach()) <= 32 * half + 1e-5
    for k, v in got.items():
        assert rel(v, leaves[k].grad) <= 32 * half + 1e-5, k
