"""The row operators on the GPU against their 64-bit reference: dropout-add, layer norm and
both fused, forward and backward, at the sizes where a shape of kernel begins or ends, for
every pair of types; rows cut from wider buffers at odd addresses, whose neighbours must stay
as they were; in place; cut calls; captured calls; two streams; and a block's run of them."""
import numpy as np
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
         (1300, 136), (1201, 1032)]
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
        return v.cuda(), v.double()

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
