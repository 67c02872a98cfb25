"""The row operators (dropout-add, layer norm, both fused) in 64 bits, with bounds on what an
evaluation in f32 may be off.

Each function returns {name: (value, bound)}: the definition of include/tk.h evaluated in
float64 and, element by element, how far an f32 evaluation of it can lie from that before the
output is rounded to its type.  With u = 2^-24 (half a step of f32, relative), first-order:
- an operation adds u times its result;
- a sum of terms t_i in which no term passes more than K additions is off by at most
  K u sum |t_i|;
- errors of operands carry over through the partial derivatives.
`check` adds the rounding to the output's type: eps / 2 relative, or half of the smallest
subnormal.  Second-order terms are covered by a factor 1.01.

The keep decision is exact on both sides: the uniforms come from the C oracle.
"""
import numpy as np
import torch

import oracle

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def keep_mask(key, start, rows, cols, p):
    """Dropout's decision for every element, from the oracle's uniforms."""
    if p == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    u = oracle.fill_f32(key, start, rows * cols)
    return torch.from_numpy((u >= np.float32(p)).astype(np.float64)).view(rows, cols)


def quotient(p):
    """1 - p as the f32 operation gives it."""
    return float(np.float32(1.0) - np.float32(p))


def additions(cols):
    """At most how many additions a term of a row's sum passes: a thread's own elements (32, or
    one in 1024 of a wide row, chunk by chunk), six steps in a wave and sixteen waves."""
    return max(32, -(-cols // 1024) + 8) + 6 + 16


def _dropped(v, err, keep, p):
    """drop(v): the quotient's rounding, or a rounded reciprocal and a product (2 u)."""
    if p == 0:
        return v, err
    q = quotient(p)
    # a product with 0 would keep a dropped NaN; a dropped element is 0 whatever it was
    return torch.where(keep > 0, v / q, 0.0), torch.where(keep > 0, err / q + 2 * U * (v / q).abs(), 0.0)


def dropout_add(x, bias, residual, keep, p):
    z, e = x, torch.zeros_like(x)
    if bias is not None:
        z = x + bias
        e = U * z.abs()
    v, e = _dropped(z, e, keep, p)
    if residual is not None:
        v = v + residual
        e = e + U * v.abs()
    return v, e


def layer_norm(v, e, gamma, beta, eps):
    """From the norm's input and its error bound: y, mean, rstd."""
    cols = v.shape[1]
    k = additions(cols)
    mean = v.mean(1, keepdim=True)
    e_mean = e.mean(1, keepdim=True) + (k + 1) * U * v.abs().mean(1, keepdim=True)
    d = v - mean
    e_d = e + e_mean + U * d.abs()
    var = d.square().mean(1, keepdim=True)
    e_var = 2 * (d.abs() * e_d).mean(1, keepdim=True) + e_d.square().mean(1, keepdim=True) + (k + 2) * U * var
    rstd = (var + eps) ** -0.5
    rel = 0.5 * e_var / (var + eps) + 4 * U  # the sum with eps, the root and the reciprocal
    h = d * rstd
    e_h = rstd * e_d + h.abs() * (rel + 2 * U)
    g = torch.ones(cols, dtype=torch.float64) if gamma is None else gamma
    y = h * g + (0.0 if beta is None else beta)
    return {"y": (y, g.abs() * e_h + U * (h * g).abs() + U * y.abs()), "mean": (mean[:, 0], e_mean[:, 0]),
            "rstd": (rstd[:, 0], (rstd * rel)[:, 0])}


def column_sum(t, e):
    """Any order of additions: no term passes more than the number of rows, and a few."""
    return t.sum(0), e.sum(0) + (t.shape[0] + 16) * U * t.abs().sum(0)


def layer_norm_backward(dy, v, gamma, mean, rstd):
    """(gradient at the norm's input, its bound), and {dgamma, dbeta}.  mean and rstd are f32
    inputs."""
    cols = v.shape[1]
    k = additions(cols)
    mean, rstd = mean[:, None], rstd[:, None]
    h = (v - mean) * rstd
    e_h = 2 * U * h.abs()
    g = dy if gamma is None else dy * gamma
    e_g = U * g.abs()
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    ag, agh = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    e_mg, e_mgh = (k + 3) * U * ag, (k + 6) * U * agh
    inner = g - mg - h * mgh
    e_inner = e_g + e_mg + h.abs() * e_mgh + e_h * mgh.abs() + 3 * U * (g.abs() + mg.abs() + (h * mgh).abs())
    dv = rstd * inner
    return dv, rstd * e_inner + U * dv.abs(), {"dgamma": column_sum(dy * h, dy.abs() * (e_h + U * h.abs())),
                                               "dbeta": column_sum(dy, torch.zeros_like(dy))}


def dropout_add_layer_norm_backward(dy, dsum, v, gamma, mean, rstd, keep, p):
    dv, e, out = layer_norm_backward(dy, v, gamma, mean, rstd)
    if dsum is not None:
        dv = dv + dsum
        e = e + U * dv.abs()
    out["dresidual"] = (dv, e)
    dx, e = _dropped(dv, e, keep, p)
    out["dx"] = (dx, e)
    out["dbias"] = column_sum(dx, e)
    return out


def check(got, want, what):
    """`got` (a tensor of its own type) against (value, bound)."""
    value, bound = want
    t = got.dtype
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    limit = 1.01 * bound + (value.abs() + 1.01 * bound) * (torch.finfo(t).eps / 2) + TINY[t]
    big = torch.finfo(t).max
    far = ((got - value).abs() > limit) & (value.abs() < big)
    same = torch.isfinite(got) == torch.isfinite(value)
    over = value.abs() >= big  # rounds to infinity, or to the largest value
    bad = far | (~same & ~over) | (torch.isnan(got) != torch.isnan(value))
    bad |= torch.isinf(value) & (got != value)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]!r}, want "
                             f"{value[i]!r} within {limit[i]!r}")
