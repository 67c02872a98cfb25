"""The embedding, the head norms and the checkpoints in 64 bits, with bounds on what an evaluation in
f32 may be off (row_reference.py says how bounds are made, and checks against them).

Functions return {name: (value, bound)}, or for codes and scales the exact values: those follow from
the definition's own float operations, of which numpy's float32 ones are the correctly rounded results.
"""
import numpy as np
import torch

import oracle
import row_reference as ref
from row_reference import U

BLOCK = 128


def embedding(ids, table, keep, p, scale):
    """table in float64; ids int64, any of them outside the table."""
    there = (ids >= 0) & (ids < table.shape[0])
    z = torch.zeros(len(ids), table.shape[1], dtype=torch.float64)
    z[there] = table[ids[there]] * scale
    return ref._dropped(z, U * z.abs(), keep, p)


def embedding_backward(ids, dy, keep, p, scale, vocab, old=None):
    there = (ids >= 0) & (ids < vocab)
    v, e = ref._dropped(dy, torch.zeros_like(dy), keep, p)
    at = ids[there]
    total = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    sums = total.clone().index_add_(0, at, v[there])
    sizes = total.clone().index_add_(0, at, v[there].abs())
    errors = total.clone().index_add_(0, at, e[there])
    many = torch.bincount(at, minlength=vocab).double()[:, None] if len(at) else torch.zeros(vocab, 1, dtype=torch.float64)
    # no term passes more additions than there are rows of its token, and one for the first
    errors = errors + (many + 1) * U * sizes
    value = sums * scale
    bound = errors * abs(scale) + U * value.abs()
    if old is not None:
        value = value + old
        bound = bound + U * value.abs()
    return value, bound


def turned(x, cos, sin, interleaved):
    """The first pairs of x [rows, heads, dim] by the angles [rows, pairs], and the size of the products."""
    half = cos.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = cos[:, None], sin[:, None]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a], size[..., b] = (x[..., a] * c).abs(), (x[..., b] * c).abs()
    return y, size


def turned_bound(e, x, cos, sin, interleaved):
    """The bound after turning values of bound e: theirs carried over, one product's rounding and one
    fused multiply-add's."""
    y, size = turned(x, cos, sin, interleaved)
    half = cos.shape[1]
    out = turned(e, cos.abs(), -sin.abs(), interleaved)[0]
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    out[..., b] = e[..., b] * cos.abs()[:, None] + e[..., a] * sin.abs()[:, None]
    turns = torch.zeros_like(y)
    turns[..., :2 * half] = 1.0
    return y, out + turns * U * (size + y.abs())


# A head's sums: a lane's 16 elements and six steps over the lanes.
HEAD_ADDITIONS = 16 + 6


def head_norm(x, gamma, eps):
    ms = x.square().mean(-1, keepdim=True)
    rstd = (ms + eps) ** -0.5
    # the sum's roundings, its product with 1 / dim (both rounded) and the sum with eps; the root to two units
    rel = 0.5 * (HEAD_ADDITIONS + 4) * U + 4 * U
    h = x * rstd
    return rstd, rel, h, h.abs() * (rel + U)


def head_norm_rotate(x, gamma, cos, sin, interleaved, eps):
    rstd, rel, h, e = head_norm(x, gamma, eps)
    if gamma is not None:
        h, e = h * gamma, e * gamma.abs() + U * (h * gamma).abs()
    return turned_bound(e, h, cos, sin, interleaved)


def head_norm_rotate_backward(dy, x, gamma, cos, sin, interleaved, eps):
    rstd, rel, h, e_h = head_norm(x, gamma, eps)
    g, e_g = turned_bound(torch.zeros_like(dy), dy, cos, -sin, interleaved)
    t = g * h
    e_t = h.abs() * e_g + g.abs() * e_h + U * t.abs()
    dgamma = t.sum((0, 1)), e_t.sum((0, 1)) + (t.shape[0] * t.shape[1] + 16) * U * t.abs().sum((0, 1))
    if gamma is not None:
        g, e_g = g * gamma, e_g * gamma.abs() + U * (g * gamma).abs()
    m = (g * h).mean(-1, keepdim=True)
    e_m = (h.abs() * e_g + g.abs() * e_h).mean(-1, keepdim=True) + (HEAD_ADDITIONS + 3) * U * (g * h).abs().mean(-1, keepdim=True)
    inner = g - h * m
    e = e_g + h.abs() * e_m + m.abs() * e_h + U * ((h * m).abs() + inner.abs())
    dx = rstd * inner
    return {"dx": (dx, rstd * e + dx.abs() * (rel + U)), "dgamma": dgamma}


def checkpoint(x, key, start):
    """codes (int8) and scales of x, a float32 array."""
    rows, cols = x.shape
    n = -(-cols // BLOCK)
    wide = np.zeros((rows, n * BLOCK), np.float32)
    wide[:, :cols] = x
    blocks = wide.reshape(rows, n, BLOCK)
    with np.errstate(all="ignore"):
        most = np.abs(blocks).max(-1, keepdims=True)  # NaN where one is
        fine = np.isfinite(most)
        held = fine & (most >= np.float32(2.0 ** -100))
        scale = np.where(held, most / np.float32(127), np.where(fine, np.float32(0), np.float32(np.nan)))
        inverse = np.where(held, np.float32(127) / most, np.float32(0))
        t = np.where(held, np.abs(blocks) * inverse, np.float32(0))
    u = np.zeros((rows, n * BLOCK), np.float32)
    u[:, :cols] = oracle.fill_f32(key, start, rows * cols).reshape(rows, cols)
    up = u.reshape(blocks.shape) < t - np.floor(t)
    code = np.minimum(np.floor(t) + up, 127) * np.where(held, np.sign(blocks), np.float32(0))
    return code.astype(np.int8).reshape(rows, -1)[:, :cols], scale.astype(np.float32)[..., 0]


def restored(codes, scales):
    """The float values of codes (torch int8, float32), as float64."""
    at = torch.arange(codes.shape[1]) // BLOCK
    return (codes.float() * scales[:, at]).double()
