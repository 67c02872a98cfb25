"""The row operators' argument checks (no device: every call here is refused, or has nothing
to do), and the formulas of their 64-bit reference against differences."""
import ctypes as C

import numpy as np
import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref

L = tk.lib
OK, EINVAL, ERANGE = tk.TK_OK, tk.TK_EINVAL, tk.TK_ERANGE
A, B, D, E, F, G, H, W = (0x1000000 * k for k in range(1, 9))  # device addresses never dereferenced
WS = 1 << 40
TYPES = ["f32", "f16", "bf16"]
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def add(t, key=1, start=0, rows=4, cols=8, p=0.1, flags=0, x=A, ldx=8, bias=None, r=B, ldr=8, y=D, ldy=8):
    return getattr(L, "tk_dropout_add_" + t)(key, start, rows, cols, p, flags, x, ldx, bias, r, ldr, y, ldy, None)


def add_b(t, key=1, start=0, rows=4, cols=8, p=0.1, flags=0, dy=A, lddy=8, dx=B, lddx=8, dbias=None, ws=None, n=0):
    return getattr(L, "tk_dropout_add_backward_" + t)(key, start, rows, cols, p, flags, dy, lddy, dx, lddx, dbias, ws, n,
                                                      None)


def norm(t, rows=4, cols=8, eps=1e-5, flags=0, x=A, ldx=8, gamma=None, beta=None, y=B, ldy=8, mean=None, rstd=None):
    return getattr(L, "tk_layer_norm_" + t)(rows, cols, eps, flags, x, ldx, gamma, beta, y, ldy, mean, rstd, None)


def norm_b(t, rows=4, cols=8, flags=0, dy=A, lddy=8, x=B, ldx=8, gamma=None, mean=D, rstd=E, dx=F, lddx=8, dgamma=None,
           dbeta=None, ws=None, n=0):
    return getattr(L, "tk_layer_norm_backward_" + t)(rows, cols, flags, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx,
                                                     dgamma, dbeta, ws, n, None)


def both(t, start=0, rows=4, cols=8, p=0.1, eps=1e-5, flags=0, x=A, ldx=8, bias=None, r=B, ldr=8, gamma=None, beta=None,
         s=D, lds=8, y=E, ldy=8, mean=None, rstd=None):
    return getattr(L, "tk_dropout_add_layer_norm_" + t)(1, start, rows, cols, p, eps, flags, x, ldx, bias, r, ldr, gamma,
                                                        beta, s, lds, y, ldy, mean, rstd, None)


def both_b(t, start=0, rows=4, cols=8, p=0.1, flags=0, dy=A, lddy=8, ds=None, ldds=8, s=B, lds=8, gamma=None, mean=D,
           rstd=E, dx=F, lddx=8, dr=G, lddr=8, dgamma=None, dbeta=None, dbias=None, ws=None, n=0):
    return getattr(L, "tk_dropout_add_layer_norm_backward_" + t)(
        1, start, rows, cols, p, flags, dy, lddy, ds, ldds, s, lds, gamma, mean, rstd, dx, lddx, dr, lddr, dgamma, dbeta,
        dbias, ws, n, None)


CALLS = [add, add_b, norm, norm_b, both, both_b]


@pytest.mark.parametrize("t", TYPES)
def test_nothing_to_do(t):
    for f in CALLS:
        assert f(t, cols=0) == OK, f.__name__
        assert f(t, rows=0) == OK, f.__name__
    assert add(t, rows=0, x=None, y=None) == OK
    assert norm(t, cols=0, x=None, y=None) == OK


@pytest.mark.parametrize("t", TYPES)
def test_bad_numbers(t):
    for p in (1.0, -0.25, float("nan"), float("inf")):
        for f in (add, add_b, both, both_b):
            assert f(t, p=p) == EINVAL, (f.__name__, p)
            assert f(t, p=p, rows=0) == EINVAL
    for eps in (-1e-9, float("nan"), float("inf")):
        for f in (norm, both):
            assert f(t, eps=eps) == EINVAL, (f.__name__, eps)
    for f in CALLS:
        assert f(t, flags=4) == EINVAL, f.__name__
        assert f(t, rows=1 << 31) == ERANGE, f.__name__
        assert f(t, cols=1 << 31) == ERANGE, f.__name__
        assert f(t, rows=(1 << 64) - 1) == ERANGE, f.__name__
    for f in (add, add_b, both, both_b):
        assert f(t, start=(1 << 32) - 31) == ERANGE, f.__name__
        assert f(t, start=1 << 63) == ERANGE, f.__name__
        assert f(t, rows=1 << 20, cols=(1 << 12) + 1) == ERANGE, f.__name__


@pytest.mark.parametrize("t", TYPES)
def test_missing_misaligned_and_short_rows(t):
    for f, names in ((add, ("x", "y")), (add_b, ("dy", "dx")), (norm, ("x", "y")), (norm_b, ("dy", "x", "mean", "rstd", "dx")),
                     (both, ("x", "y")), (both_b, ("dy", "s", "mean", "rstd", "dx"))):
        for name in names:
            assert f(t, **{name: None}) == EINVAL, (f.__name__, name)
            assert f(t, **{name: A * 8 + 1}) == EINVAL, (f.__name__, name)
    for f, names in ((add, ("ldx", "ldr", "ldy")), (add_b, ("lddy", "lddx")), (norm, ("ldx", "ldy")),
                     (norm_b, ("lddy", "ldx", "lddx")), (both, ("ldx", "ldr", "lds", "ldy")),
                     (both_b, ("lddy", "lds", "lddx", "lddr"))):
        for name in names:
            assert f(t, **{name: 7}) == EINVAL, (f.__name__, name)
            assert f(t, **{name: 1 << 31}) == ERANGE, (f.__name__, name)
    for name in ("bias", "gamma", "beta", "mean", "rstd"):
        assert both(t, **{name: H + 1}) == EINVAL
    for name in ("dgamma", "dbeta", "dbias"):
        assert both_b(t, **{name: H + 1}, ws=WS, n=1 << 30) == EINVAL


@pytest.mark.parametrize("t", TYPES)
def test_flags_change_the_alignment(t):
    """A 16-bit operator with a float residual stream or float parameters refuses addresses that
    are only 2-byte aligned for those."""
    assert add(t, flags=tk.TK_RESIDUAL_F32, r=B + 2) == EINVAL
    assert add(t, flags=tk.TK_RESIDUAL_F32, y=D + 2) == EINVAL
    assert norm(t, flags=tk.TK_RESIDUAL_F32, x=A + 2) == EINVAL
    assert add(t, flags=tk.TK_PARAMS_F32, bias=H + 2) == EINVAL
    assert norm(t, flags=tk.TK_PARAMS_F32, gamma=H + 2) == EINVAL


@pytest.mark.parametrize("t", TYPES)
def test_overlaps(t):
    z = SIZE[t]
    assert add(t, y=A + z) == EINVAL                       # shifted by an element
    assert add(t, y=A, ldy=9) == EINVAL                    # the input's address with another pitch
    assert add(t, bias=D + 8 * z) == EINVAL                # a bias inside the output
    assert add(t, ldx=16, ldy=16, y=A + 7 * z) == EINVAL   # slices of one buffer that share a column
    assert add(t, ldx=16, ldy=16, ldr=16, y=A + 16 * 2 * z + 9 * z, rows=4) == EINVAL  # ... across a row's end
    assert norm(t, mean=B) == EINVAL                       # statistics inside the output
    assert norm(t, mean=D, rstd=D + 8) == EINVAL
    assert both(t, s=E) == EINVAL                          # both outputs in one place
    assert both(t, gamma=E) == EINVAL
    assert both_b(t, dx=G) == EINVAL
    assert both_b(t, dgamma=H, dbeta=H, ws=WS, n=1 << 30) == EINVAL
    assert both_b(t, dgamma=H, rows=4000, ws=H, n=1 << 30) == EINVAL
    assert both_b(t, dgamma=H, rows=4000, ws=F, n=1 << 30) == EINVAL
    if t != "f32":
        assert add(t, flags=tk.TK_RESIDUAL_F32, y=A) == EINVAL  # one address, two types


@pytest.mark.parametrize("t", TYPES)
def test_workspace(t):
    need = tk.tk_backward_workspace_bytes(4000, 8)
    assert need > 0
    for f in (add_b, norm_b, both_b):
        name = "dbias" if f is add_b else "dgamma"
        assert f(t, rows=4000, **{name: H}) == EINVAL
        assert f(t, rows=4000, **{name: H}, ws=WS, n=need - 1) == EINVAL
        assert f(t, rows=4000, **{name: H}, ws=WS + 2, n=need) == EINVAL
    # wide rows need one even without parameter gradients
    assert norm_b(t, cols=8193, lddy=8193, ldx=8193, lddx=8193) == EINVAL
    assert tk.tk_backward_workspace_bytes(4, 8) == 0  # one work-group's sums
    assert tk.tk_backward_workspace_bytes(0, 8) == 0 and tk.tk_backward_workspace_bytes(8, 0) == 0
    v = C.c_uint64()
    assert L.tk_backward_workspace_bytes(4, 8, None) == EINVAL
    assert L.tk_backward_workspace_bytes(1 << 31, 8, C.byref(v)) == ERANGE
    assert L.tk_backward_workspace_bytes(8, 1 << 31, C.byref(v)) == ERANGE


@pytest.mark.parametrize("cols", [1, 5, 8, 40, 64, 129, 300, 513, 1024, 1500, 2049, 4096, 5001, 8192, 8193, 20000, 70001,
                                  140000])
def test_a_workspace_serves_fewer_rows(cols):
    rows = list(range(1, 1500)) + list(range(1500, 80000, 997)) + [1 << 20, (1 << 20) + 1, 1 << 30]
    sizes = [tk.tk_backward_workspace_bytes(r, cols) for r in rows]
    assert sizes == sorted(sizes)


def test_binding_refuses_bad_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="HIP device"):
        tk.tk_dropout_add_f32(1, 0, 4, 8, 0.1, 0, x, None, None, None, None, x, None)
    with pytest.raises(ValueError, match="type"):
        tk.tk_layer_norm_bf16(4, 8, 1e-5, 0, x, None, None, None, x, None)
    with pytest.raises(ValueError, match="type"):
        tk.tk_layer_norm_f32(4, 8, 1e-5, 0, x.double(), None, None, None, x, None)


def directional(f, at, name, seed):
    """The central difference of f along a random direction of one of its arguments."""
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(at[name].shape, generator=g, dtype=torch.float64)
    h = 1e-5
    up, down = (f(**{**at, name: at[name] + s * h * d}) for s in (1, -1))
    return (up - down) / (2 * h), d


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_reference_gradients_are_those_of_differences(p):
    """The backward formulas of the reference against central differences of its forward ones
    (float64, step 1e-5: truncation about 1e-10 of the values, rounding about 1e-11)."""
    rows, cols = 6, 37
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    keep = ref.keep_mask(3, 11, rows, cols, p)
    assert p == 0 or 0 < keep.sum() < keep.numel()
    at = {"x": rnd(rows, cols), "bias": rnd(cols), "residual": rnd(rows, cols), "gamma": rnd(cols), "beta": rnd(cols)}
    dy, dsum = rnd(rows, cols), rnd(rows, cols)

    def loss(x, bias, residual, gamma, beta):
        v, e = ref.dropout_add(x, bias, residual, keep, p)
        return float((ref.layer_norm(v, e, gamma, beta, 1e-3)["y"][0] * dy).sum() + (v * dsum).sum())

    v, e = ref.dropout_add(at["x"], at["bias"], at["residual"], keep, p)
    st = ref.layer_norm(v, e, at["gamma"], at["beta"], 1e-3)
    out = ref.dropout_add_layer_norm_backward(dy, dsum, v, at["gamma"], st["mean"][0], st["rstd"][0], keep, p)
    for name, grad in (("x", "dx"), ("bias", "dbias"), ("residual", "dresidual"), ("gamma", "dgamma"), ("beta", "dbeta")):
        slope, d = directional(loss, at, name, 9)
        assert abs(slope - float((out[grad][0] * d).sum())) <= 1e-7 * (1 + abs(slope)), name


def test_reference_norm_is_torchs():
    x, g, b = torch.randn(5, 33, dtype=torch.float64), torch.randn(33, dtype=torch.float64), torch.randn(33, dtype=torch.float64)
    y = ref.layer_norm(x, torch.zeros_like(x), g, b, 1e-5)["y"][0]
    assert np.allclose(y, torch.nn.functional.layer_norm(x, (33,), g, b, 1e-5), rtol=1e-12, atol=1e-12)
