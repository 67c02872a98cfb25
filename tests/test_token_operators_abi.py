"""The argument checks of the embedding, the head norms and the checkpoints (no device: every call here
is refused, or has nothing to do), and the formulas of their 64-bit reference against differences."""
import ctypes as C

import numpy as np
import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref
import token_reference as tok
from test_row_operators_abi import directional

L = tk.lib
OK, EINVAL, ERANGE = tk.TK_OK, tk.TK_EINVAL, tk.TK_ERANGE
A, B, D, E, F, G, H, I, J, K, M = (0x1000000 * k for k in range(1, 12))  # device addresses never dereferenced
WS, BIG = 1 << 40, 1 << 36
TYPES = ["f32", "f16", "bf16"]
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def emb(t, start=0, rows=4, cols=8, p=0.1, scale=2.0, flags=0, vocab=10, ids=A, table=B, ldt=8, y=D, ldy=8):
    return getattr(L, "tk_embedding_" + t)(1, start, rows, cols, p, scale, flags, vocab, ids, table, ldt, y, ldy, None)


def emb_b(t, start=0, rows=4, cols=8, p=0.1, scale=2.0, flags=0, vocab=10, ids=A, dy=B, lddy=8, dt=D, lddt=8, ws=WS, n=BIG):
    return getattr(L, "tk_embedding_backward_" + t)(1, start, rows, cols, p, scale, flags, vocab, ids, dy, lddy, dt, lddt, ws,
                                                    n, None)


def head(t, rows=4, hq=4, hk=2, dim=8, rotary=8, eps=1e-5, flags=0, q=A, ldq=32, k=B, ldk=16, gq=None, gk=None, pos=None,
         tab=100, cos=D, sin=E, yq=F, ldyq=32, yk=G, ldyk=16):
    return getattr(L, "tk_head_norm_rotate_" + t)(rows, hq, hk, dim, rotary, eps, flags, q, ldq, k, ldk, gq, gk, pos, tab, cos,
                                                  sin, yq, ldyq, yk, ldyk, None)


def head_b(t, rows=4, hq=4, hk=2, dim=8, rotary=8, eps=1e-5, flags=0, dyq=H, lddyq=32, dyk=I, lddyk=16, q=A, ldq=32, k=B,
           ldk=16, gq=None, gk=None, pos=None, tab=100, cos=D, sin=E, dq=F, lddq=32, dk=G, lddk=16, dgq=None, dgk=None,
           ws=None, n=0):
    return getattr(L, "tk_head_norm_rotate_backward_" + t)(rows, hq, hk, dim, rotary, eps, flags, dyq, lddyq, dyk, lddyk, q,
                                                           ldq, k, ldk, gq, gk, pos, tab, cos, sin, dq, lddq, dk, lddk, dgq,
                                                           dgk, ws, n, None)


def pack(t, start=0, rows=4, cols=8, flags=0, x=A, ldx=8, codes=B, ldc=8, scales=D):
    return getattr(L, "tk_checkpoint_" + t)(1, start, rows, cols, flags, x, ldx, codes, ldc, scales, None)


def unpack(t, rows=4, cols=8, flags=0, codes=B, ldc=8, scales=D, y=A, ldy=8):
    return getattr(L, "tk_checkpoint_restore_" + t)(rows, cols, flags, codes, ldc, scales, y, ldy, None)


def norm_c(t, rows=4, cols=8, flags=0, dy=A, lddy=8, codes=B, ldc=8, scales=H, gamma=None, mean=D, rstd=E, dx=F, lddx=8,
           dgamma=None, dbeta=None, ws=None, n=0):
    return getattr(L, "tk_layer_norm_backward_checkpoint_" + t)(rows, cols, flags, dy, lddy, codes, ldc, scales, gamma, mean,
                                                                rstd, dx, lddx, dgamma, dbeta, ws, n, None)


def both_c(t, start=0, rows=4, cols=8, p=0.1, flags=0, dy=A, lddy=8, ds=None, ldds=8, codes=B, ldc=8, scales=H, gamma=None,
           mean=D, rstd=E, dx=F, lddx=8, dr=G, lddr=8, dgamma=None, dbeta=None, dbias=None, ws=None, n=0):
    return getattr(L, "tk_dropout_add_layer_norm_backward_checkpoint_" + t)(
        1, start, rows, cols, p, flags, dy, lddy, ds, ldds, codes, ldc, scales, gamma, mean, rstd, dx, lddx, dr, lddr, dgamma,
        dbeta, dbias, ws, n, None)


CALLS = [emb, emb_b, head, head_b, pack, unpack, norm_c, both_c]


@pytest.mark.parametrize("t", TYPES)
def test_nothing_to_do(t):
    for f in (emb, pack, unpack, norm_c, both_c):
        assert f(t, rows=0) == OK, f.__name__
        assert f(t, cols=0) == OK, f.__name__
    assert emb(t, rows=0, ids=None, table=None, y=None) == OK
    assert emb_b(t, cols=0, dt=None) == OK
    assert emb_b(t, vocab=0, dt=None) == OK
    assert emb_b(t, rows=0, flags=tk.TK_ACCUMULATE, dt=None) == OK
    for f in (head, head_b):
        assert f(t, rows=0) == OK and f(t, dim=0, rotary=0) == OK and f(t, hq=0, hk=0) == OK
    assert pack(t, cols=0, x=None, codes=None, scales=None) == OK


@pytest.mark.parametrize("t", TYPES)
def test_bad_numbers(t):
    nan, inf = float("nan"), float("inf")
    for p in (1.0, -0.25, nan, inf):
        for f in (emb, emb_b, both_c):
            assert f(t, p=p) == EINVAL and f(t, p=p, rows=0) == EINVAL, (f.__name__, p)
    for s in (nan, inf, -inf):
        assert emb(t, scale=s) == EINVAL and emb_b(t, scale=s) == EINVAL
    for eps in (-1e-9, nan, inf):
        assert head(t, eps=eps) == EINVAL and head_b(t, eps=eps) == EINVAL
    for f in CALLS:
        assert f(t, flags=4) == EINVAL, f.__name__
        assert f(t, flags=64) == EINVAL, f.__name__
        assert f(t, rows=1 << 31) == ERANGE, f.__name__
        assert f(t, rows=(1 << 64) - 1) == ERANGE, f.__name__
    # flags of other operators
    assert emb(t, flags=tk.TK_ACCUMULATE) == EINVAL and emb(t, flags=tk.TK_INTERLEAVED) == EINVAL
    assert emb_b(t, flags=tk.TK_INTERLEAVED) == EINVAL
    for f in (head, head_b):
        assert f(t, flags=tk.TK_RESIDUAL_F32) == EINVAL and f(t, flags=tk.TK_ACCUMULATE) == EINVAL
        assert f(t, rotary=7) == EINVAL and f(t, rotary=10) == EINVAL
        assert f(t, dim=513, rotary=8) == ERANGE
        assert f(t, hq=1 << 31) == ERANGE and f(t, hk=1 << 31) == ERANGE
        assert f(t, hq=1 << 28, ldq=(1 << 31) - 1) == ERANGE  # a row's elements
        assert f(t, tab=1 << 31) == ERANGE
        assert f(t, rows=1 << 30, hq=1, hk=1, ldq=8, ldk=8) == ERANGE  # the heads of all rows
    for f in (pack, unpack):
        for bad in (tk.TK_PARAMS_F32, tk.TK_INDEX_I64, tk.TK_ACCUMULATE):
            assert f(t, flags=bad) == EINVAL
    for f in (norm_c, both_c):
        assert f(t, flags=tk.TK_INDEX_I64) == EINVAL
    for f in (emb, emb_b, pack, unpack, norm_c, both_c):
        assert f(t, cols=1 << 31) == ERANGE, f.__name__
    for f in (emb, emb_b):
        assert f(t, vocab=1 << 31) == ERANGE
    for f in (emb, emb_b, pack, both_c):
        assert f(t, start=(1 << 32) - 31) == ERANGE, f.__name__
        assert f(t, start=1 << 63) == ERANGE, f.__name__
        assert f(t, rows=1 << 20, cols=(1 << 12) + 1) == ERANGE, f.__name__


@pytest.mark.parametrize("t", TYPES)
def test_missing_misaligned_and_short_rows(t):
    needed = ((emb, ("ids", "table", "y")), (emb_b, ("ids", "dy", "dt")), (head, ("q", "k", "cos", "sin", "yq", "yk")),
              (head_b, ("dyq", "dyk", "q", "k", "cos", "sin", "dq", "dk")), (pack, ("x", "scales")), (unpack, ("scales", "y")),
              (norm_c, ("dy", "scales", "mean", "rstd", "dx")), (both_c, ("dy", "scales", "mean", "rstd", "dx")))
    for f, names in needed:
        for name in names:
            assert f(t, **{name: None}) == EINVAL, (f.__name__, name)
            assert f(t, **{name: A * 64 + 1}) == EINVAL, (f.__name__, name)
    for f in (pack, unpack, norm_c, both_c):  # codes are bytes
        assert f(t, codes=None) == EINVAL
    for f, names, short in ((emb, ("ldt", "ldy"), 7), (emb_b, ("lddy", "lddt"), 7), (head, ("ldq", "ldyq"), 31),
                            (head, ("ldk", "ldyk"), 15), (head_b, ("lddyq", "ldq", "lddq"), 31),
                            (head_b, ("lddyk", "ldk", "lddk"), 15), (pack, ("ldx", "ldc"), 7), (unpack, ("ldc", "ldy"), 7),
                            (norm_c, ("lddy", "ldc", "lddx"), 7), (both_c, ("lddy", "ldc", "lddx", "lddr"), 7)):
        for name in names:
            assert f(t, **{name: short}) == EINVAL, (f.__name__, name)
            assert f(t, **{name: 1 << 31}) == ERANGE, (f.__name__, name)
    for f in (head, head_b):
        assert f(t, gq=J + 1) == EINVAL and f(t, gk=J + 1) == EINVAL and f(t, pos=J + 2) == EINVAL
        assert f(t, pos=J + 4, flags=tk.TK_INDEX_I64) == EINVAL
    assert emb(t, ids=A + 4, flags=tk.TK_INDEX_I64) == EINVAL
    assert emb(t, vocab=0, table=None, y=None) == EINVAL  # y is still to be written
    for f in (head_b,):
        assert f(t, dgq=J + 1, ws=WS, n=BIG) == EINVAL and f(t, dgk=J + 1, ws=WS, n=BIG) == EINVAL
    # a side without heads needs nothing, tables without pairs or rows neither
    assert head(t, rows=4, hq=0, hk=2, yk=None) == EINVAL
    if t != "f32":
        assert emb(t, flags=tk.TK_RESIDUAL_F32, y=D + 2) == EINVAL
        assert emb(t, flags=tk.TK_PARAMS_F32, table=B + 2) == EINVAL
        assert head(t, flags=tk.TK_PARAMS_F32, gq=J + 2) == EINVAL
        assert pack(t, flags=tk.TK_RESIDUAL_F32, x=A + 2) == EINVAL


@pytest.mark.parametrize("t", TYPES)
def test_overlaps(t):
    z = SIZE[t]
    assert emb(t, y=B) == EINVAL and emb(t, y=B, vocab=4) == EINVAL     # the output in the table, also of its very shape
    assert emb(t, y=A) == EINVAL                                        # ... in the ids
    assert emb_b(t, dt=B, vocab=4) == EINVAL and emb_b(t, dt=A) == EINVAL
    assert emb_b(t, ws=B) == EINVAL and emb_b(t, ws=D) == EINVAL and emb_b(t, ws=A) == EINVAL
    assert head(t, yq=A + z) == EINVAL and head(t, yq=A, ldyq=33) == EINVAL
    assert head(t, yq=B) == EINVAL                                      # the queries' output in the keys
    assert head(t, hq=2, ldq=16, yq=B, ldyq=16) == EINVAL               # ... also of their very shape
    assert head(t, yk=F) == EINVAL and head(t, yq=D) == EINVAL and head(t, yq=J, pos=J) == EINVAL
    assert head(t, yk=J, gk=J) == EINVAL
    # slices of one buffer: q's 32 columns, then k's 16; one that shares a column
    assert head(t, q=A, ldq=48, k=A + 32 * z, ldk=48, yq=J, ldyq=48, yk=J + 31 * z, ldyk=48) == EINVAL
    assert head_b(t, dq=G) == EINVAL and head_b(t, dq=I) == EINVAL and head_b(t, dk=A) == EINVAL
    assert head_b(t, dgq=J, dgk=J, ws=WS, n=BIG) == EINVAL
    assert head_b(t, dgq=J, ws=J, n=BIG) == EINVAL and head_b(t, dgq=J, ws=F, n=BIG) == EINVAL
    assert pack(t, codes=A) == EINVAL and pack(t, scales=A) == EINVAL and pack(t, scales=B) == EINVAL
    assert unpack(t, y=B) == EINVAL and unpack(t, y=D) == EINVAL
    for f in (norm_c, both_c):
        assert f(t, dx=B) == EINVAL and f(t, dx=H) == EINVAL and f(t, dgamma=B, ws=WS, n=BIG) == EINVAL


@pytest.mark.parametrize("t", TYPES)
def test_workspaces(t):
    need = tk.tk_embedding_workspace_bytes(400, 8, 10)
    assert need > 0
    for ws, n in ((None, BIG), (WS, need - 1), (WS + 2, need)):
        assert emb_b(t, rows=400, ws=ws, n=n) == EINVAL
    need = tk.tk_head_norm_workspace_bytes(4, 4, 2, 8)
    assert need > 0
    for ws, n in ((None, BIG), (WS, need - 1), (WS + 2, need)):
        assert head_b(t, dgq=J, ws=ws, n=n) == EINVAL and head_b(t, dgk=J, ws=ws, n=n) == EINVAL
    need = tk.tk_backward_workspace_bytes(4000, 8)
    for f in (norm_c, both_c):
        for ws, n in ((None, BIG), (WS, need - 1), (WS + 2, need)):
            assert f(t, rows=4000, dgamma=J, ws=ws, n=n) == EINVAL
    assert norm_c(t, cols=8193, lddy=8193, ldc=8193, lddx=8193) == EINVAL  # wide rows need one without gradients too


def test_workspace_sizes():
    for cols, vocab in ((1, 1), (8, 10), (4096, 32768), (1001, 50001)):
        rows = list(range(1, 300)) + [2 ** k + d for k in range(9, 31) for d in (-1, 0, 1)]
        sizes = [tk.tk_embedding_workspace_bytes(r, cols, vocab) for r in rows]
        assert sizes == sorted(sizes)
    assert tk.tk_embedding_workspace_bytes(0, 8, 8) == tk.tk_embedding_workspace_bytes(8, 0, 8) == 0
    assert tk.tk_embedding_workspace_bytes(8, 8, 0) == 0
    assert tk.tk_head_norm_workspace_bytes(0, 4, 2, 8) == tk.tk_head_norm_workspace_bytes(4, 0, 0, 8) == 0
    for dim in (1, 64, 65, 512):
        sizes = [tk.tk_head_norm_workspace_bytes(r, 4, 2, dim) for r in (1, 2, 100, 1 << 20, (1 << 28) - 1)]
        assert sizes == sorted(sizes)
    v = C.c_uint64()
    assert L.tk_embedding_workspace_bytes(4, 8, 8, None) == EINVAL
    assert L.tk_head_norm_workspace_bytes(4, 8, 8, 8, None) == EINVAL
    for bad in ((1 << 31, 8, 8), (8, 1 << 31, 8), (8, 8, 1 << 31)):
        assert L.tk_embedding_workspace_bytes(*bad, C.byref(v)) == ERANGE
    for bad in ((1 << 31, 8, 8, 8), (8, 1 << 31, 8, 8), (8, 8, 1 << 31, 8), (8, 8, 8, 513)):
        assert L.tk_head_norm_workspace_bytes(*bad, C.byref(v)) == ERANGE


class OtherStream:
    """A stream of another device than the current one."""
    device_index, cuda_stream = 7, 0


def test_binding_refusals(monkeypatch):
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="type"):  # int64 ids need their flag
        tk.tk_embedding_f32(1, 0, 4, 8, 0.0, 1.0, 0, 10, ids, None, None, x, None)
    with pytest.raises(ValueError, match="HIP device"):
        tk.tk_embedding_f32(1, 0, 4, 8, 0.0, 1.0, tk.TK_INDEX_I64, 10, ids, None, None, x, None)
    with pytest.raises(ValueError, match="type"):
        tk.tk_checkpoint_f32(1, 0, 4, 8, 0, A, None, x, None, D)
    with pytest.raises(ValueError, match="type"):
        tk.tk_head_norm_rotate_bf16(4, 1, 0, 8, 8, 1e-5, 0, x, None, None, None, None, None, None, 0, None, None, x, None, None,
                                    None)
    with pytest.raises(ValueError, match="HIP device"):
        wide = torch.zeros(4, 3, 16)[:, :, :8]  # heads that are apart
        tk.tk_head_norm_rotate_f32(4, 3, 0, 8, 8, 1e-5, 0, wide, None, None, None, None, None, None, 0, None, None, A, None,
                                   None, None)
    monkeypatch.setattr(tk, "_device", lambda: 0)
    s = OtherStream()
    for t in TYPES:
        f = lambda n: getattr(tk, f"tk_{n}_{t}")  # noqa: E731
        for call in (lambda: f("embedding")(1, 0, 4, 8, 0.0, 1.0, 0, 10, A, B, None, D, None, s),
                     lambda: f("embedding_backward")(1, 0, 4, 8, 0.0, 1.0, 0, 10, A, B, None, D, None, (WS, BIG), s),
                     lambda: f("embedding_backward")(1, 0, 4, 8, 0.0, 1.0, 0, 10, A, B, None, D, None, None, s),
                     lambda: f("head_norm_rotate")(4, 1, 1, 8, 8, 0.0, 0, A, None, B, None, None, None, None, 9, D, E, F, None,
                                                   G, None, s),
                     lambda: f("head_norm_rotate_backward")(4, 1, 1, 8, 8, 0.0, 0, A, None, B, None, H, None, I, None, None,
                                                            None, None, 9, D, E, F, None, G, None, None, None, None, s),
                     lambda: f("checkpoint")(1, 0, 4, 8, 0, A, None, B, None, D, s),
                     lambda: f("checkpoint_restore")(4, 8, 0, A, None, B, D, None, s),
                     lambda: f("layer_norm_backward_checkpoint")(4, 8, 0, A, None, B, None, H, None, D, E, F, None, None, None,
                                                                 None, s),
                     lambda: f("dropout_add_layer_norm_backward_checkpoint")(1, 0, 4, 8, 0.1, 0, A, None, None, None, B, None,
                                                                             H, None, D, E, F, None, G, None, None, None, None,
                                                                             None, s)):
            with pytest.raises(ValueError, match="stream"):
                call()


# ---- the reference's formulas ----

def test_reference_embedding_gradient_is_that_of_differences():
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    ids = torch.tensor([3, 0, 3, -1, 5, 2, 3, 1 << 40])
    keep = ref.keep_mask(3, 11, 8, 7, 0.3)
    at, dy = {"table": rnd(5, 7)}, rnd(8, 7)
    loss = lambda table: float((tok.embedding(ids, table, keep, 0.3, 1.5)[0] * dy).sum())  # noqa: E731
    grad = tok.embedding_backward(ids, dy, keep, 0.3, 1.5, 5)[0]
    slope, d = directional(loss, at, "table", 9)
    assert abs(slope - float((grad * d).sum())) <= 1e-7 * (1 + abs(slope))
    assert not bool(grad[1].any()) and not bool(grad[4].any())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,half", [(8, 4), (10, 3), (5, 0), (7, 3)])
def test_reference_head_gradients_are_those_of_differences(interleaved, dim, half):
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    angle = rnd(6, half)
    cos, sin = angle.cos(), angle.sin()
    at, dy = {"x": rnd(6, 3, dim), "gamma": rnd(dim)}, rnd(6, 3, dim)
    loss = lambda x, gamma: float((tok.head_norm_rotate(x, gamma, cos, sin, interleaved, 1e-3)[0] * dy).sum())  # noqa: E731
    out = tok.head_norm_rotate_backward(dy, at["x"], at["gamma"], cos, sin, interleaved, 1e-3)
    for name in ("x", "gamma"):
        slope, d = directional(loss, at, name, 9)
        assert abs(slope - float((out["d" + name][0] * d).sum())) <= 1e-7 * (1 + abs(slope)), name


def test_reference_turns_keep_lengths():
    x, a = torch.randn(4, 2, 12, dtype=torch.float64), torch.randn(4, 5, dtype=torch.float64)
    for interleaved in (False, True):
        y = tok.turned(x, a.cos(), a.sin(), interleaved)[0]
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1), rtol=1e-12)
        assert torch.equal(y[..., 10:], x[..., 10:])
        assert torch.allclose(tok.turned(y, a.cos(), -a.sin(), interleaved)[0], x, rtol=0, atol=1e-12)
        pairs = torch.complex(y[..., 0], y[..., 1 if interleaved else 5])
        first = torch.complex(x[..., 0], x[..., 1 if interleaved else 5])
        assert torch.allclose(pairs, first * torch.polar(torch.ones_like(a[:, :1]), a[:, :1]), rtol=0, atol=1e-12)


def test_reference_codes():
    """Within a code of the quotient and right on average; the largest of a block is +-127; special blocks."""
    x = np.random.default_rng(3).standard_normal((40, 300)).astype(np.float32)
    codes, scales = tok.checkpoint(x, 5, 7)
    at = np.arange(300) // 128
    t = x.astype(np.float64) / scales[:, at]
    assert np.abs(codes - t).max() < 1.0 + 1e-4
    # 12000 errors, each within a code and 0 on average: their mean within five of its deviations
    assert abs((codes - t).mean()) < 5 * 0.5 / np.sqrt(t.size)
    for b in range(3):
        assert (np.abs(codes[:, at == b].astype(int)).max(1) == 127).all()
    x[0, :] = 0
    x[1, :] = 1e-31  # below 2^-100
    x[2, 130] = np.inf
    x[3, 299] = np.nan
    codes, scales = tok.checkpoint(x, 5, 7)
    assert not codes[0].any() and not scales[0].any() and not codes[1].any() and not scales[1].any()
    assert np.isnan(scales[2, 1]) and not codes[2, 128:256].any() and np.isfinite(scales[2, [0, 2]]).all()
    assert np.isnan(scales[3, 2]) and np.isfinite(scales[3, :2]).all()
