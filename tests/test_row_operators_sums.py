"""The row operators' column sums over many rows, within the rounding of the additions that a term
can pass, and the operators at further changes of kernel shape."""
import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref
import test_row_operators as base
from gpu_harness import log
from row_reference import U
from test_row_operators import FILL, IDS, KINDS, flags, fn, types

pytestmark = pytest.mark.gpu

# Work-groups that go round several times, with every number of lanes to a row; several groups of
# each; strips of columns with one line over many rows (chunks of four and of eight elements); and
# reads beyond what goes through the caches (the last four).
SUMS = [(70000, 5), (70000, 40), (300, 100), (40000, 100), (20000, 200), (20000, 257), (9000, 1000), (3000, 5001), (2000, 9000),
        (100, 33001), (100, 66001), (500000, 40), (200000, 130), (15000, 2000), (4000, 12000)]


def depth(rows, cols):
    """At most how many additions a term passes.  A lane takes every n-th row, or one in four of few
    rows: of 256 work-groups of sixteen waves with at most 16 lanes to a row up to 64 columns, 32 up
    to 128, a wave up to 256; 128 rows up to 8192 columns and 16 beyond.  Then 3 steps in a wave, 16
    waves, and of 256 lines 16, 1 and 16."""
    side = 16384 if cols <= 64 else 8192 if cols <= 128 else 4096 if cols <= 256 else 128 if cols <= 8192 else 16
    return rows // side + 4 + 3 + 16 + 33


def near(got, terms, err, what):
    """`got` against the column sums of float64 `terms`, each off by up to `err`; and a limit that a
    mistake in the sums would pass: the oracle with some rows left out, in the beginning, the middle
    and the end, and an oracle of zeros are beyond it.  16 rows, whose sum is about 4; of
    a 16-bit gradient a sixteenth of all rows, about sqrt(n) / 4, since rounding to the type alone
    is off by up to 2^-9 of the sum, about sqrt(n) (16 of 70000 rows are less than that)."""
    rows, cols = terms.shape
    want = terms.sum(0)
    limit = 1.01 * (err.sum(0) + depth(rows, cols) * U * terms.abs().sum(0))
    limit = limit + (want.abs() + limit) * torch.finfo(got.dtype).eps / 2 + ref.TINY[got.dtype]
    far = (got.double() - want).abs() > limit
    assert not bool(far.any()), (what, int(far.sum()), far.nonzero()[0].item())
    assert float((want.abs() > limit).double().mean()) > 0.5, f"{what}: zeros would pass"
    some = 16 if got.dtype is torch.float32 else max(16, rows // 16)
    for at in (0, rows // 2, rows - some):
        assert bool((terms[at:at + some].sum(0).abs() > 2 * limit).any()), f"{what}: {some} rows from {at} could be missing"


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows,cols", SUMS)
def test_column_sums(kind, rows, cols):
    T, R, W = types(kind)
    p = 0.25
    log(f"column sums {kind} {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    mat = lambda t: torch.empty(rows, cols, dtype=t, device="cuda").normal_(generator=g)  # noqa: E731
    out = lambda: torch.full((cols,), FILL, dtype=W, device="cuda")  # noqa: E731
    keep = ref.keep_mask(8, 3, rows, cols, p).cuda()

    dy, dx, db = mat(R), torch.empty(rows, cols, dtype=T, device="cuda"), out()
    fn("dropout_add_backward", kind)(8, 3, rows, cols, p, flags(kind), dy, None, dx, None, db)
    v, e = ref._dropped(dy.double(), torch.zeros_like(dy, dtype=torch.float64), keep, p)
    near(db, v, e, "dropout_add_backward dbias")
    del dy, v, e

    dy, ds, x = mat(T), mat(R), mat(R)
    gamma = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(W)
    mean, rstd = x.double().mean(1).float(), (x.double().var(1, unbiased=False) + 1e-5).rsqrt().float()
    dr, dg, dt = torch.empty_like(x), out(), out()
    fn("layer_norm_backward", kind)(rows, cols, flags(kind), dy, None, x, None, gamma, mean, rstd, dr, None, dg, dt)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None] * dy.double()
    near(dg, h, 3 * U * h.abs(), "layer_norm_backward dgamma")
    near(dt, dy.double(), torch.zeros_like(h), "layer_norm_backward dbeta")

    dg2, dt2, db = out(), out(), out()
    fn("dropout_add_layer_norm_backward", kind)(8, 3, rows, cols, p, flags(kind), dy, None, ds, None, x, None, gamma, mean, rstd,
                                                dx, None, dr, None, dg2, dt2, db)
    near(dg2, h, 3 * U * h.abs(), "dropout_add_layer_norm_backward dgamma")
    near(dt2, dy.double(), torch.zeros_like(h), "dropout_add_layer_norm_backward dbeta")
    del h
    want = ref.dropout_add_layer_norm_backward(dy.double(), ds.double(), x.double(), gamma.double(), mean.double(),
                                               rstd.double(), keep, p)
    near(db, *want["dx"], "dropout_add_layer_norm_backward dbias")


# rows, cols: full rows of 16, 32 lanes, of one and twelve waves, of 24 elements a lane, and one column
# more; strips of wide rows with several lines, and with one line over several sets of rows
MORE = [(70, 65), (9, 128), (600, 128), (9, 256), (70, 257), (70, 1024), (5, 6144), (5, 6145), (4, 16384), (4, 24576), (200, 9000),
        (40, 33001), (40, 66001)]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("test", [base.test_dropout_add, base.test_layer_norm, base.test_dropout_add_layer_norm],
                         ids=["dropout_add", "layer_norm", "dropout_add_layer_norm"])
def test_further_sizes(kind, test, monkeypatch):
    monkeypatch.setattr(base, "SIZES", MORE)
    test(kind)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(2, 8192), (5, 2), (40, 512), (64, 128), (200, 8000), (600, 5001), (33, 9000), (50, 66001)])
def test_gradients_without_column_sums(kind, rows, cols):
    """Calls that want none of them are cut otherwise and give the rows' gradients bit for bit."""
    T, R, W = types(kind)
    g = torch.Generator(device="cuda").manual_seed(cols)
    mat = lambda t: torch.empty(rows, cols, dtype=t, device="cuda").normal_(generator=g)  # noqa: E731
    dy, ds, x, gamma = mat(T), mat(R), mat(R), torch.randn(cols, generator=g, device="cuda").to(W)
    mean, rstd = x.float().mean(1), (x.float().var(1, unbiased=False) + 1e-5).rsqrt()
    ws = torch.empty(max(4, tk.tk_backward_workspace_bytes(rows, cols)), dtype=torch.uint8, device="cuda")
    got = []
    for wanted in (True, False):
        sums = [torch.empty(cols, dtype=W, device="cuda") if wanted else None for _ in range(3)]
        d = [torch.full((rows, cols), FILL, dtype=t, device="cuda") for t in (R, T, R)]
        fn("layer_norm_backward", kind)(rows, cols, flags(kind), dy, None, x, None, gamma, mean, rstd, d[0], None, sums[0], sums[1],
                                        ws)
        fn("dropout_add_layer_norm_backward", kind)(8, 3, rows, cols, 0.25, flags(kind), dy, None, ds, None, x, None, gamma, mean,
                                                    rstd, d[1], None, d[2], None, *sums, ws)
        got.append(d)
    assert all(torch.equal(a, b) for a, b in zip(*got))
