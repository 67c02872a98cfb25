"""How exact the row operators are where the general bounds of row_reference.py are wide: rows
whose mean is many of their standard deviations."""
import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref
from gpu_harness import log
from row_reference import U
from test_row_operators import IDS, KINDS, flags, fn, types

pytestmark = pytest.mark.gpu

WIDTHS = [5, 40, 100, 200, 400, 1000, 2000, 5001, 9000, 20000, 30000, 40000]  # one of every forward kernel


def norm_of(v, gamma, beta, eps):
    """Layer norm of f32 values v: (value, bound) of y, mean and rstd, where the mean that the first
    sum gives is off by D <= (K + 1) U mean|v|, and its distances d make up for that where it is more
    than four standard deviations (surely where mean^2 > 17 variance: D^2 is far below mean^2).

    d is rounded once (U |d|); the sum of K additions that gives delta, what the first mean is off
    by, is off by (K + 2) U mean|d| a row; |d| is at most |v - mean| + D.  The variance is
    (sum d^2 - (sum d) delta) / n: its first term, at most variance + D^2, is off by
    (K + 6) U of itself (squares of rounded distances, additions, the division), its second, at most
    D^2, by (2 K + 8) U.  Without delta the mean is off by D and the variance by D^2 more.
    h = (d - delta) rstd takes two roundings more, its parts' sizes together at most |h| + D rstd;
    y one or two."""
    cols = v.shape[1]
    k = ref.additions(cols)
    v = v.double()
    mean = v.mean(1, keepdim=True)
    far = (k + 1) * U * v.abs().mean(1, keepdim=True)
    d = v - mean
    var = d.square().mean(1, keepdim=True)
    big = d.abs() + far
    e_delta = (k + 2) * U * big.mean(1, keepdim=True)
    e_var = (k + 6) * U * (var + far.square()) + (2 * k + 8) * U * far.square()
    kept = mean.square() <= 17 * var
    e_delta = torch.where(kept, torch.maximum(e_delta, far), e_delta)
    e_var = torch.where(kept, e_var + far.square(), e_var)
    rstd = (var + eps) ** -0.5
    rel = 0.5 * e_var / (var + eps) + 4 * U
    h = d * rstd
    e_h = rstd * (U * big + e_delta) + rel * h.abs() + 3 * U * (h.abs() + far * rstd)
    y = h * gamma + beta
    return {"y": (y, gamma.abs() * e_h + 2 * U * (h * gamma).abs() + U * y.abs()),
            "mean": (mean[:, 0], (e_delta + U * mean.abs())[:, 0]), "rstd": (rstd[:, 0], (rstd * rel)[:, 0])}


def far_rows(cols, R, seed):
    """Rows far from zero against their spread, constant rows among them, between ordinary rows and
    one with an outlier."""
    g = torch.Generator().manual_seed(seed)
    m = torch.tensor([1e4, 0.5, -1e4, 3000.0, 0.0, 1e3, 10304.0, 0.0, 10000.1, 0.1, -50.3], dtype=torch.float64)[:, None]
    s = torch.tensor([0.1, 1.0, 1e-2, 1e-3, 2.0, 8.0, 0.0, 1.0, 0.0, 0.0, 0.0], dtype=torch.float64)[:, None]
    x = (m + s * torch.randn(len(m), cols, generator=g, dtype=torch.float64)).to(R)
    x[7, 0] = 2000.0  # one element far from all others
    return x


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_far_from_zero(kind, cols):
    T, R, W = types(kind)
    log(f"far rows {kind} {cols}")
    g = torch.Generator().manual_seed(cols)
    gamma, beta = torch.randn(cols, generator=g).to(W), torch.randn(cols, generator=g).to(W)
    x = far_rows(cols, R, cols)
    rows = x.shape[0]
    y, mean, rstd = torch.empty(rows, cols, dtype=T, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(
        rows, device="cuda")
    fn("layer_norm", kind)(rows, cols, 1e-5, flags(kind), x.cuda(), None, gamma.cuda(), beta.cuda(), y, None, mean, rstd)
    want = norm_of(x.float(), gamma.double(), beta.double(), 1e-5)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        ref.check(got, want[name], f"layer norm {kind} {cols} {name}")

    # the same rows as the sum of two: x is a half of it in T, the residual the rest, and their sum
    # an f32 operation
    a = (x.double() / 2).to(T)
    r = (x.double() - a.double()).to(R)
    v = a.float() + r.float()
    s = torch.empty(rows, cols, dtype=R, device="cuda")
    fn("dropout_add_layer_norm", kind)(3, 0, rows, cols, 0.0, 1e-5, flags(kind), a.cuda(), None, None, r.cuda(), None,
                                       gamma.cuda(), beta.cuda(), s, None, y, None, mean, rstd)
    assert torch.equal(s.cpu(), v.to(R))
    want = norm_of(v, gamma.double(), beta.double(), 1e-5)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        ref.check(got, want[name], f"dropout-add and layer norm {kind} {cols} {name}")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_do_not_see_their_neighbours(kind, cols):
    """Rows far from zero among ordinary ones, many times over so that work-groups go round, give
    the bits that they give alone."""
    T, R, W = types(kind)
    log(f"neighbours {kind} {cols}")
    x = far_rows(cols, R, cols).cuda()
    n, times = x.shape[0], max(3, min(1500, 4_000_000 // (11 * cols)))

    def run(v):
        out = (torch.empty(v.shape, dtype=T, device="cuda"), torch.empty(len(v), device="cuda"), torch.empty(len(v), device="cuda"))
        fn("layer_norm", kind)(len(v), cols, 1e-5, flags(kind), v, None, None, None, out[0], None, out[1], out[2])
        return out

    alone = [run(x[k:k + 1]) for k in range(n)]
    order = torch.randperm(n * times, generator=torch.Generator().manual_seed(cols)).cuda() % n
    many = run(x[order])
    for k in range(3):
        want = torch.cat([a[k] for a in alone])[order]
        assert torch.equal(many[k], want), ("y", "mean", "rstd")[k]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [1000, 1536, 7000, 12000, 20000, 28000, 40000])
def test_a_constant_row_gives_beta(kind, cols):
    """A row of one value whose sums a float holds at every step (6 bits by cols up to 2^16 of them)
    has that value as its mean, no distance from it, and beta as its norm, bit for bit."""
    T, R, W = types(kind)
    beta = torch.randn(cols, generator=torch.Generator().manual_seed(cols)).to(W).cuda()
    for c in (10304.0, -3.0, 0.171875):
        x = torch.full((2, cols), c, dtype=R, device="cuda")
        assert float(x[0, 0]) == c
        y, mean, rstd = torch.empty(2, cols, dtype=T, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
        fn("layer_norm", kind)(2, cols, 1e-5, flags(kind), x, None, None, beta, y, None, mean, rstd)
        assert bool((mean == c).all()), (c, mean)
        assert torch.equal(y, beta.to(T).expand(2, cols)), c


@pytest.mark.parametrize("kind", KINDS[:1], ids=IDS[:1])
@pytest.mark.parametrize("cols", [100, 1000, 9000, 40000])
def test_rows_at_the_ends_of_f32(kind, cols):
    """The mean of a row with an infinity is that infinity; of a constant row whose squared
    distances might leave the range, the value; distances whose squares do leave it give beta."""
    x = torch.full((5, cols), 2.0 ** 80, device="cuda")
    x[1] = 1.1e30
    x[2] = 1.0
    x[2, 3] = float("inf")
    x[3] = 1.0
    x[3, 7] = -float("inf")
    x[4] = torch.where(torch.arange(cols, device="cuda") % 2 > 0, 2.0 ** 70, -(2.0 ** 70))
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    fn("layer_norm", kind)(5, cols, 1e-5, 0, x, None, None, None, y, None, mean, rstd)
    assert float(mean[2]) == float("inf") and float(mean[3]) == -float("inf")
    assert bool(torch.isnan(y[2:4]).all())
    assert float(mean[0]) == 2.0 ** 80 and not bool(y[0].any())
    assert abs(float(mean[1]) / 1.1e30 - 1) <= ref.additions(cols) * U and bool(torch.isfinite(y[1]).all())
    assert float(rstd[4]) == 0 and not bool(y[4].any())


def is_quotient(got, v, keep, p, what):
    """`got` (f32) is v over 1 - p where kept, rounded once: off by half a step, and by 2^-20 of that
    for a quotient that lies within 2^-46 of the middle of two floats; else +0."""
    want = torch.where(keep > 0, v.double() / ref.quotient(p), 0.0)
    got = got.detach().cpu()
    assert not bool(((got.double() - want).abs() > (1 + 2.0 ** -20) * U * want.abs() + 2.0 ** -149).any()), what
    assert not bool(got[keep == 0].view(torch.int32).any()), what


@pytest.mark.parametrize("kind", [k for k in KINDS if k[1] or k[2]], ids=[i for i, k in zip(IDS, KINDS) if k[1] or k[2]])
@pytest.mark.parametrize("cols", [5, 100, 1000, 5001, 20000, 40000])
@pytest.mark.parametrize("p", [0.1, 0.3, 0.5, 0.9, 1.0 - 2.0 ** -24, 2.0 ** -25])
def test_float_outputs_are_quotients(kind, cols, p):
    """16-bit operators with a float residual stream or float parameters: kept values in float
    outputs are the quotient by 1 - p, not a product with a rounded reciprocal."""
    T, R, W = types(kind)
    log(f"quotients {kind} {cols} {p}")
    rows = 3
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols, generator=g).to(T)
    keep = ref.keep_mask(6, 2, rows, cols, p)
    e = lambda t: torch.empty(rows, cols, dtype=t, device="cuda")  # noqa: E731
    if kind[1]:
        y, s = e(R), e(R)
        fn("dropout_add", kind)(6, 2, rows, cols, p, flags(kind), x.cuda(), None, None, None, None, y, None)
        is_quotient(y, x, keep, p, "dropout_add")
        fn("dropout_add_layer_norm", kind)(6, 2, rows, cols, p, 1e-5, flags(kind), x.cuda(), None, None, None, None, None, None,
                                           s, None, e(T), None)
        is_quotient(s, x, keep, p, "dropout_add_layer_norm sum")
    if kind[2]:  # over one row the bias's gradient is the kept gradient itself
        dy = torch.randn(1, cols, generator=g).to(R)
        keep = ref.keep_mask(6, 2, 1, cols, p)
        db, dx = torch.empty(cols, device="cuda"), torch.empty(1, cols, dtype=T, device="cuda")
        fn("dropout_add_backward", kind)(6, 2, 1, cols, p, flags(kind), dy.cuda(), None, dx, None, db)
        is_quotient(db[None], dy, keep, p, "dropout_add_backward dbias")
        if kind[1]:  # the sum's gradient comes out in float too
            dt = torch.randn(1, cols, generator=g).to(T).cuda()
            v, dr = torch.randn(1, cols, generator=g).to(R).cuda(), torch.empty(1, cols, device="cuda")
            st = torch.ones(1, device="cuda")
            fn("dropout_add_layer_norm_backward", kind)(6, 2, 1, cols, p, flags(kind), dt, None, dy.cuda(), None, v, None, None,
                                                        st, st, dx, None, dr, None, None, None, db)
            is_quotient(db[None], dr.cpu(), keep, p, "dropout_add_layer_norm_backward dbias")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("p", [0.1, 0.3, 0.5, 0.75])
def test_kept_infinities_stay(kind, p):
    """An infinity over 1 - p is that infinity, also where 1 / (1 - p) is a float itself."""
    T, R, _ = types(kind)
    cols = 64
    x = torch.full((2, cols), float("inf"), dtype=T, device="cuda")
    x[1] = -float("inf")
    y = torch.empty(2, cols, dtype=R, device="cuda")
    fn("dropout_add", kind)(6, 0, 2, cols, p, flags(kind), x, None, None, None, None, y, None)
    keep = ref.keep_mask(6, 0, 2, cols, p).cuda() > 0
    assert torch.equal(y, torch.where(keep, x.to(R), torch.zeros_like(y)))


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("cols", [40, 1000, 8000, 30000])
def test_calls_of_one_mask_agree(kind, cols):
    """The fused operator's sum is dropout-add's y bit for bit, and dx does not depend on whether the
    bias's gradient is wanted, nor on who makes it from the same dresidual."""
    T, R, W = types(kind)
    rows, p = 200, 0.3
    log(f"one mask {kind} {cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    mat = lambda t: torch.empty(rows, cols, dtype=t, device="cuda").normal_(generator=g)  # noqa: E731
    x, r, bias = mat(T), mat(R), torch.randn(cols, generator=g, device="cuda").to(W)
    y, s = torch.empty_like(r), torch.empty_like(r)
    fn("dropout_add", kind)(6, 2, rows, cols, p, flags(kind), x, None, bias, r, None, y, None)
    fn("dropout_add_layer_norm", kind)(6, 2, rows, cols, p, 1e-5, flags(kind), x, None, bias, r, None, None, None, s, None,
                                       torch.empty_like(x), None)
    assert torch.equal(s, y)
    dy, st = mat(T), torch.ones(rows, device="cuda")
    got = []
    for wanted in (True, False):
        db = torch.empty(cols, dtype=W, device="cuda") if wanted else None
        dx, dr, dx2 = torch.empty_like(x), torch.empty_like(r), torch.empty_like(x)
        fn("dropout_add_layer_norm_backward", kind)(6, 2, rows, cols, p, flags(kind), dy, None, r, None, s, None, None, st, st, dx,
                                                    None, dr, None, None, None, db)
        fn("dropout_add_backward", kind)(6, 2, rows, cols, p, flags(kind), r, None, dx2, None, db)
        got.append((dx, dr, dx2))
    assert all(torch.equal(a, b) for a, b in zip(*got))
