"""The embedding, the head norms and the checkpoints on the GPU against their 64-bit reference: every
pair of types, the sizes where a shape of kernel begins or ends, rows cut from wider buffers at
odd addresses, tokens and positions outside their tables, in place, cut calls, captured calls, two
streams, and a training step's run of them with the row operators."""
import numpy as np
import pytest
import torch

import bulk_fills_amd as tk
import row_reference as ref
import token_reference as tok
from gpu_harness import log
from test_row_operators import FILL, IDS, KINDS, Maker, flags, fn, types

pytestmark = pytest.mark.gpu

# rows, cols, vocab: single ones, both sides of a tile of 64 rows, of a strip's and a lane's columns, of the
# sort's ranges of 8, 32, 128 and 512 tokens, and many tiles
LOOKUPS = [(1, 1, 1), (3, 7, 5), (64, 16, 1), (65, 8, 4), (130, 65, 3), (1000, 129, 50), (5000, 40, 17), (2047, 513, 700),
           (300, 2049, 4000), (1500, 264, 16384), (1500, 130, 32768), (700, 33, 32769), (500, 100, 65537), (66000, 5, 900),
           (4099, 1032, 200), (40, 8200, 30), (200, 12, 2048), (200, 12, 2049), (300, 20, 8192), (300, 20, 8193)]
SPREADS = ("even", "skewed", "one", "outside")


def tokens(rows, vocab, spread, i64, seed):
    """ids on the CPU (int64): even, mostly the lowest, all one, or many of them outside."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(rows, generator=g, dtype=torch.float64)
    if spread == "one":
        return torch.full((rows,), seed % vocab)
    ids = ((vocab + 1.0) ** u).long() - 1 if spread == "skewed" else (u * vocab).long()
    ids.clamp_(max=vocab - 1)
    if spread == "outside":
        far = torch.tensor([-1, vocab, -(1 << 31), (1 << 31) - 1] + ([1 << 40, -(1 << 40), (1 << 32) + 1] if i64 else []))
        some = torch.randint(0, len(far), (rows,), generator=g)
        ids = torch.where(torch.rand(rows, generator=g) < 0.6, far[some], ids)
    return ids


def on_device(ids, i64):
    return ids.to("cuda", torch.int64 if i64 else torch.int32)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_embedding(kind):
    T, R, W = types(kind)
    for i, (rows, cols, vocab) in enumerate(LOOKUPS):
        for spread in SPREADS:
            i64, p, scale = i % 2 == 0, (0.0, 0.25)[(i + len(spread)) % 2], (1.0, 11.3)[i % 2]
            pad = (0, 3, 8)[i % 3]
            what = f"embedding {kind} {rows}x{cols} of {vocab} {spread} p {p} pad {pad}"
            log(what)
            fl = flags(kind) | (tk.TK_INDEX_I64 if i64 else 0)
            ids = tokens(rows, vocab, spread, i64, i)
            m, mt = Maker(rows, cols, pad, i), Maker(vocab, cols, pad, i + 50)
            table, tr = mt.mat(W)
            y = m.out(R)
            fn("embedding", kind)(8, 5 + i, rows, cols, p, scale, fl, vocab, on_device(ids, i64), table, None, y, None)
            keep = ref.keep_mask(8, 5 + i, rows, cols, p)
            scale32 = float(np.float32(scale))
            ref.check(y, tok.embedding(ids, tr, keep, p, scale32), what)
            m.untouched(what)
            dy, dr = m.mat(R)
            want = tok.embedding_backward(ids, dr, keep, p, scale32, vocab)
            dt = mt.out(W)
            fn("embedding_backward", kind)(8, 5 + i, rows, cols, p, scale, fl, vocab, on_device(ids, i64), dy, None, dt, None)
            ref.check(dt, want, what + " backward")
            mt.untouched(what)
            # added to what is there; tokens that do not occur keep theirs
            old = dt.clone()
            fn("embedding_backward", kind)(8, 5 + i, rows, cols, p, scale, fl | tk.TK_ACCUMULATE, vocab, on_device(ids, i64),
                                           dy, None, dt, None)
            ref.check(dt, tok.embedding_backward(ids, dr, keep, p, scale32, vocab, old.cpu().double()), what + " accumulate")
            mt.untouched(what)


def test_embedding_without_rows_or_tokens():
    x, t = torch.full((5, 8), FILL, device="cuda"), torch.full((4, 8), FILL, device="cuda")
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    tk.tk_embedding_f32(1, 0, 5, 8, 0.1, 2.0, 0, 0, ids, None, None, x, None)  # no table: zeros
    assert not bool(x.any())
    tk.tk_embedding_backward_f32(1, 0, 0, 8, 0.1, 2.0, tk.TK_ACCUMULATE, 4, ids[:0], x[:0], None, t, None)
    assert bool((t == FILL).all())
    tk.tk_embedding_backward_f32(1, 0, 0, 8, 0.1, 2.0, 0, 4, ids[:0], x[:0], None, t, None)
    assert not bool(t.any())
    t.fill_(FILL)
    x.fill_(float("nan"))  # rows without a token are not read
    tk.tk_embedding_backward_f32(1, 0, 5, 8, 0.1, 2.0, 0, 4, ids - 1, x, None, t, None)
    assert not bool(t.any())
    x[3] = 1.5
    ids.fill_(9)
    ids[3] = 2
    tk.tk_embedding_backward_f32(1, 0, 5, 8, 0.0, 2.0, 0, 4, ids, x, None, t, None)
    assert bool((t[2] == 3.0).all()) and not bool(t[[0, 1, 3]].any())


def test_embedding_of_non_finite_values():
    table = torch.randn(6, 300, device="cuda")
    table[1, 5], table[2, 6], table[3, 7] = float("nan"), float("inf"), -float("inf")
    ids = torch.arange(6, device="cuda")
    y = torch.empty(6, 300, device="cuda")
    tk.tk_embedding_f32(1, 0, 6, 300, 0.5, 2.0, tk.TK_INDEX_I64, 6, ids, table, None, y, None)
    keep = ref.keep_mask(1, 0, 6, 300, 0.5).cuda() > 0
    want = torch.where(keep, table * 2.0 / 0.5, 0.0)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.nan_to_num())
    d = torch.empty(3, 300, device="cuda")
    tk.tk_embedding_backward_f32(1, 0, 6, 300, 0.0, 1.0, tk.TK_INDEX_I64, 3, ids // 2, table, None, d, None)
    want = table[0::2] + table[1::2]  # each token's own rows and no others'
    assert torch.equal(d.isnan(), want.isnan()) and torch.equal(d.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("spread", ["even", "skewed", "one"])
def test_embedding_gradients_have_one_order(spread):
    """Equal bits in every run, also while another stream's calls take the compute units."""
    rows, cols, vocab = 9000, 520, 3001
    ids = on_device(tokens(rows, vocab, spread, True, 3), True)
    dy = torch.randn(rows, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    n = tk.tk_embedding_workspace_bytes(rows, cols, vocab)
    side, outs = torch.cuda.Stream(), []
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    other = torch.empty(vocab, cols, device="cuda")
    torch.cuda.synchronize()
    for k in range(6):
        d = torch.full((vocab, cols), FILL, device="cuda")
        torch.cuda.synchronize()
        if k % 2:
            tk.tk_embedding_backward_f32(1, 7, rows, cols, 0.1, 3.0, tk.TK_INDEX_I64, vocab, ids, dy, None, other, None, ws[1], side)
        tk.tk_embedding_backward_f32(1, 7, rows, cols, 0.1, 3.0, tk.TK_INDEX_I64, vocab, ids, dy, None, d, None, ws[0])
        torch.cuda.synchronize()
        outs.append(d)
        if k % 2:
            assert torch.equal(other, outs[0])
    assert all(torch.equal(outs[0], d) for d in outs[1:])


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[2], KINDS[3]], ids=["f32", "f16-r32-p32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2900, 4096), (5000, 4096), (9000, 4096), (17000, 4096), (140000, 100), (140000, 200)])
def test_embedding_gradients_of_every_tile(kind, rows, cols):
    """Tiles of 8 to 64 rows, and of 8 to 32 rows of fewer lanes, against sums in float64 on the device."""
    T, R, W = types(kind)
    vocab, p = 3000, 0.25
    g = torch.Generator("cuda").manual_seed(rows)
    dy = torch.empty(rows, cols, dtype=R, device="cuda").normal_(generator=g)
    u = torch.empty(rows * cols, device="cuda")
    tk.tk_fill_f32(8, 5, rows * cols, u)
    v = torch.where(u.view(rows, cols) >= p, dy.double() / ref.quotient(p), 0.0)
    for spread in ("even", "skewed", "one"):
        log(f"tiles {kind} {rows}x{cols} {spread}")
        ids = tokens(rows, vocab, spread, True, rows)
        ids[::7] = -1
        there = (ids >= 0).cuda()
        at = ids.cuda()[there]
        want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, at, v[there])
        size = torch.zeros_like(want).index_add_(0, at, v[there].abs())
        many = torch.bincount(at, minlength=vocab)[:, None]
        # each term's quotient (2 u), additions of no more than a token's rows, and the product with the scale
        bound = 3.0 * size * (many + 3) * ref.U + ref.U * 3 * want.abs()
        d = torch.full((vocab, cols), FILL, dtype=W, device="cuda")
        fn("embedding_backward", kind)(8, 5, rows, cols, p, 3.0, flags(kind) | tk.TK_INDEX_I64, vocab, ids.cuda(), dy, None, d,
                                       None)
        want = want * 3.0
        limit = 1.01 * bound + (want.abs() + 1.01 * bound) * torch.finfo(W).eps / 2 + ref.TINY[W]
        assert not bool(((d.double() - want).abs() > limit).any())
        assert not bool(d[many[:, 0] == 0].any())


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1500, 4096), (2900, 4096), (5000, 4096), (9000, 4096), (17000, 4096), (140000, 3),
                                       (140000, 20), (140000, 40), (140000, 100), (140000, 200), (20, 300000)])
def test_embedding_gradients_are_whole(kind, rows, cols):
    """No row or tile left out or taken twice, also where one token has them all: small whole numbers, whose sums
    below 2^24 are exact in floats in any order, so the result is the exact sum rounded to the table's type.
    With p 1/2 an element counts twice or not at all.  Tiles of 8, 16, 32 and 64 rows at each number of lanes
    that has them, more tiles and more columns than a launch of the join takes at once."""
    T, R, W = types(kind)
    vocab, fl = 300, flags(kind) | tk.TK_INDEX_I64
    g = torch.Generator("cuda").manual_seed(rows + cols)
    dy = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").to(R)
    u = torch.empty(rows * cols, device="cuda")
    tk.tk_fill_f32(8, 5, rows * cols, u)
    for i, spread in enumerate(("even", "skewed", "one")):
        p = (0.0, 0.5, 0.5)[i] if rows % 2000 else (0.5, 0.0, 0.0)[i]
        log(f"whole {kind} {rows}x{cols} {spread} p {p}")
        ids = tokens(rows, vocab, spread, True, rows)
        ids[::11] = -1
        there = (ids >= 0).cuda()
        at = ids.cuda()[there]
        v = dy.double() if p == 0 else torch.where(u.view(rows, cols) >= p, dy.double() * 2, 0.0)
        want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, at, v[there]) * 2
        assert 2 * 6 * rows < 1 << 24
        d = torch.full((vocab, cols), FILL, dtype=W, device="cuda")
        run = lambda f: fn("embedding_backward", kind)(8, 5, rows, cols, p, 2.0, f, vocab, ids.cuda(), dy, None, d, None)  # noqa: E731
        run(fl)
        assert torch.equal(d, want.to(W)), (kind, rows, cols, spread)
        d.copy_(torch.randint(-100, 101, (vocab, cols), generator=g, device="cuda"))
        want += d.double()
        run(fl | tk.TK_ACCUMULATE)
        assert torch.equal(d, want.to(W)), (kind, rows, cols, spread, "accumulate")


@pytest.mark.parametrize("cols,gap", [(1, 0), (3, 0), (37, 0), (100, 0), (1001, 0), (4100, 0), (20000, 0), (37, 2), (1001, 7)])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_embedding_gradient_clears_absent_tokens(kind, cols, gap):
    """Runs of absent tokens of every length, from a base off the 16-byte lines; nothing beside the table changes."""
    T, R, W = types(kind)
    ld, off = cols + gap, 3
    for vocab, ids in ((1, []), (1, [0]), (64, []), (65, [64]), (131, [0, 63, 64, 130]), (200, [1, 7, 66, 128, 199]), (131, [-1, 131])):
        log(f"absent {kind} {vocab} of {cols}+{gap} {ids}")
        buf = torch.full((off + vocab * ld + 5,), FILL, dtype=W, device="cuda")
        d = buf[off : off + vocab * ld].view(vocab, ld)[:, :cols]
        at = torch.tensor(ids, dtype=torch.int64, device="cuda")
        dy = torch.ones(len(ids), cols, dtype=R, device="cuda")
        want = buf.clone()
        rows = want[off : off + vocab * ld].view(vocab, ld)[:, :cols]
        rows.zero_()
        rows[[i for i in ids if 0 <= i < vocab]] = 1
        fn("embedding_backward", kind)(1, 0, len(ids), cols, 0.0, 1.0, flags(kind) | tk.TK_INDEX_I64, vocab, at, dy, None, d, ld,
                                       None)
        assert torch.equal(buf, want)


def test_embedding_sums_of_one_token_are_float_sums():
    """Whole numbers below 2^24 add up exactly in any order, and only in floats: no 16-bit partial sums."""
    rows, cols = 40000, 24
    dy = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    d = torch.empty(9, cols, device="cuda")
    tk.tk_embedding_backward_bf16(1, 0, rows, cols, 0.0, 1.0, tk.TK_PARAMS_F32, 9, ids, dy, None, d, None)
    assert bool((d[5] == rows).all()) and not bool(d[[0, 1, 2, 3, 4, 6, 7, 8]].any())


def test_embedding_beyond_32_bits():
    """A table and its gradient whose last rows begin past 2^32 elements."""
    vocab, cols, ld = (1 << 19) + 3, 200, 8200
    log("embedding beyond 32 bits")
    buf = torch.zeros((vocab - 1) * ld + cols, dtype=torch.bfloat16, device="cuda")
    table = buf.as_strided((vocab, cols), (ld, 1))
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1, (1 << 19) - 1], dtype=torch.int64)
    g = torch.Generator().manual_seed(4)
    for i in ids.unique().tolist():
        table[i] = torch.randn(cols, generator=g).bfloat16().cuda()
    y = torch.empty(5, cols, dtype=torch.bfloat16, device="cuda")
    tk.tk_embedding_bf16(1, 0, 5, cols, 0.0, 1.0, tk.TK_INDEX_I64, vocab, ids.cuda(), table, None, y, None)
    assert torch.equal(y, table[ids.cuda()])
    dy = torch.randn(5, cols, generator=g).bfloat16().cuda()
    want = tok.embedding_backward(torch.tensor([3, 0, 2, 3, 1]), dy.cpu().double(), ref.keep_mask(1, 0, 5, cols, 0.0), 0.0, 1.0, 4)
    at = torch.tensor([0, (1 << 19) - 1, vocab - 2, vocab - 1], device="cuda")
    for fl in (0, tk.TK_ACCUMULATE):
        buf.fill_(0 if fl else FILL)
        tk.tk_embedding_backward_bf16(1, 0, 5, cols, 0.0, 1.0, tk.TK_INDEX_I64 | fl, vocab, ids.cuda(), dy, None, table, None)
        ref.check(table[at], want, "gradient beyond 32 bits")
        others = torch.ones(vocab, dtype=torch.bool, device="cuda")
        others[at] = False
        assert not bool((table.abs().amax(1) * others).any())
        assert bool((buf.as_strided((vocab - 1, ld - cols), (ld, 1), cols) == (0 if fl else FILL)).all())


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_embedding_gradients_are_added_as_floats(kind):
    """scale * sum is a float, and so is what it makes with the old value before the table's type: bit for
    bit, of tokens within a tile and across tiles.  The sums themselves are whole numbers, so exact."""
    T, R, W = types(kind)
    rows, cols, vocab, scale = 700, 130, 40, 1.1
    g = torch.Generator("cuda").manual_seed(2)
    ids = tokens(rows, vocab, "skewed", False, 2)
    dy = torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").to(R)
    sums = torch.zeros(vocab, cols, device="cuda").index_add_(0, ids.cuda(), dy.float())
    old = torch.randn(vocab, cols, generator=g, device="cuda").to(W)
    d = old.clone()
    fn("embedding_backward", kind)(1, 0, rows, cols, 0.0, scale, flags(kind) | tk.TK_ACCUMULATE, vocab, on_device(ids, False), dy,
                                   None, d, None)
    product = sums * torch.full((), scale, device="cuda")
    here = torch.bincount(ids, minlength=vocab).cuda()[:, None] > 0
    assert torch.equal(d, torch.where(here, (product + old.float()).to(W), old))


@pytest.mark.parametrize("vocab", [(1 << 25) + 700, (1 << 28) + 900], ids=["2^25", "2^28"])
def test_embedding_gradient_of_more_tokens_than_a_grid(vocab):
    """The sort's work-groups take further ranges of tokens, and those that clear further rows."""
    log(f"gradient of {vocab} tokens")
    edges = [k for r in range(0, vocab, 1 << 25) for k in (r, r + 1, r + 511, r + 512, r + 699)] + [(1 << 28) - 1, 1 << 28, vocab - 1]
    edges = torch.tensor([k for k in edges if k < vocab])
    g = torch.Generator().manual_seed(3)
    ids = edges[torch.randint(0, len(edges), (3000,), generator=g)]
    ids[:len(edges)] = edges  # each of them, and many rows of some
    ids[700:1400] = vocab - 1
    ids[5::50] = -1
    ids[6::50] = vocab
    dy = torch.randint(1, 4, (3000, 1), generator=g).bfloat16().cuda()
    there = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab, dtype=torch.float32, device="cuda").index_add_(0, ids[there].cuda(), dy[there.cuda(), 0].float())
    buf = torch.full((vocab + 8,), FILL, dtype=torch.bfloat16, device="cuda")
    d = buf[3:3 + vocab].view(vocab, 1)
    tk.tk_embedding_backward_bf16(1, 0, 3000, 1, 0.0, 1.0, tk.TK_INDEX_I64, vocab, ids.cuda(), dy, None, d, None)
    assert torch.equal(d[:, 0], want.bfloat16()) and bool((buf[:3] == FILL).all()) and bool((buf[-5:] == FILL).all())
    d.fill_(1.0)
    tk.tk_embedding_backward_bf16(1, 0, 3000, 1, 0.0, 1.0, tk.TK_INDEX_I64 | tk.TK_ACCUMULATE, vocab, ids.cuda(), dy, None, d, None)
    assert torch.equal(d[:, 0], (want + 1.0).bfloat16())


def test_embedding_of_more_rows_than_a_launch():
    """2^30 chunks are a launch's: rows of one column beyond it, also with the counters' range nearly used up."""
    rows, n, vocab = (1 << 30) + 1000, 3000, 97
    log("embedding of more rows than a launch")
    table = torch.arange(1, vocab + 1, device="cuda").bfloat16().view(vocab, 1)
    ids = torch.full((rows,), 41, dtype=torch.int32, device="cuda")
    ids[-n:] = torch.randint(-5, vocab + 5, (n,), device="cuda", dtype=torch.int32)
    y = torch.full((rows, 1), FILL, dtype=torch.bfloat16, device="cuda")
    tk.tk_embedding_bf16(4, 9, rows, 1, 0.0, 2.0, 0, vocab, ids, table, None, y, None)
    tail = ids[-n:].long()
    there = (tail >= 0) & (tail < vocab)
    assert torch.equal(y[-n:, 0], torch.where(there, 2 * table[tail.clamp(0, vocab - 1), 0], 0.0))
    assert bool((y[:-n] == 84.0).all())
    tk.tk_embedding_bf16(4, 9, rows, 1, 0.5, 2.0, 0, vocab, ids, table, None, y, None)
    for lo in (0, (1 << 30) - 1500):  # both sides of the cut
        hi = min(lo + 2500, rows)
        part = torch.empty(hi - lo, 1, dtype=torch.bfloat16, device="cuda")
        tk.tk_embedding_bf16(4, 9 + lo, hi - lo, 1, 0.5, 2.0, 0, vocab, ids[lo:hi], table, None, part, None)
        assert torch.equal(y[lo:hi], part)


# ---- heads ----
# dim, rotary: one element, no pairs, all and parts of a head, odd widths, every number of lanes
DIMS = [(1, 0), (2, 2), (8, 8), (16, 16), (17, 6), (32, 32), (33, 32), (64, 64), (65, 16), (80, 40), (96, 96), (100, 10),
        (128, 128), (128, 64), (130, 130), (192, 64), (256, 256), (300, 100), (500, 2), (512, 512), (511, 510), (512, 2)]
HEADS = [(1, 0), (0, 3), (5, 2), (32, 8), (7, 7), (1, 1)]


class HeadCase:
    def __init__(self, kind, rows, hq, hk, dim, rotary, interleaved, i, given=True, gamma=True):
        T, _, W = types(kind)
        self.kind, self.rows, self.hq, self.hk, self.dim, self.rotary, self.T, self.W = kind, rows, hq, hk, dim, rotary, T, W
        self.interleaved, self.length = interleaved, 50
        g = self.g = torch.Generator().manual_seed(i)
        self.i64 = i % 2 == 0
        self.flags = (flags(kind) & tk.TK_PARAMS_F32) | (tk.TK_INDEX_I64 if self.i64 else 0)
        self.flags |= tk.TK_INTERLEAVED if interleaved else 0
        angle = torch.rand(self.length, rotary // 2, generator=g) * 700
        self.tables = angle.cos(), angle.sin()
        if given:  # a fifth of them outside
            pos = torch.randint(0, self.length, (rows,), generator=g)
            far = torch.tensor([-1, self.length, (1 << 31) - 1] + ([1 << 40, -(1 << 33)] if self.i64 else []))
            pos = torch.where(torch.rand(rows, generator=g) < 0.2, far[torch.randint(0, len(far), (rows,), generator=g)], pos)
        else:
            pos = torch.arange(rows)
        self.pos = pos
        there = ((pos >= 0) & (pos < self.length))[:, None]
        at = pos.clamp(0, self.length - 1)
        self.cos = torch.where(there, self.tables[0][at].double(), 1.0)
        self.sin = torch.where(there, self.tables[1][at].double(), 0.0)
        self.positions = pos.to("cuda", torch.int64 if self.i64 else torch.int32) if given else None
        self.gq, self.gk = ((1 + 0.3 * torch.randn(dim, generator=g)).to(W) if gamma else None for _ in range(2))
        self.cu = [t.cuda() if t.numel() else None for t in self.tables] + [None if t is None else t.cuda() for t in (self.gq, self.gk)]

    def makers(self, pad, i):
        return Maker(self.rows, self.hq * self.dim, pad, i), Maker(self.rows, self.hk * self.dim, pad, i + 1)

    def shape(self):
        return self.rows, self.hq, self.hk, self.dim, self.rotary, 1e-5, self.flags

    def tail(self):
        return self.cu[2], self.cu[3], self.positions, self.length, self.cu[0], self.cu[1]

    def forward(self, q, k, yq, yk, stream=None):
        fn("head_norm_rotate", self.kind)(*self.shape(), q, None, k, None, *self.tail(), yq, None, yk, None, stream)

    def backward(self, dyq, dyk, q, k, dq, dk, dgq, dgk, ws=None, stream=None):
        fn("head_norm_rotate_backward", self.kind)(*self.shape(), dyq, None, dyk, None, q, None, k, None, *self.tail(), dq, None,
                                                   dk, None, dgq, dgk, ws, stream)

    def want(self, x, gamma):
        v, e = tok.head_norm_rotate(x.view(self.rows, -1, self.dim), None if gamma is None else gamma.double(), self.cos,
                                    self.sin, self.interleaved, 1e-5)
        return v.reshape(self.rows, -1), e.reshape(self.rows, -1)

    def want_back(self, dy, x, gamma):
        out = tok.head_norm_rotate_backward(dy.view(self.rows, -1, self.dim), x.view(self.rows, -1, self.dim),
                                            None if gamma is None else gamma.double(), self.cos, self.sin, self.interleaved, 1e-5)
        return tuple(t.reshape(self.rows, -1) for t in out["dx"]), out["dgamma"]


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1], KINDS[3], KINDS[5]], ids=[IDS[0], IDS[1], IDS[3], IDS[5]])
def test_heads(kind, interleaved):
    for i, (dim, rotary) in enumerate(DIMS):
        for j, (hq, hk) in enumerate(HEADS):
            rows = (1, 3, 70, 130)[(i + j) % 4]
            what = f"heads {kind} {rows}x({hq}+{hk})x{dim} rotary {rotary} {'neighbours' if interleaved else 'halves'}"
            log(what)
            c = HeadCase(kind, rows, hq, hk, dim, rotary, interleaved, i + j, given=j % 3 != 1, gamma=j % 4 != 3)
            mq, mk = c.makers((0, 3, 8)[(i + j) % 3], i)
            q, qr = mq.mat(c.T, 1.5)
            k, kr = mk.mat(c.T, 0.2)
            yq, yk = mq.out(c.T), mk.out(c.T)
            c.forward(q if hq else None, k if hk else None, yq if hq else None, yk if hk else None)
            dyq, dqr = mq.mat(c.T)
            dyk, dkr = mk.mat(c.T)
            dq, dk, dgq, dgk = mq.out(c.T), mk.out(c.T), mq.flat(dim, c.W), mk.flat(dim, c.W)
            c.backward(dyq if hq else None, dyk if hk else None, q if hq else None, k if hk else None, dq if hq else None,
                       dk if hk else None, dgq, dgk)
            for n, h, x, dy, y, d, dg, gamma in (("q", hq, qr, dqr, yq, dq, dgq, c.gq), ("k", hk, kr, dkr, yk, dk, dgk, c.gk)):
                if h == 0:
                    assert not bool(dg.any()), what  # no heads: no gradient
                    continue
                ref.check(y, c.want(x, gamma), f"{what} y{n}")
                dx, dgamma = c.want_back(dy, x, gamma)
                ref.check(d, dx, f"{what} d{n}")
                ref.check(dg, dgamma, f"{what} dgamma_{n}")
            mq.untouched(what)
            mk.untouched(what)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[3]], ids=["f32", "bf16"])
def test_heads_of_many_rows(kind):
    """More rows than the backward's waves take at once; dgamma against float64."""
    c = HeadCase(kind, 6001, 6, 2, 72, 72, False, 5)
    mq, mk = c.makers(0, 3)
    (q, qr), (k, kr), (dyq, dqr), (dyk, dkr) = mq.mat(c.T), mk.mat(c.T), mq.mat(c.T), mk.mat(c.T)
    dq, dk, dgq, dgk = mq.out(c.T), mk.out(c.T), mq.flat(72, c.W), mk.flat(72, c.W)
    c.backward(dyq, dyk, q, k, dq, dk, dgq, dgk)
    for x, dy, d, dg, gamma in ((qr, dqr, dq, dgq, c.gq), (kr, dkr, dk, dgk, c.gk)):
        dx, dgamma = c.want_back(dy, x, gamma)
        ref.check(d, dx, "dx")
        ref.check(dg, dgamma, "dgamma")
        # the terms are independent of each other: their roundings too, so the sum's error is far within that
        # bound, and a row left out is not
        assert float((dg.cpu().double() - dgamma[0]).norm() / dgamma[0].norm()) < 1e-5 + torch.finfo(c.W).eps


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("kind", [KINDS[0], KINDS[3]], ids=["f32", "bf16"])
def test_heads_of_large_calls(kind, interleaved):
    """Calls whose reads pass the caches (over 96 MB of them) against calls on parts of their rows, which do
    not: bit for bit by rows."""
    rows, dim = (24000, 256) if kind[0] == "bf16" else (12000, 250)
    log(f"large heads {kind} {rows}")
    c = HeadCase(kind, rows, 8, 2, dim, 96, interleaved, 4)
    g = torch.Generator("cuda").manual_seed(1)
    mat = lambda n: torch.empty(rows, n * dim, dtype=c.T, device="cuda").normal_(generator=g)  # noqa: E731
    q, k, dyq, dyk = mat(8), mat(2), mat(8), mat(2)
    dg = [torch.empty(dim, dtype=c.W, device="cuda") for _ in range(2)]
    outs = []
    for parts in (1, 5):
        o = [torch.full((rows, n * dim), FILL, dtype=c.T, device="cuda") for n in (8, 2, 8, 2)]
        for i in range(parts):
            sl = slice(rows * i // parts, rows * (i + 1) // parts)
            d = HeadCase(kind, 1, 8, 2, dim, 96, interleaved, 4)
            d.rows, d.positions, d.cu, d.flags = sl.stop - sl.start, c.positions[sl], c.cu, c.flags
            d.forward(q[sl], k[sl], o[0][sl], o[1][sl])
            d.backward(dyq[sl], dyk[sl], q[sl], k[sl], o[2][sl], o[3][sl], *dg)
        outs.append(o)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_heads_of_more_rows_than_a_grid():
    """Past 2^22 rows a wave goes on to further ones."""
    rows = (1 << 22) + 9
    log("heads of more rows than a grid")
    g = torch.Generator("cuda").manual_seed(1)
    q, dy = (torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    pos = torch.randint(-1, 51, (rows,), generator=g, device="cuda", dtype=torch.int32)
    angle = torch.rand(50, 1, generator=g, device="cuda") * 7
    cos, sin = angle.cos(), angle.sin()
    outs = []
    for cuts in ((0, rows), (0, 5, 1 << 21, (1 << 22) - 3, rows)):
        y, d = (torch.full((rows, 2), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for lo, hi in zip(cuts, cuts[1:]):
            at = slice(lo, hi)
            tk.tk_head_norm_rotate_bf16(hi - lo, 1, 0, 2, 2, 1e-5, 0, q[at], None, None, None, None, None, pos[at], 50, cos, sin, y[at],
                                        None, None, None)
            tk.tk_head_norm_rotate_backward_bf16(hi - lo, 1, 0, 2, 2, 1e-5, 0, dy[at], None, None, None, q[at], None, None, None, None,
                                                 None, pos[at], 50, cos, sin, d[at], None, None, None, None, None)
        outs.append((y, d))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    n = 2000  # and against the definition at both ends
    for at in (slice(0, n), slice(rows - n, rows)):
        p = pos[at].long().cpu()
        there = ((p >= 0) & (p < 50))[:, None]
        c = torch.where(there, cos.cpu()[p.clamp(0, 49)].double(), 1.0)
        s = torch.where(there, sin.cpu()[p.clamp(0, 49)].double(), 0.0)
        x, e = tok.head_norm_rotate(q[at].cpu().double().view(n, 1, 2), None, c, s, False, 1e-5)
        ref.check(outs[0][0][at], (x.view(n, 2), e.view(n, 2)), "far rows")
        x, e = tok.head_norm_rotate_backward(dy[at].cpu().double().view(n, 1, 2), q[at].cpu().double().view(n, 1, 2), None, c, s, False,
                                             1e-5)["dx"]
        ref.check(outs[0][1][at], (x.view(n, 2), e.view(n, 2)), "far rows' gradient")


@pytest.mark.parametrize("hq,hk", [(140000, 9), (600000, 1000)])
def test_heads_of_more_heads_than_a_grid(hq, hk):
    """Past 4096 units a row's work-groups go on to further heads: the bits of as many rows of one head."""
    log(f"{hq}+{hk} heads")
    g = torch.Generator("cuda").manual_seed(hq)
    q, k, dyq, dyk = (torch.empty(1, n * 2, device="cuda").normal_(generator=g) for n in (hq, hk, hq, hk))
    gamma = [1 + 0.3 * torch.randn(2, generator=g, device="cuda") for _ in range(2)]
    angle = torch.rand(9, 1, generator=g, device="cuda") * 7
    cos, sin = angle.cos(), angle.sin()
    yq, yk, dq, dk = (torch.full_like(t, FILL) for t in (q, k, q, k))
    pos = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    tail = (*gamma, pos, 9, cos, sin)
    tk.tk_head_norm_rotate_f32(1, hq, hk, 2, 2, 1e-5, 0, q, None, k, None, *tail, yq, None, yk, None)
    tk.tk_head_norm_rotate_backward_f32(1, hq, hk, 2, 2, 1e-5, 0, dyq, None, dyk, None, q, None, k, None, *tail, dq, None, dk, None,
                                        None, None)
    for x, dy, y, d, ga, n in ((q, dyq, yq, dq, gamma[0], hq), (k, dyk, yk, dk, gamma[1], hk)):
        at, y1, d1 = pos.expand(n).contiguous(), torch.empty(n, 2, device="cuda"), torch.empty(n, 2, device="cuda")
        one = lambda t: t.view(n, 2)  # noqa: E731
        tk.tk_head_norm_rotate_f32(n, 1, 0, 2, 2, 1e-5, 0, one(x), None, None, None, ga, None, at, 9, cos, sin, y1, None, None, None)
        tk.tk_head_norm_rotate_backward_f32(n, 1, 0, 2, 2, 1e-5, 0, one(dy), None, None, None, one(x), None, None, None, ga, None, at, 9,
                                            cos, sin, d1, None, None, None, None, None)
        assert torch.equal(one(y), y1) and torch.equal(one(d), d1)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[3]], ids=["f32", "bf16"])
def test_heads_in_place_and_in_slices(kind):
    """Slices of one projection's output (as matrices and as views of heads), outputs in place of inputs,
    and rows one by one: the bits of separate matrices."""
    T = types(kind)[0]
    hq, hk, dim, rows = 5, 2, 96, 67
    c = HeadCase(kind, rows, hq, hk, dim, 64, True, 4)
    nq, nk = hq * dim, hk * dim
    m = Maker(rows, nq + 2 * nk, 0, 1)
    qkv, dqkv = m.mat(T)[0], m.mat(T)[0]
    q, k, dyq, dyk = (t[:, s].contiguous() for t in (qkv, dqkv) for s in (slice(0, nq), slice(nq, nq + nk)))
    new = lambda n, t=T: torch.full((rows, n), FILL, dtype=t, device="cuda")  # noqa: E731
    yq, yk, dq, dk = new(nq), new(nk), new(nq), new(nk)
    dg = [torch.empty(dim, dtype=c.W, device="cuda") for _ in range(4)]
    c.forward(q, k, yq, yk)
    c.backward(dyq, dyk, q, k, dq, dk, dg[0], dg[1])
    heads = lambda t: (t[:, :nq].view(rows, hq, dim), t[:, nq:nq + nk].view(rows, hk, dim))  # noqa: E731
    out = torch.full_like(qkv, FILL)
    c.forward(*heads(qkv), *heads(out))
    assert torch.equal(out[:, :nq], yq) and torch.equal(out[:, nq:nq + nk], yk) and bool((out[:, nq + nk:] == FILL).all())
    out = dqkv.clone()
    c.backward(*heads(out), *heads(qkv), *heads(out), dg[2], dg[3])  # in place of dy
    assert torch.equal(out[:, :nq], dq) and torch.equal(out[:, nq:nq + nk], dk)
    assert torch.equal(out[:, nq + nk:], dqkv[:, nq + nk:])
    assert torch.equal(dg[0], dg[2]) and torch.equal(dg[1], dg[3])
    x = qkv.clone()
    c.backward(*heads(dqkv), *heads(x), *heads(x), dg[2], None)  # in place of x
    assert torch.equal(x[:, :nq], dq) and torch.equal(x[:, nq:nq + nk], dk) and torch.equal(dg[0], dg[2])
    x = qkv.clone()
    c.forward(*heads(x), *heads(x))
    assert torch.equal(x[:, :nq], yq) and torch.equal(x[:, nq:nq + nk], yk)
    for r in (0, 33, 66):  # a row does not see the others
        one = HeadCase(kind, 1, hq, hk, dim, 64, True, 4)
        one.positions, one.cu, one.flags = c.positions[r:r + 1], c.cu, c.flags
        a, b = new(nq)[:1], new(nk)[:1]
        one.forward(q[r:r + 1], k[r:r + 1], a, b)
        assert torch.equal(a[0], yq[r]) and torch.equal(b[0], yk[r])


def test_heads_of_non_finite_values_and_zeros():
    """A NaN or an infinity stays in its head; what does not turn is not touched by one in a pair's other place."""
    c = HeadCase(KINDS[0], 4, 3, 1, 40, 16, False, 2, gamma=False)
    q, k = torch.randn(4, 120, device="cuda"), torch.randn(4, 40, device="cuda")
    q[1, 45], k[2, 3] = float("nan"), float("inf")
    q[3, 80:] = 0
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    c.forward(q, k, yq, yk)
    bad = yq.isnan().view(4, 3, 40)
    assert bool(bad[1, 1].all()) and int(bad.sum()) == 40
    assert int(yk.isnan().sum()) >= 1 and not bool(yk[[0, 1, 3]].isnan().any())
    assert not bool(yq[3, 80:].any())  # zeros give zeros: eps keeps the root away from them


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("kind", [KINDS[0], KINDS[3]], ids=["f32", "bf16"])
def test_heads_beyond_floats_range(kind, interleaved):
    """A head whose squares pass float's range is zeros, as are its gradients, and the other heads and the sums of
    the gammas are as without it; with eps 0 a head whose squares vanish is infinite or NaN, alone."""
    T, _, W = types(kind)
    rows, hq, hk, dim = 5, 3, 2, 40
    log(f"heads beyond float's range {kind} {interleaved}")
    c = HeadCase(kind, rows, hq, hk, dim, 16, interleaved, 2)
    g = torch.Generator("cuda").manual_seed(3)
    q, k, dyq, dyk = (torch.randn(rows, n * dim, generator=g, device="cuda").to(T) for n in (hq, hk, hq, hk))
    big = [(q, 1, 2, torch.finfo(T).min), (q, 3, 0, 2.0 ** 100), (k, 0, 1, torch.finfo(T).max)]  # matrix, row, head, value
    at = lambda t, r, h: t[r, h * dim:(h + 1) * dim]  # noqa: E731
    outs = []
    for with_big in (False, True):
        for x, r, h, v in big:
            at(x, r, h).fill_(0)  # a head of zeros: its h is 0 too, so nothing of it in the gammas' gradients
            if with_big:
                at(x, r, h)[torch.arange(h, dim, 7)] = v
        o = [torch.full_like(t, FILL) for t in (q, k, q, k)] + [torch.empty(dim, dtype=W, device="cuda") for _ in range(2)]
        c.forward(q, k, *o[:2])
        c.backward(dyq, dyk, q, k, *o[2:])
        outs.append(o)
    for x, r, h, _ in big:
        i = 0 if x is q else 1
        assert not bool(at(outs[1][i], r, h).any()) and not bool(at(outs[1][i + 2], r, h).any())
        assert not bool(at(outs[0][i], r, h).any())
        at(outs[0][i + 2], r, h).fill_(0)  # zeros have a gradient, at 1 / sqrt(eps)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    q = torch.randn(rows, hq * dim, generator=g, device="cuda").to(T)
    at(q, 2, 1).fill_(2.0 ** -80)
    y = torch.full_like(q, FILL)
    fn("head_norm_rotate", kind)(rows, hq, 0, dim, 0, 0.0, 0, q, None, None, None, None, None, None, 0, None, None, y, None, None, None)
    assert not bool(at(y, 2, 1).isfinite().any())
    at(y, 2, 1).fill_(0)
    assert bool(y.isfinite().all())


# ---- checkpoints ----
CODED = [(1, 1), (3, 7), (2, 8), (5, 9), (4, 127), (9, 128), (3, 129), (33, 200), (2, 1000), (70, 256), (5, 2049), (130, 513),
         (1, 70001)]


@pytest.mark.parametrize("kind", [k for k in KINDS if not k[2]] + [("f16", True, False)],
                         ids=["f32", "f16", "bf16", "bf16-r32", "f16-r32"])
def test_checkpoint(kind):
    T, R, _ = types(kind)
    for i, (rows, cols) in enumerate(CODED):
        pad = (0, 3, 8)[i % 3]
        what = f"checkpoint {kind} {rows}x{cols} pad {pad}"
        log(what)
        m = Maker(rows, cols, pad, i)
        x, xr = m.mat(R, 3.0)
        codes, scales = m.out(torch.int8), m.flat(rows * -(-cols // 128), torch.float32)
        fn("checkpoint", kind)(8, 5 + i, rows, cols, flags(kind), x, None, codes, None, scales)
        c, s = tok.checkpoint(xr.float().numpy(), 8, 5 + i)
        assert np.array_equal(codes.cpu().numpy(), c), what
        assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.reshape(-1).view(np.uint32)), what
        y = m.out(R)
        fn("checkpoint_restore", kind)(rows, cols, flags(kind), codes, None, scales, y, None)
        v = tok.restored(torch.from_numpy(c), torch.from_numpy(s))
        assert torch.equal(y.cpu(), v.to(R)), what  # a float, rounded once to the type
        m.untouched(what)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1], KINDS[3]], ids=["f32", "f16", "bf16"])
def test_checkpoint_of_special_blocks(kind):
    R = types(kind)[1]
    g = torch.Generator().manual_seed(6)
    x = torch.randn(12, 300, generator=g).to(R)
    x[0] = 0
    x[1, :128] = 0
    x[1, 7] = 2.0 ** -14  # alone in its block
    x[2, 5], x[3, 200], x[4, 299], x[5, 130] = float("inf"), float("nan"), -float("inf"), -float("nan")
    x[6] = torch.finfo(R).max
    x[7] = torch.finfo(R).smallest_normal * (1.0 if R is torch.float16 else 2.0 ** 30)
    x[8] = -0.0
    x[9] *= torch.finfo(R).smallest_normal
    x[10] = torch.arange(300).to(R)  # whole codes where the largest is 127
    x[11, :128] = torch.arange(128).to(R)
    codes, scales = torch.full((12, 300), 99, dtype=torch.int8, device="cuda"), torch.full((12, 3), FILL, device="cuda")
    fn("checkpoint", kind)(8, 3, 12, 300, 0, x.cuda(), None, codes, None, scales)
    c, s = tok.checkpoint(x.float().numpy(), 8, 3)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.isnan().cpu().numpy(), np.isnan(s))
    assert np.array_equal(np.nan_to_num(scales.cpu().numpy(), nan=-1), np.nan_to_num(s, nan=-1))
    assert torch.equal(codes[11, :128].cpu().float(), torch.arange(128.0))
    y = torch.empty(12, 300, dtype=R, device="cuda")
    fn("checkpoint_restore", kind)(12, 300, 0, codes, None, scales, y, None)
    bad = y.isnan().cpu()
    for r, lo in ((2, 0), (3, 128), (4, 256), (5, 128)):
        assert bool(bad[r, lo:lo + 128].all())
        bad[r, lo:lo + 128] = False
    assert not bool(bad.any()) and not bool(y[[0, 8]].any())


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[2], KINDS[4]], ids=["f32", "f16-r32-p32", "bf16-r32"])
@pytest.mark.parametrize("cols", [3, 300, 9001])
def test_checkpoint_of_floats_largest(kind, cols):
    """A block that holds float's largest, either sign, comes back finite, and the backward passes from its codes
    see those values.  Its scale, m / 127 rounded, is a step too high: 127 times it is infinite."""
    T, R, W = types(kind)
    rows, most = 5, np.finfo(np.float32).max
    log(f"float's largest {kind} {cols}")
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols, generator=g)
    x[0], x[1], x[2, 1], x[3, cols - 1] = float(most), -float(most), float(most), -float(most)
    codes, scales = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, -(-cols // 128), device="cuda")
    fl = flags(kind)
    fn("checkpoint", kind)(8, 3, rows, cols, fl & tk.TK_RESIDUAL_F32, x.cuda(), None, codes, None, scales)
    c, s = tok.checkpoint(x.numpy(), 8, 3)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    high = most / np.float32(127)
    assert int((s == high).sum()) >= 4
    with np.errstate(over="ignore"):
        assert np.isinf(high * np.float32(127))
    held = np.minimum(s, np.nextafter(high, np.float32(0)))  # most / 127 rounded down
    v = tok.restored(torch.from_numpy(c), torch.from_numpy(held))
    assert bool(torch.isfinite(v.float()).all())
    y = torch.empty(rows, cols, dtype=R, device="cuda")
    fn("checkpoint_restore", kind)(rows, cols, fl & tk.TK_RESIDUAL_F32, codes, None, scales, y, None)
    assert torch.equal(y.cpu(), v.to(R))
    # a norm of such rows: as the forward's statistics are inputs, any in range serve
    mean, rstd = torch.zeros(rows), torch.full((rows,), 2.0 ** -120)
    m = Maker(rows, cols, 0, 1)
    (dy, dyr), (ds, dsr), (gamma, gr) = m.mat(T), m.mat(R), m.vec(W, 1.0)
    dx, dr, dg, db, dbias = m.out(T), m.out(R), m.flat(cols, W), m.flat(cols, W), m.flat(cols, W)
    fn("dropout_add_layer_norm_backward_checkpoint", kind)(8, 5, rows, cols, 0.25, fl, dy, None, ds, None, codes, None, scales,
                                                           gamma, mean.cuda(), rstd.cuda(), dx, None, dr, None, dg, db, dbias)
    want = ref.dropout_add_layer_norm_backward(dyr, dsr, v, gr, mean.double(), rstd.double(), ref.keep_mask(8, 5, rows, cols, 0.25),
                                               0.25)
    for name, t in (("dx", dx), ("dresidual", dr), ("dgamma", dg), ("dbeta", db), ("dbias", dbias)):
        ref.check(t, want[name], f"{kind} {cols} {name}")
    m.untouched(f"{kind} {cols}")


def test_checkpoint_is_cut_at_any_row_and_right_on_average():
    rows, cols = 300, 1111
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    whole, parts = (torch.empty(rows, cols, dtype=torch.int8, device="cuda") for _ in range(2))
    sw, sp = (torch.empty(rows, 9, device="cuda") for _ in range(2))
    tk.tk_checkpoint_bf16(4, 100, rows, cols, 0, x, None, whole, None, sw)
    for lo, hi in ((0, 1), (1, 140), (140, 300)):
        tk.tk_checkpoint_bf16(4, 100 + lo * cols, hi - lo, cols, 0, x[lo:hi], None, parts[lo:hi], None, sp[lo:hi])
    assert torch.equal(whole, parts) and torch.equal(sw, sp)
    # the same values 64 times over, other draws each: a mean's error is within five of its deviations (a code
    # is off by less than one step, with a variance of at most a quarter)
    x = torch.randn(1, 128, device="cuda").expand(4096, 128).contiguous()
    codes, scales = torch.empty(4096, 128, dtype=torch.int8, device="cuda"), torch.empty(4096, device="cuda")
    tk.tk_checkpoint_f32(4, 0, 4096, 128, 0, x, None, codes, None, scales)
    mean = (codes.double() * scales.double()[:, None]).mean(0)
    assert bool(((mean - x[0].double()).abs() <= 6 * 0.5 / 64 * float(scales[0])).all())


def test_checkpoint_of_very_many_rows():
    """More chunks than one launch takes (2^30): rows of one column, each a block."""
    rows, n = (1 << 27) + 5, 1000
    log("checkpoint of very many rows")
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    x[-n:, 0] = torch.randn(n, device="cuda").bfloat16()
    codes, scales = torch.full((rows, 1), 99, dtype=torch.int8, device="cuda"), torch.full((rows,), FILL, device="cuda")
    tk.tk_checkpoint_bf16(4, 9, rows, 1, 0, x, None, codes, None, scales)
    assert bool((codes[:-n] == 127).all())
    c, s = tok.checkpoint(x[-n:].float().cpu().numpy(), 4, 9 + rows - n)
    assert np.array_equal(codes[-n:].cpu().numpy(), c) and np.array_equal(scales[-n:].cpu().numpy(), s[:, 0])
    assert bool((scales[:-n] == scales[0]).all())


def test_restore_of_very_many_rows():
    """More chunks than one launch of the restore takes (2^30): rows of one column."""
    rows, n = (1 << 30) + 700, 2000
    log("restore of very many rows")
    codes = torch.full((rows, 1), 3, dtype=torch.int8, device="cuda")
    scales = torch.full((rows,), 0.5, device="cuda")
    codes[-n:, 0] = torch.randint(-127, 128, (n,), device="cuda", dtype=torch.int8)
    scales[-n:] = torch.rand(n, device="cuda")
    y = torch.full((rows, 1), FILL, dtype=torch.bfloat16, device="cuda")
    tk.tk_checkpoint_restore_bf16(rows, 1, 0, codes, None, scales, y, None)
    assert torch.equal(y[-n:, 0], (codes[-n:, 0].float() * scales[-n:]).bfloat16())
    assert bool((y[:-n] == 1.5).all())


def test_checkpoint_at_the_counters_end():
    """The last draws of a key, and one more element refused."""
    rows, cols = 2, 300
    x = torch.randn(rows, cols, device="cuda")
    codes, scales = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, 3, device="cuda")
    start = (1 << 32) - rows * cols
    tk.tk_checkpoint_f32(9, start, rows, cols, 0, x, None, codes, None, scales)
    assert np.array_equal(codes.cpu().numpy(), tok.checkpoint(x.cpu().numpy(), 9, start)[0])
    with pytest.raises(tk.TkError):
        tk.tk_checkpoint_f32(9, start + 1, rows, cols, 0, x, None, codes, None, scales)


# rows, cols of the backward passes from codes: every shape of their kernels
BACK = [(1, 1), (3, 5), (33, 8), (9, 60), (50, 128), (7, 129), (6, 300), (70, 512), (5, 1000), (33, 2049), (5, 5001), (2, 8192),
        (3, 8193), (2, 16385), (2500, 40), (1201, 1032), (300, 1500), (4200, 600)]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_backward_from_codes(kind):
    T, R, W = types(kind)
    for i, (rows, cols) in enumerate(BACK):
        for p, with_dsum, with_bias, fused in ((0.25, True, True, True), (0.0, False, False, True), (0.0, False, False, False)):
            what = f"backward from codes {kind} {rows}x{cols} p {p} dsum {with_dsum} bias {with_bias} fused {fused}"
            log(what)
            m = Maker(rows, cols, (0, 3, 8)[i % 3], i)
            x = (torch.randn(rows, cols, generator=m.g) * 2 + 0.5).numpy()
            c, s = tok.checkpoint(x, 3, i)
            v = tok.restored(torch.from_numpy(c), torch.from_numpy(s))
            codes = m.place(torch.int8)[1]
            codes.copy_(torch.from_numpy(c))
            scales = torch.from_numpy(s).cuda()
            mean = torch.from_numpy(x.mean(1))
            rstd = torch.from_numpy(1 / np.sqrt(x.var(1) + np.float32(1e-3)))
            dy, dyr = m.mat(T)
            g, gr = m.vec(W, 1.0)
            dg, db = m.flat(cols, W), m.flat(cols, W)
            if not fused:
                dx = m.out(R)
                fn("layer_norm_backward_checkpoint", kind)(rows, cols, flags(kind), dy, None, codes, None, scales, g, mean.cuda(),
                                                           rstd.cuda(), dx, None, dg, db)
                grad, e, more = ref.layer_norm_backward(dyr, v, gr, mean.double(), rstd.double())
                ref.check(dx, (grad, e), what + " dx")
                want = more
            else:
                ds, dsr = m.mat(R) if with_dsum else (None, None)
                dx, dr, dbias = m.out(T), m.out(R), m.flat(cols, W) if with_bias else None
                keep = ref.keep_mask(8, 5 + i, rows, cols, p)
                fn("dropout_add_layer_norm_backward_checkpoint", kind)(
                    8, 5 + i, rows, cols, p, flags(kind), dy, None, ds, None, codes, None, scales, g, mean.cuda(), rstd.cuda(),
                    dx, None, dr, None, dg, db, dbias)
                want = ref.dropout_add_layer_norm_backward(dyr, dsr, v, gr, mean.double(), rstd.double(), keep, p)
                ref.check(dx, want["dx"], what + " dx")
                ref.check(dr, want["dresidual"], what + " dresidual")
                if with_bias:
                    ref.check(dbias, want["dbias"], what + " dbias")
            ref.check(dg, want["dgamma"], what + " dgamma")
            ref.check(db, want["dbeta"], what + " dbeta")
            m.untouched(what)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[4]], ids=["f32", "bf16-r32"])
@pytest.mark.parametrize("cols", [200, 1000, 9001])
def test_backward_from_codes_is_that_of_their_values(kind, cols):
    """The row operators' own backward passes at the restored float values give the same bits, where the
    residual stream is float; also where the reads pass the caches."""
    T, R, W = types(kind)
    for rows in (37, -(-40_000_000 // cols)):
        log(f"{kind} {rows}x{cols}")
        g = torch.Generator("cuda").manual_seed(rows)
        mat = lambda t: torch.empty(rows, cols, dtype=t, device="cuda").normal_(generator=g)  # noqa: E731
        x, dy, ds = mat(torch.float32), mat(T), mat(R)
        codes, scales = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, -(-cols // 128), device="cuda")
        fl = flags(kind)
        fn("checkpoint", kind)(2, 7, rows, cols, fl, x, None, codes, None, scales)
        v = torch.empty_like(x)
        fn("checkpoint_restore", kind)(rows, cols, fl, codes, None, scales, v, None)
        mean, rstd = x.mean(1), x.var(1).rsqrt()
        outs = []
        for name, args in (("", (v, None)), ("_checkpoint", (codes, None, scales))):
            o = [torch.empty(rows, cols, dtype=t, device="cuda") for t in (T, R)]
            o += [torch.empty(cols, dtype=W, device="cuda") for _ in range(3)]
            fn("dropout_add_layer_norm_backward" + name, kind)(8, 9, rows, cols, 0.1, fl, dy, None, ds, None, *args, None, mean,
                                                               rstd, o[0], None, o[1], None, *o[2:])
            o2 = [torch.empty(rows, cols, dtype=R, device="cuda")] + [torch.empty(cols, dtype=W, device="cuda") for _ in range(2)]
            fn("layer_norm_backward" + name, kind)(rows, cols, fl, dy, None, *args, None, mean, rstd, o2[0], None, *o2[1:])
            outs.append(o + o2)
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_rows_beyond_32_bits():
    """Heads and checkpoints whose last rows begin past 2^32 elements, at the largest row distance: the bits of
    dense rows, and nothing written beside the rows."""
    rows, ld, hq, hk, dim = 4, (1 << 31) - 1, 3, 2, 64
    cols = (hq + hk) * dim
    log("rows beyond 32 bits")
    g = torch.Generator("cuda").manual_seed(6)
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    far = torch.full((3 * ld + cols + 9,), FILL, dtype=torch.bfloat16, device="cuda")
    at = far.as_strided((rows, cols), (ld, 1))
    beside = lambda b: all(bool((b[r * ld + cols:r * ld + cols + 9] == FILL).all()) for r in range(rows))  # noqa: E731
    angle = torch.rand(rows, 32, generator=g, device="cuda") * 7
    shape = (rows, hq, hk, dim, dim, 1e-5, 0)
    tail = (None, None, None, rows, angle.cos(), angle.sin())
    q, k = slice(0, hq * dim), slice(hq * dim, cols)
    y, d = (torch.full((rows, cols), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tk.tk_head_norm_rotate_bf16(*shape, x[:, q], None, x[:, k], None, *tail, y[:, q], None, y[:, k], None)
    at.copy_(x)
    tk.tk_head_norm_rotate_bf16(*shape, at[:, q], None, at[:, k], None, *tail, at[:, q], None, at[:, k], None)
    assert torch.equal(at, y) and beside(far)
    tk.tk_head_norm_rotate_backward_bf16(*shape, dy[:, q], None, dy[:, k], None, x[:, q], None, x[:, k], None, *tail, d[:, q], None,
                                         d[:, k], None, None, None)
    at.copy_(x)
    tk.tk_head_norm_rotate_backward_bf16(*shape, dy[:, q], None, dy[:, k], None, at[:, q], None, at[:, k], None, *tail, at[:, q], None,
                                         at[:, k], None, None, None)
    assert torch.equal(at, d) and beside(far)
    at.copy_(x)
    codes, scales = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, 3, device="cuda")
    tk.tk_checkpoint_bf16(1, 2, rows, cols, 0, x, None, codes, None, scales)
    far_codes, far_scales = torch.full((3 * ld + cols + 9,), int(FILL), dtype=torch.int8, device="cuda"), torch.empty(rows, 3, device="cuda")
    at_codes = far_codes.as_strided((rows, cols), (ld, 1))
    tk.tk_checkpoint_bf16(1, 2, rows, cols, 0, at, None, at_codes, None, far_scales)
    assert torch.equal(at_codes, codes) and torch.equal(far_scales, scales) and beside(far_codes)
    tk.tk_checkpoint_restore_bf16(rows, cols, 0, codes, None, scales, y, None)
    tk.tk_checkpoint_restore_bf16(rows, cols, 0, at_codes, None, scales, at, None)
    assert torch.equal(at, y) and beside(far)
    mean, rstd = x.float().mean(1), x.float().var(1).rsqrt()
    dx, dr = (torch.full((rows, cols), FILL, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sums = [torch.empty(cols, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    tk.tk_dropout_add_layer_norm_backward_checkpoint_bf16(1, 2, rows, cols, 0.1, 0, dy, None, None, None, codes, None, scales, None, mean,
                                                          rstd, dx, None, dr, None, *sums[:3])
    at.copy_(dy)
    tk.tk_dropout_add_layer_norm_backward_checkpoint_bf16(1, 2, rows, cols, 0.1, 0, at, None, None, None, at_codes, None, scales, None,
                                                          mean, rstd, at, None, d, None, *sums[3:])
    assert torch.equal(at, dx) and torch.equal(d, dr) and beside(far)
    for a, b in zip(sums[:3], sums[3:]):
        assert torch.equal(a, b)


# ---- together ----
class Step:
    """A training step's run: tokens -> embedding -> checkpoint -> layer norm -> head norms of slices of the norm's
    output (in a projection's place), given gradients, and back to the table's gradient."""

    def __init__(self, kind, rows=150, hq=4, hk=2, dim=40, vocab=90, seed=3):
        self.kind, self.rows, self.vocab, self.p = kind, rows, vocab, 0.2
        self.T, self.R, self.W = T, R, W = types(kind)
        self.cols, self.hq, self.hk, self.dim = 264, hq, hk, dim
        self.nq, self.nk = hq * dim, hk * dim
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, k=1.0: torch.randn(*s, generator=g) * k  # noqa: E731
        self.host = {"table": rnd(vocab, self.cols).to(W), "gamma": (1 + rnd(self.cols, k=0.2)).to(W),
                     "beta": rnd(self.cols, k=0.2).to(W), "gq": (1 + rnd(dim, k=0.2)).to(W), "gk": (1 + rnd(dim, k=0.2)).to(W)}
        self.dout = rnd(rows, self.nq + self.nk).to(T)
        self.ids = tokens(rows, vocab, "skewed", True, seed)
        self.ids[5] = -1
        angle = torch.arange(rows)[:, None] * 50.0 ** (-torch.arange(dim // 2) / (dim // 2))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.d = {k: v.cuda() for k, v in self.host.items()}
        for k in ("dout", "ids", "cos", "sin"):
            self.d[k] = getattr(self, k).cuda()
        e = lambda n, t: torch.full((rows, n), FILL, dtype=t, device="cuda")  # noqa: E731
        self.d.update(x=e(self.cols, R), codes=e(self.cols, torch.int8), scales=e(3, torch.float32), h=e(self.cols, T),
                      mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"),
                      y=e(self.nq + self.nk, T), dh=torch.zeros(rows, self.cols, dtype=T, device="cuda"), dx=e(self.cols, R))
        self.outs = {k: torch.full_like(self.d[k], FILL) for k in self.host}
        self.ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
            tk.tk_embedding_workspace_bytes(rows, self.cols, vocab), tk.tk_head_norm_workspace_bytes(rows, hq, hk, dim),
            tk.tk_backward_workspace_bytes(rows, self.cols) + 1)]

    def run(self, stream=None):
        d, k, f, rows, cols = self.d, self.kind, flags(self.kind), self.rows, self.cols
        hf = f & tk.TK_PARAMS_F32
        shape = (rows, self.hq, self.hk, self.dim, self.dim, 1e-5, hf)
        nq, n = self.nq, self.nq + self.nk
        q, kk, dq, dk = d["h"][:, :nq], d["h"][:, nq:n], d["dh"][:, :nq], d["dh"][:, nq:n]
        fn("embedding", k)(1, 3, rows, cols, self.p, 2.0, f | tk.TK_INDEX_I64, self.vocab, d["ids"], d["table"], None, d["x"], None,
                           stream)
        fn("checkpoint", k)(2, 0, rows, cols, f & tk.TK_RESIDUAL_F32, d["x"], None, d["codes"], None, d["scales"], stream)
        fn("layer_norm", k)(rows, cols, 1e-5, f, d["x"], None, d["gamma"], d["beta"], d["h"], None, d["mean"], d["rstd"], stream)
        fn("head_norm_rotate", k)(*shape, q, None, kk, None, d["gq"], d["gk"], None, rows, d["cos"], d["sin"], d["y"][:, :nq], None,
                                  d["y"][:, nq:], None, stream)
        o = self.outs
        fn("head_norm_rotate_backward", k)(*shape, d["dout"][:, :nq], None, d["dout"][:, nq:], None, q, None, kk, None, d["gq"],
                                           d["gk"], None, rows, d["cos"], d["sin"], dq, None, dk, None,
                                           o["gq"], o["gk"], self.ws[1], stream)
        fn("layer_norm_backward_checkpoint", k)(rows, cols, f, d["dh"], None, d["codes"], None, d["scales"], d["gamma"], d["mean"],
                                                d["rstd"], d["dx"], None, o["gamma"], o["beta"], self.ws[2], stream)
        fn("embedding_backward", k)(1, 3, rows, cols, self.p, 2.0, f | tk.TK_INDEX_I64, self.vocab, d["ids"], d["dx"], None,
                                    o["table"], None, self.ws[0], stream)

    def results(self):
        return {**self.outs, "y": self.d["y"], "x": self.d["x"], "codes": self.d["codes"]}


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_a_steps_run(kind):
    """Against float64 autograd of the same step; the layer norm's backward sees the checkpoint there too."""
    s = Step(kind)
    s.run()
    torch.cuda.synchronize()
    v = {k: t.double().requires_grad_() for k, t in s.host.items()}
    keep = ref.keep_mask(1, 3, s.rows, s.cols, s.p)
    there = (s.ids >= 0)[:, None]
    x = torch.where(there, v["table"][s.ids.clamp(min=0)] * 2.0, 0.0) * keep / ref.quotient(s.p)
    # the values that the operator gave, with the gradient of the formula, and for the norm's gradient its checkpoint
    codes, scales = (s.d[k].cpu() for k in ("codes", "scales"))
    mean, rstd = s.d["mean"].cpu().double()[:, None], s.d["rstd"].cpu().double()[:, None]

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gamma, beta):
            return (x - mean) * rstd * gamma + beta

        @staticmethod
        def backward(ctx, dy):
            g, _, more = ref.layer_norm_backward(dy, tok.restored(codes, scales), v["gamma"].detach(), mean[:, 0], rstd[:, 0])
            return g, more["dgamma"][0], more["dbeta"][0]

    h = Norm.apply(x, v["gamma"], v["beta"])
    qk = h[:, :s.nq + s.nk]

    def heads(t, gamma):
        t = t.view(s.rows, -1, s.dim)
        t = t * (t.square().mean(-1, keepdim=True) + 1e-5) ** -0.5 * gamma
        a, b = t[..., :s.dim // 2], t[..., s.dim // 2:]
        c, sn = s.cos.double()[:, None], s.sin.double()[:, None]
        return torch.cat((a * c - b * sn, b * c + a * sn), -1).reshape(s.rows, -1)

    y = torch.cat((heads(qk[:, :s.nq], v["gq"]), heads(qk[:, s.nq:], v["gk"])), 1)
    y.backward(s.dout.double())
    # at most eight roundings to the types between the inputs and any result, each off by half a step of values
    # of the same size: 16 half steps of the coarsest type, twice that because a gradient is a difference
    limit = 32 * torch.finfo(s.T).eps / 2 + 1e-5
    rel = lambda a, b: float((a.detach().cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert rel(s.d["x"], x.detach()) <= limit and rel(s.d["y"], y.detach()) <= limit
    for k, t in s.outs.items():
        assert rel(t, v[k].grad) <= limit, k


def same(a, b, what):
    for k in a:
        assert torch.equal(a[k], b[k]), (what, k)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[4]], ids=["f32", "bf16-r32"])
def test_a_captured_step(kind):
    """Replays with other tokens and other data, the eager calls and synchronizations between them."""
    s = Step(kind)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for r in range(4):
        t = Step(kind, seed=10 + r)
        t.run()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in t.results().items()}
        for k in ("table", "gamma", "beta", "gq", "gk", "dout", "ids", "cos", "sin"):
            s.d[k].copy_(t.d[k])
        for v in s.results().values():
            v.fill_(FILL)
        for w in s.ws:
            w.fill_(255)  # a workspace holds nothing between calls
        g.replay()
        torch.cuda.synchronize()
        same(s.results(), want, f"replay {r}")


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[3]], ids=["f32", "bf16"])
def test_two_steps_on_two_streams(kind):
    steps = [Step(kind, seed=1), Step(kind, rows=700, vocab=5000, seed=2)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in s.results().items()} for s in steps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(3):
        for s in steps:
            for v in s.results().values():
                v.fill_(FILL)
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            s.run(st)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            same(s.results(), w, f"round {r}")


def test_binding_checks_on_the_device():
    """What the binding refuses of device tensors, before any launch."""
    x = torch.zeros(4, 3, 16, device="cuda")
    y, none = torch.zeros(4, 24, device="cuda"), (None,) * 2
    with pytest.raises(ValueError, match="heads"):  # heads that are apart
        tk.tk_head_norm_rotate_f32(4, 3, 0, 8, 8, 1e-5, 0, x[:, :, :8], None, None, None, *none, None, 0, *none, y, None, *none)
    with pytest.raises(ValueError, match="matrix"):
        tk.tk_head_norm_rotate_f32(4, 3, 0, 8, 8, 1e-5, 0, y, 25, None, None, *none, None, 0, *none, y, None, *none)
    with pytest.raises(ValueError, match="vector"):  # a table of other sizes
        tk.tk_head_norm_rotate_f32(4, 3, 0, 8, 8, 1e-5, 0, y, None, None, None, *none, None, 9, y, y, y, None, *none)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="vector"):
        tk.tk_embedding_f32(1, 0, 3, 24, 0.0, 1.0, tk.TK_INDEX_I64, 9, ids, torch.zeros(9, 24, device="cuda"), None, y, None)
    with pytest.raises(ValueError, match="workspace"):
        tk.tk_embedding_backward_f32(1, 0, 4, 24, 0.0, 1.0, tk.TK_INDEX_I64, 9, ids, y, None, torch.zeros(9, 24, device="cuda"),
                                     None, None, torch.cuda.Stream())
    codes, scales = torch.zeros(4, 24, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
    with pytest.raises(ValueError, match="vector"):  # a scale to every block
        tk.tk_checkpoint_f32(1, 0, 4, 24, 0, y, None, codes, None, scales)
    with pytest.raises(ValueError, match="vector"):
        tk.tk_checkpoint_restore_f32(4, 24, 0, codes, None, scales, y, None)
