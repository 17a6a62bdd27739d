"""GPU tests of the calls of a layer over a paged cache against their definitions in 64 bits.

Tolerances.  A rounding to a type is off by at most half a step, u = eps / 2 relative to
the value (plus half the smallest subnormal); a chain of n 32-bit additions or fused
multiply-adds is off by at most n 2^-24 times the sum of the terms' magnitudes.  Moves without
arithmetic are held to equality."""
import math

import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
F8 = torch.float8_e4m3fn
U32 = 2.0 ** -24
NAN = float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    info = torch.finfo(dtype)
    return info.tiny * info.eps / 2


# --------------------------------------------------------------------------
# Attention
# --------------------------------------------------------------------------

class Case:
    """Sequences of new[s] new tokens and lengths[s] places, on pages in no order.  What no token
    sees is NaN: places behind a sequence's end, pages of nobody, rows of q of nobody."""

    def __init__(self, new, lengths, page, q_heads, heads, dim, v_dim, dtype, narrow="no", window=0,
                 first=False, before=0, behind=0, seed=0, spread=1.0):
        g = _gen(seed + dim)
        self.new, self.lengths, self.page, self.window, self.dtype = new, lengths, page, window, dtype
        batch, self.group = len(new), q_heads // heads
        width = max([1] + [(n + page - 1) // page for n in lengths]) + 1
        pages = batch * width + 2
        self.table = torch.randperm(pages, generator=g)[:batch * width].reshape(batch, width).to(torch.int32)
        tokens = before + sum(new) + behind
        self.starts = torch.tensor([before] + [before + sum(new[:s + 1]) for s in range(batch)],
                                   dtype=torch.int32)
        # rows of q and of the caches lie apart, at no multiple of 16 bytes where sizes are odd
        self.q = torch.full((tokens, q_heads, dim + 3), NAN).to(dtype)[..., 1:dim + 1]
        self.q[before:before + sum(new)] = (torch.randn(sum(new), q_heads, dim, generator=g) * spread).to(dtype)
        kind = F8 if narrow != "no" else dtype

        def pool(d):
            x = torch.randn(pages, page, heads, d, generator=g)
            x = (x * 40).clamp(-448, 448).to(F8) if kind == F8 else x.to(dtype)
            seen = torch.zeros(pages, page, dtype=torch.bool)
            for s, length in enumerate(lengths):
                for p in range(max(length, 0)):
                    seen[self.table[s, p // page].long(), p % page] = True
            return torch.where(seen[..., None, None], x.float(), NAN).to(kind)
        self.k, self.v = pool(dim), pool(v_dim)
        self.first, self.scales = first, (None, None)
        if narrow == "head":
            self.scales = tuple(torch.rand(heads, generator=g) * 0.03 + 0.01 for _ in range(2))
        elif narrow == "one":
            self.scales = tuple(torch.rand((), generator=g) * 0.03 + 0.01 for _ in range(2))
        elif narrow == "row":
            self.scales = tuple(torch.rand(pages, page, heads, generator=g) * 0.03 + 0.01 for _ in range(2))

    def rows(self, s, which):
        """[length, heads, dim] of a sequence, in 64 bits."""
        at = torch.arange(max(self.lengths[s], 0))
        page, place = self.table[s, at // self.page].long(), at % self.page
        there = (page >= 0) & (page < self.k.shape[0])
        page = torch.where(there, page, 0)
        x = (self.k, self.v)[which][page, place].double()
        scale = self.scales[which]
        if scale is not None:
            scale = scale.double()
            x = x * (scale[page, place] if scale.dim() == 3 else scale.expand(x.shape[1]))[..., None]
        return x, there

    def want(self, scale):
        """The result, and what it may be off by."""
        heads, v_dim = self.k.shape[2], self.v.shape[3]
        out = torch.zeros(*self.q.shape[:2], v_dim, dtype=torch.float64)
        slack = torch.zeros_like(out)
        u = _u(self.dtype)
        for s, n in enumerate(self.new):
            if n == 0:
                continue
            (k, there), (v, _) = self.rows(s, 0), self.rows(s, 1)
            length = max(self.lengths[s], 0)
            at, i = torch.arange(length), torch.arange(n)
            place = length - n + i
            see = (at <= place[:, None]) & there
            if self.window:
                see &= at > place[:, None] - self.window
            x = self.q[self.starts[s]:self.starts[s + 1]].double()
            for h in range(self.q.shape[1]):
                kh, vh, xh = k[:, h // self.group], v[:, h // self.group], x[:, h]
                a = scale * (xh @ kh.t())
                # scores: a chain of products, and the scale, the maximum and the power of two
                off = scale * (xh.shape[1] + 16) * U32 * (xh.abs() @ kh.abs().t()) + 4 * U32
                a, off = a.masked_fill(~see, -math.inf), off.masked_fill(~see, 0.0)
                top = a.amax(1, keepdim=True) if length else a.sum(1, keepdim=True)
                w = torch.exp(a - torch.where(top.isfinite(), top, 0.0))
                total = w.sum(1, keepdim=True)
                w = torch.where(total > 0, w / total, 0.0)
                vz = torch.where(there[:, None], vh, 0.0)
                rows = slice(int(self.starts[s]), int(self.starts[s + 1]))
                size = w @ vz.abs()
                out[rows, h] = w @ vz
                # weights off by twice the scores' worst, rounded to the type; both sums; lost
                # below 2^-32 of the largest weight where the type has 5 exponent bits
                worst = 2 * off.amax(1, keepdim=True) if length else 0.0
                lost = 2.0 ** -31 * vz.abs().sum(0) if self.dtype == torch.float16 else 0.0
                slack[rows, h] = size * (u + worst + 2 * (length + 16) * U32) * 1.01 + lost
        return out, slack

    def on(self, x):
        x = x.to(DEV)
        return x.transpose(1, 2).contiguous().transpose(1, 2) if self.first and x.dim() >= 3 else x

    def args(self, starts=True):
        wide = torch.full((*self.q.shape[:2], self.q.shape[2] + 3), NAN, dtype=self.dtype, device=DEV)
        q = wide[..., 1:self.q.shape[2] + 1]
        q.copy_(self.q)
        return (q, self.on(self.k), self.on(self.v), self.table.to(DEV),
                torch.tensor(self.lengths, dtype=torch.int32, device=DEV)), dict(
                    starts=self.starts.to(DEV) if starts else None, window=self.window,
                    k_scale=None if self.scales[0] is None else self.on(self.scales[0]),
                    v_scale=None if self.scales[1] is None else self.on(self.scales[1]))

    def check(self, starts=True, scale=None, **kw):
        args, named = self.args(starts)
        got = bm.cache_attention(*args, scale=scale, **named, **kw)
        want, slack = self.want(scale or self.q.shape[2] ** -0.5)
        _within(got, want, slack, self.dtype)
        return got


def _within(got, want, slack, dtype):
    u = _u(dtype)
    got = got.double().cpu()
    assert got.shape == want.shape
    bound = slack * (1 + u) + u * want.abs() + _least(dtype)
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), "%d of %d values off, the worst by %g of what it may be" % (
        int(bad.sum()), bad.numel(), float(((got - want).abs() / bound)[bad].max()))


ATTEND = [  # new, lengths, page, q heads, heads, size, of values, window
    ([1], [1], 1, 1, 1, 8, 8, 0), ([1, 1, 1], [1, 0, 5], 4, 2, 1, 9, 15, 0),
    ([1, 1], [300, 17], 16, 8, 2, 64, 64, 0), ([1, 1], [700, 90], 16, 16, 1, 128, 128, 0),
    ([3, 0, 1, 5], [40, 9, 1, 5], 16, 6, 2, 80, 72, 0), ([17, 2], [64, 300], 32, 4, 4, 128, 40, 0),
    ([33], [33], 48, 5, 1, 96, 96, 0), ([20, 7], [400, 1000], 64, 8, 1, 128, 128, 100),
    ([1, 1, 1], [1000, 64, 65], 64, 4, 2, 128, 128, 64), ([2], [600], 7, 3, 3, 31, 33, 1),
    ([9], [200], 16, 2, 1, 192, 128, 0), ([5, 1], [130, 260], 16, 8, 2, 256, 256, 0),
    ([3, 1], [70, 200], 16, 4, 2, 320, 512, 0), ([1], [300], 16, 20, 1, 512, 257, 33),
    ([70], [170], 16, 40, 2, 64, 64, 0), ([130, 3], [150, 4], 16, 4, 1, 128, 128, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attention(case, dtype):
    new, lengths, page, q_heads, heads, dim, v_dim, window = case
    Case(new, lengths, page, q_heads, heads, dim, v_dim, dtype, window=window,
         first=page % 3 == 1).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("narrow", ["one", "head", "row"])
@pytest.mark.parametrize("case", ATTEND[1:14:2] + ATTEND[-2:], ids=str)
def test_attention_over_8_bits(case, narrow, dtype):
    new, lengths, page, q_heads, heads, dim, v_dim, window = case
    Case(new, lengths, page, q_heads, heads, dim, v_dim, dtype, narrow, window=window,
         first=page % 3 == 0).check()


@pytest.mark.parametrize("narrow", ["no", "row"])
def test_attention_one_token_each(narrow):
    """Without starts row s is sequence s's; an empty sequence gives zeros."""
    for dtype in TYPES:
        c = Case([1] * 5, [1, 0, 33, 200, -7], 16, 8, 2, 64, 48, dtype, narrow)
        got = c.check(starts=False)
        assert not bool(got[1].any()) and not bool(got[4].any())
        assert torch.equal(got, c.check(starts=True))


def test_attention_leaves_rows_of_nobody():
    """Rows before the first and behind the last sequence: zeros in a new tensor, left in a given one,
    between whose heads nothing is written."""
    for dtype in TYPES:
        c = Case([3, 1, 20], [5, 40, 90], 16, 4, 2, 40, 24, dtype, before=4, behind=30)
        got = c.check()
        mine = torch.zeros(len(got), dtype=torch.bool)
        mine[4:28] = True
        assert not bool(got.cpu()[~mine].any())
        wide = torch.full((got.shape[0], 4, 31), 5.0, dtype=dtype, device=DEV)
        args, named = c.args()
        out = bm.cache_attention(*args, **named, out=wide[..., 3:27])
        assert out.data_ptr() == wide[..., 3:27].data_ptr()
        assert torch.equal(wide[mine][..., 3:27], got[mine])
        assert bool((wide[~mine.to(DEV)] == 5).all())
        assert bool((wide[..., :3] == 5).all()) and bool((wide[..., 27:] == 5).all())


def test_attention_without_sequences_or_tokens():
    c = Case([2], [9], 4, 2, 1, 16, 16, torch.float32)
    (q, k, v, table, lengths), _ = c.args()
    none = lengths[:0]
    got = bm.cache_attention(q, k, v, table[:0], none, starts=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert got.shape == (2, 2, 16) and not bool(got.any())
    assert bm.cache_attention(q[:0], k, v, table[:0], none).shape == (0, 2, 16)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert bm.cache_attention(q[:0], k, v, table, lengths, starts=zero).shape == (0, 2, 16)
    # caches of no pages, and tables of no columns
    args = q, k[:0], v[:0]
    starts = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    assert not bool(bm.cache_attention(*args, table, lengths, starts=starts).any())
    assert not bool(bm.cache_attention(q, k, v, table[:, :0], lengths, starts=starts).any())


@pytest.mark.parametrize("narrow", ["no", "row"])
@pytest.mark.parametrize("tokens", [2, 40])
def test_attention_skips_wrong_pages_and_numbers(tokens, narrow):
    """Pages out of range are not seen; lengths past the table end with it; rows that no sequence
    can have are not read or written."""
    dtype = torch.bfloat16
    c = Case([tokens, tokens], [90, 200], 16, 4, 2, 64, 64, dtype, narrow)
    c.table[0, 2], c.table[0, 4], c.table[1, 0], c.table[1, 7] = -1, 2 ** 31 - 1, c.k.shape[0], -2 ** 31
    c.check()
    (q, k, v, table, _), named = c.args()
    for lengths, starts in (([10 ** 9, 2 ** 31 - 1], None), ([-5, -2 ** 31], None),
                            ([90, 200], [0, 2 ** 31 - 1, 5]), ([90, 200], [-2 ** 31, -5, 10 ** 6]),
                            ([90, 200], [2 * tokens, tokens, 0])):
        named["starts"] = c.starts.to(DEV) if starts is None else \
            torch.tensor(starts, dtype=torch.int32, device=DEV)
        out = torch.full((2 * tokens, 6, 64), 7.0, dtype=dtype, device=DEV)
        bm.cache_attention(q, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=DEV),
                           **named, out=out[:, 1:5])
        assert bool((out[:, 0] == 7).all()) and bool((out[:, 5] == 7).all())
        if starts is None and lengths[0] < 0:
            assert not bool(out[:, 1:5].any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(4, 2, 64, 64, 3), (4, 1, 128, 104, 30), (8, 2, 96, 96, 70), (2, 1, 512, 300, 5),
                                   (4, 2, 256, 256, 40)],
                         ids=str)
def test_numbers_that_are_none_reach_only_those_that_see_them(shape, dtype):
    """A NaN or an infinity in a value or a key shows in the rows that see its place, and in no other:
    here in the middle of a chunk, where some tokens of a tile see it and others do not."""
    q_heads, heads, dim, v_dim, n = shape
    length, page = 4 * n + 50, 16
    for window in (0, n // 2 + 1):
        c = Case([n], [length], page, q_heads, heads, dim, v_dim, dtype, window=window, seed=5)
        args, named = c.args()
        clean = bm.cache_attention(*args, **named)
        for back, what in ((0, NAN), (n // 2, math.inf), (n - 1, NAN), (n + 3, -math.inf)):
            at = length - 1 - back
            home = int(c.table[0, at // page]), at % page
            place = torch.arange(length - n, length)
            sees = (place >= at) & ((place < at + window) if window else True)
            k, v = args[1].clone(), args[2].clone()
            v[home][0, v_dim // 2] = what
            got = bm.cache_attention(args[0], k, v, *args[3:], **named)
            group = q_heads // heads
            odd = ~got.isfinite().cpu()
            want = torch.zeros_like(odd)
            want[sees, :group, v_dim // 2] = True
            assert torch.equal(odd, want)
            # rows next to it may take another way to the same sums
            u = _u(dtype)
            off = (got.double() - clean.double()).abs()[~odd.to(DEV)]
            size = clean.double().abs().amax()
            assert bool((off <= (4 * u + 4 * length * U32) * max(1.0, float(size)) * 4).all())
            k[home][0] = NAN
            got = bm.cache_attention(args[0], k, args[2], *args[3:], **named).isfinite().cpu()
            assert bool(got[~sees].all()) and bool(got[:, group:].all())
            assert not bool(got[sees, :group].any())


def test_attention_of_special_scores():
    """Scores of minus infinity weigh nothing, alone they leave zeros; plus infinity is no number."""
    for dtype in TYPES:
        q = torch.ones(3, 1, 16, dtype=dtype, device=DEV)
        k = torch.zeros(3, 4, 1, 16, dtype=dtype, device=DEV)
        v = torch.arange(12, device=DEV).to(dtype).reshape(3, 4, 1, 1).expand(3, 4, 1, 16).contiguous()
        k[0, :, 0, 3] = -math.inf
        k[1, 1, 0, 2] = -math.inf
        k[2, 2, 0, 1] = math.inf
        table = torch.arange(3, dtype=torch.int32, device=DEV)[:, None]
        lengths = torch.tensor([4, 3, 4], dtype=torch.int32, device=DEV)
        got = bm.cache_attention(q, k, v, table, lengths).float().cpu()
        assert not bool(got[0].any()) and bool((got[1] == 5.0).all()) and bool(got[2].isnan().all())


def test_attention_scale_and_large_scores():
    for dtype in TYPES:
        c = Case([4, 1], [100, 300], 16, 4, 2, 64, 64, dtype, spread=6.0)
        c.check()
        c.check(scale=0.5)
        c.check(scale=2.0 ** -10)


def test_small_weights_are_not_lost():
    """One key of weight 1 and many of 2^-26 of it, which together are a tenth of a percent."""
    n, dtype = 70000, torch.float16
    q = torch.zeros(1, 1, 16, dtype=dtype, device=DEV)
    q[..., 0] = 1.0
    k = torch.zeros(n // 1000, 1000, 1, 16, dtype=dtype, device=DEV)
    k[..., 0] = -26.0 * math.log(2.0)
    v = torch.ones_like(k)
    k[0, 0, 0, 0] = 0.0
    v[0, 0] = 0.0
    table = torch.arange(n // 1000, dtype=torch.int32, device=DEV)[None]
    got = float(bm.cache_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                                   scale=1.0)[0, 0, 0])
    w = math.exp(float(k[0, 1, 0, 0]))
    want = w * (n - 1) / (1 + w * (n - 1))
    # weights below the type's normal numbers keep 5 bits, v and the result half a step each
    assert abs(got - want) <= want * (2.0 ** -5 + 2.0 ** -9)


def test_attention_past_32_bits():
    """Pages whose offsets pass 32 bits, in elements and in bytes."""
    page, step = 16, (1 << 31) // 2 + 8 * 1024
    big = torch.zeros(3 * step, dtype=torch.float16, device=DEV)
    kc = big.as_strided((3, page, 2, 64), (step, 128, 64, 1))
    vc = big.as_strided((3, page, 2, 64), (step, 128, 64, 1), page * 128)
    c = Case([1, 2], [16, 40], page, 4, 2, 64, 64, torch.float16)
    (q, k, v, table, lengths), named = c.args()
    want = bm.cache_attention(q, k, v, table, lengths, **named)
    small = torch.tensor([[2, 0, 0], [1, 0, 2]], dtype=torch.int32, device=DEV)
    for s, n in ((0, 1), (1, 2)):
        for i in range(n):
            kc[small[s, i].long()], vc[small[s, i].long()] = k[table[s, i].long()], v[table[s, i].long()]
    # the second sequence's third page is the first one's
    lengths = torch.tensor([16, 32], dtype=torch.int32, device=DEV)
    got = bm.cache_attention(q, kc, vc, small, lengths, **named)
    want = bm.cache_attention(q, k, v, table, lengths, **named)
    assert torch.equal(got, want)
    out = big.as_strided((3, 4, 64), (step, 64, 1), 8192)
    bm.cache_attention(q, k, v, table, lengths, **named, out=out)
    assert torch.equal(out, want)


def test_long_and_short_sequences_together():
    """A long sequence among short ones, cut into many parts, against parts of the same made by hand."""
    g = torch.Generator(device=DEV).manual_seed(3)
    page, lengths = 64, [50000, 3, 700, 1]
    need = [(n + page - 1) // page for n in lengths]
    k, v = (torch.randn(sum(need), page, 2, 128, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.full((4, need[0]), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.arange(at, at + n, dtype=torch.int32, device=DEV)
        at += n
    q = torch.randn(4, 16, 128, device=DEV, generator=g).to(torch.bfloat16)
    got = bm.cache_attention(q, k, v, table, torch.tensor(lengths, dtype=torch.int32, device=DEV))
    for s, n in enumerate(lengths):
        ks, vs = (x[table[s, :need[s]].long()].flatten(0, 1)[:n].double() for x in (k, v))
        for h in range(16):
            w = torch.softmax(ks[:, h // 8] @ q[s, h].double() / 128 ** 0.5, dim=0)
            want, size = w @ vs[:, h // 8], w @ vs[:, h // 8].abs()
            off = (got[s, h].double() - want).abs()
            # weights and result half a step each, the scores' and the sums' chains in 32 bits
            assert bool((off <= size * (2.0 ** -8 + 2.0 ** -11) + 2.0 ** -8 * want.abs()).all())


def test_the_results_are_the_same_each_time():
    for new, lengths in (([1] * 6, [1, 900, 33, 2000, 5, 64]), ([50, 3], [700, 64])):
        c = Case(new, lengths, 16, 8, 2, 128, 128, torch.bfloat16)
        args, named = c.args()
        first = bm.cache_attention(*args, **named)
        assert all(torch.equal(first, bm.cache_attention(*args, **named)) for _ in range(3))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new", [3, 130])
def test_scales_of_values_in_the_hundreds(new, dtype):
    """A weight times its value's scale fits the type while scores rise along the keys."""
    c = Case([new], [400], 16, 4, 1, 64, 64, dtype, "row")
    c.v = (c.v.float() / 64).to(F8)
    c.scales = c.scales[0], 400.0 + 2000 * (c.scales[1] - 0.01)
    at = torch.arange(400)
    rise = torch.zeros_like(c.scales[0])
    rise[c.table[0, at // 16].long(), at % 16] = (at / 400.0)[:, None]
    c.scales = c.scales[0] * rise, c.scales[1]
    assert 450 < float(c.scales[1].max()) < 500
    got = c.check()
    assert bool(got.isfinite().all())


@pytest.mark.parametrize("tokens", [1, 40])
def test_more_sequences_than_lanes(tokens):
    """150 sequences, some of them empty, without new tokens or shorter than their new tokens."""
    g = _gen(11)
    lengths = (torch.rand(150, generator=g) ** 4 * 700).long().tolist()
    new = [0 if i % 13 == 5 else min(tokens, i + 1) for i in range(150)]
    Case(new, lengths, 16, 4, 2, 64, 64, torch.bfloat16).check()
    Case(new[:70], lengths[:70], 16, 4, 2, 64, 64, torch.float32).check()


def test_tables_of_more_places_than_31_bits_count():
    """A wide table of few pages in use: the number of parts that it could make needs 64 bits."""
    page, width, batch = 1 << 16, 1 << 15, 300
    c = Case([1] * batch, [5 + i % 7 for i in range(batch)], 16, 2, 1, 64, 64, torch.bfloat16)
    (q, k, v, table, _), named = c.args()
    lengths = torch.tensor([5 + i % 2 for i in range(batch)], dtype=torch.int32, device=DEV)
    two = torch.arange(batch, device=DEV) % 2
    wide = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    wide[:, 0] = two
    pools = []
    for x in (k, v):
        pools.append(torch.zeros(2, page, 1, 64, dtype=torch.bfloat16, device=DEV))
        pools[-1][:, :16] = x[table[:2, 0].long()]
    table[:, 0] = table[two, 0]
    want = bm.cache_attention(q, k, v, table, lengths, **named)
    got = bm.cache_attention(q, *pools, wide, lengths, **named)
    assert torch.equal(got, want) and bool(got.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", [
    ([1, 2], [500, 90], 16, 64, 1, 64, 64, 0), ([40], [170], 16, 4, 1, 36, 44, 0),
    ([90, 2], [500, 3], 16, 4, 2, 100, 84, 77), ([80], [400], 128, 6, 2, 200, 256, 0),
    ([65, 65], [65, 1000], 1, 2, 2, 8, 17, 0), ([5], [5], 16, 3, 1, 128, 128, 2)], ids=str)
def test_attention_of_other_shapes(case, dtype):
    """Rows of no multiple of 16 bytes in tiles of many rows, groups past a tile, pages of one place."""
    new, lengths, page, q_heads, heads, dim, v_dim, window = case
    for narrow in ("no", "row"):
        Case(new, lengths, page, q_heads, heads, dim, v_dim, dtype, narrow, window=window, before=2,
             behind=3).check()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("narrow", ["no", "row"])
@pytest.mark.parametrize("width", [3, 1 << 13])
def test_attention_in_shares_of_many_rows(width, narrow, dtype):
    """Tiles of 128 rows whose keys are cut into shares, as by tables that are wide, and not."""
    for new, lengths in (([60, 33, 1, 0], [700, 40, 64, 5]), ([70], [900]), ([5] * 70, list(range(5, 215, 3)))):
        c = Case(new, lengths, 16, 8, 2, 128, 96, dtype, narrow, behind=1)
        args, named = c.args()
        table = torch.full((len(new), c.table.shape[1] + width), -1, dtype=torch.int32, device=DEV)
        table[:, :c.table.shape[1]] = c.table
        want, slack = c.want(128 ** -0.5)
        _within(bm.cache_attention(*args[:3], table, args[4], **named), want, slack, dtype)


@pytest.mark.parametrize("sequences", [3, 600])
def test_attention_with_a_table_of_no_pages(sequences):
    """No sequence has a place that could be seen: zeros, and rows of nobody left as they are."""
    table = torch.zeros(sequences, 0, dtype=torch.int32, device=DEV)
    lengths = torch.full((sequences,), 40, dtype=torch.int32, device=DEV)
    starts = 2 + 3 * torch.arange(sequences + 1, dtype=torch.int32, device=DEV)
    for dtype in TYPES:
        q = torch.randn(3 * sequences + 4, 40, 64, device=DEV).to(dtype)
        pools = [torch.full((2, 16, 2, 64), NAN, device=DEV).to(dtype) for _ in range(2)]
        out = torch.full((3 * sequences + 4, 40, 64), 7.0, device=DEV).to(dtype)
        bm.cache_attention(q, *pools, table, lengths, starts=starts, out=out)
        assert bool((out[:2] == 7).all()) and bool((out[-2:] == 7).all()) and not bool(out[2:-2].any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,width", [(1, 0), (6, 0), (6, 300)])
def test_attention_of_hundreds_of_short_sequences(new, width, dtype):
    """More sequences than tiles are looked for in, shorter than a tile of keys; of a wide table too."""
    c = Case([new] * 600, [new + i % 97 for i in range(600)], 16, 6, 2, 64, 64, dtype)
    args, named = c.args()
    table = torch.full((600, c.table.shape[1] + width), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table
    want, slack = c.want(64 ** -0.5)
    _within(bm.cache_attention(*args[:3], table, args[4], **named), want, slack, dtype)


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("tokens", [2, 100])
def test_attention_over_a_cache_without_pages(tokens, page):
    """Every entry of the table is out of range, and there may be no scales at all."""
    q = torch.randn(tokens, 4, 64, device=DEV)
    table = torch.zeros(1, 3, dtype=torch.int32, device=DEV)
    where = dict(starts=torch.tensor([0, tokens], dtype=torch.int32, device=DEV))
    lengths = torch.tensor([3 * page], dtype=torch.int32, device=DEV)
    for dtype in TYPES:
        for kind in (dtype, F8):
            pools = [torch.zeros(0, page, 2, 64, dtype=kind, device=DEV) for _ in range(2)]
            scales = dict(zip(("k_scale", "v_scale"), (torch.zeros(0, page, 2, device=DEV) for _ in range(2)))) \
                if kind == F8 else {}
            got = bm.cache_attention(q.to(dtype), *pools, table, lengths, **where, **scales)
            assert got.shape == (tokens, 4, 64) and not bool(got.any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("narrow", ["no", "head", "row"])
@pytest.mark.parametrize("dim,v_dim", [(64, 60), (80, 96), (96, 65), (72, 128), (128, 112), (130, 256), (260, 512)])
def test_attention_of_each_padded_size(dim, v_dim, narrow, dtype):
    """Heads that are padded to each of the sizes, in shares of few rows and of many."""
    for new, lengths in (([1, 3], [70, 333]), ([40, 1], [150, 9]), ([90], [290])):
        Case(new, lengths, 16, 6, 2, dim, v_dim, dtype, narrow).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,v_dim,narrow", [(96, 96, "no"), (80, 96, "row"), (128, 70, "head"), (250, 256, "no")])
def test_attention_of_whole_tiles(dim, v_dim, narrow, dtype):
    """As many rows as make a workgroup a tile: of 16 rows in 32 bits, of 128 in 16."""
    if dtype == torch.float32:
        Case([130, 1, 200], [180, 40, 200], 16, 128, 32, dim, v_dim, dtype, narrow).check()
    else:
        Case([20] * 63 + [50], [20 + 3 * i for i in range(63)] + [300], 16, 128, 32, dim, v_dim, dtype,
             narrow).check()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    cases = [Case([1] * 6, [1, 900, 33, 2000, 5, 64], 16, 8, 2, 128, 128, torch.bfloat16),
             Case([50, 3], [700, 64], 16, 8, 2, 128, 128, torch.bfloat16, seed=1)]
    work = [c.args() for c in cases]
    want = [bm.cache_attention(*a, **named) for a, named in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [bm.cache_attention(*a, **named, stream=s) for (a, named), s in zip(work, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# --------------------------------------------------------------------------
# The cache in 8 bits
# --------------------------------------------------------------------------

def _freqs(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)


def _turned(x, angle, interleaved, scale=1.0):
    """x [T, H, D] turned by angle [T, P], and what 32-bit arithmetic may be off by:
    cosine and sine by 6 roundings, the scale, two products and their sum by 5 more, and the 64-bit
    angle by 4 2^-53 of itself on either side."""
    x, pairs = x.double(), angle.shape[-1]
    c, s = torch.cos(angle)[:, None] * scale, torch.sin(angle)[:, None] * scale
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out, slack = x.clone(), torch.zeros_like(x)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    each = (x[..., lo].abs() + x[..., hi].abs()) * abs(scale) * (
        11 * U32 + 2.0 ** -50 * angle.abs()[:, None])
    slack[..., lo], slack[..., hi] = each, each
    return out, slack


class Append:
    """New tokens of several sequences, some of them padding; caches filled before."""

    def __init__(self, tokens, batch, page, heads, dim, v_dim, dtype, first=False, seed=0):
        g = _gen(seed + tokens + dim)
        self.page, self.dtype, self.first = page, dtype, first
        self.sequences = torch.randint(0, batch, (tokens,), generator=g).sort().values
        begin = torch.searchsorted(self.sequences, torch.arange(batch))
        held = torch.randint(0, 3 * page, (batch,), generator=g)
        self.positions = held[self.sequences] + torch.arange(tokens) - begin[self.sequences]
        width = int(self.positions.max()) // page + 2
        self.pages = batch * width + 3
        self.table = torch.randperm(self.pages, generator=g)[:batch * width].reshape(batch, width).to(torch.int32)
        self.k = torch.randn(tokens, heads, dim, generator=g).to(dtype)
        self.v = torch.randn(tokens, heads, v_dim, generator=g).to(dtype)
        shape = (self.pages, page, heads)
        self.caches = [torch.randn(*shape, d, generator=g).to(F8) for d in (dim, v_dim)]
        self.scales = [torch.rand(*shape, generator=g) for _ in range(2)]

    def home(self, t):
        s, p = int(self.sequences[t]), int(self.positions[t])
        return int(self.table[s, p // self.page]), p % self.page

    def on(self, x):
        if self.first:
            return x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        return x.to(DEV)

    def device(self):
        return ([self.on(x) for x in (*self.caches, *self.scales)],
                (self.table.to(DEV), self.positions.to(DEV)),
                dict(sequences=self.sequences.to(torch.int32).to(DEV)))


def _check_stored(cache, scales, c, which, x, slack):
    """What was stored of x [T, H, D] (64 bits, off by slack): scales, values, and nothing else."""
    before, scales_before = c.caches[which], c.scales[which]
    touched = torch.zeros(before.shape[:2], dtype=torch.bool)
    cache, scales = cache.cpu(), scales.cpu()
    for t in range(x.shape[0]):
        home = c.home(t)
        touched[home] = True
        most = x[t].abs().amax(-1)
        scale = scales[home].double()
        want = torch.where(most > 0, most / 448, 1.0)
        # the largest is off by its own slack, the quotient rounded once
        assert bool(((scale - want).abs() <= slack[t].amax(-1) / 448 + 2 * U32 * want).all())
        y = x[t] / scale[:, None]
        off = (cache[home].double() - y.clamp(-448, 448)).abs()
        room = slack[t] / scale[:, None] + 2 * U32 * y.abs()
        # half a step of 3 bits after the first, 2^-10 among the subnormals
        assert bool((off <= room * (1 + 2.0 ** -4) + torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10))).all())
    assert torch.equal(cache.view(torch.uint8)[~touched], before.view(torch.uint8)[~touched])
    assert torch.equal(scales[~touched], scales_before[~touched])


QUANTIZE = [  # tokens, sequences, page, heads, size of k, of v, pairs, interleaved, heads first
    (1, 1, 1, 1, 1, 1, 0, False, False), (3, 2, 4, 2, 2, 3, 1, False, False), (5, 5, 16, 2, 64, 64, 32, False, False),
    (64, 7, 16, 8, 128, 128, 64, False, True), (100, 3, 7, 2, 96, 40, 24, True, False),
    (33, 4, 32, 3, 20, 7, 3, False, False), (17, 2, 5, 2, 130, 512, 65, True, True), (17, 2, 5, 2, 130, 33, 65, False, True),
    (40, 4, 16, 4, 192, 128, 20, False, False), (9, 2, 3, 3, 512, 9, 256, False, False), (25, 1, 1, 2, 66, 9, 0, False, False),
    (5000, 9, 16, 2, 64, 64, 16, False, True), (4300, 3, 64, 1, 24, 16, 8, True, False)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", QUANTIZE, ids=str)
def test_quantize(case, dtype):
    tokens, batch, page, heads, dim, v_dim, pairs, interleaved, first = case
    c = Append(tokens, batch, page, heads, dim, v_dim, dtype, first)
    pools, where, named = c.device()
    wide = torch.zeros(tokens, 5 * heads, max(dim, v_dim) + 1, dtype=dtype, device=DEV)
    k, v = wide[:, :heads, :dim], wide[:, heads:2 * heads, :v_dim]
    k.copy_(c.k), v.copy_(c.v)
    turned, slack = c.k.double(), torch.zeros(c.k.shape, dtype=torch.float64)
    if pairs:
        q = torch.randn(tokens, 3 * heads, dim, generator=_gen(7)).to(dtype)
        angle = c.positions.double()[:, None] * _freqs(pairs)
        turned, slack = _turned(c.k, angle, interleaved, 0.75)
        want, off = _turned(q, angle, interleaved, 0.75)
        how = dict(freqs=_freqs(pairs).to(DEV), interleaved=interleaved, scale=0.75)
        got = bm.cache_quantize(k, v, *pools, *where, **named, **how, q=q.to(DEV))
        _within(got, want, off, dtype)
        mine = wide[:, 2 * heads:, :dim]
        mine.copy_(q)
        again = [x.clone() for x in pools]
        assert bm.cache_quantize(k, v, *again, *where, **named, **how, q=mine, q_out=mine) is mine
        assert torch.equal(mine, got) and all(torch.equal(a.float(), b.float()) for a, b in zip(again, pools))
    else:
        assert bm.cache_quantize(k, v, *pools, *where, **named) is None
    _check_stored(pools[0], pools[2], c, 0, turned, slack)
    _check_stored(pools[1], pools[3], c, 1, c.v.double(), torch.zeros(c.v.shape, dtype=torch.float64))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_values(dtype):
    """Zeros, infinities, NaN and the smallest numbers; rows without a place store nothing."""
    k = torch.zeros(8, 1, 16).to(dtype)
    k[1, 0, 3], k[1, 0, 4], k[1, 0, 5] = 2.0, math.inf, -math.inf
    k[2, 0, 1], k[2, 0, 2] = NAN, -7.0
    k[3, 0, 0] = math.inf
    k[4] = torch.finfo(dtype).tiny
    k[5] = _least(dtype) * 2  # the smallest of all
    k[6], k[7] = 3.0, 4.0
    pools = [torch.full((4, 2, 1, 16), 9.0).to(F8).to(DEV) for _ in range(2)]
    scales = [torch.full((4, 2, 1), 9.0, device=DEV) for _ in range(2)]
    table = torch.tensor([[0, 1, 2], [3, -1, 4]], dtype=torch.int32, device=DEV)
    sequences = torch.tensor([0, 0, 0, 0, 0, 0, 1, 1], dtype=torch.int32, device=DEV)
    positions = torch.tensor([0, 1, 2, 3, 4, 5, 2, 5], device=DEV)  # the last two: no such page
    bm.cache_quantize(k.to(DEV), k.to(DEV), *pools, *scales, table, positions, sequences=sequences)
    for cache, scale in zip(pools, scales):
        cache, scale = cache.cpu().float(), scale.cpu()
        assert scale[0].reshape(-1).tolist() == [1.0, float(torch.tensor(2.0) / 448)]
        assert not bool(cache[0, 0].any()) and cache[0, 1, 0, 3:6].tolist() == [448.0, 448.0, -448.0]
        assert bool(cache[1, 0, 0, 1].isnan()) and cache[1, 0, 0, 2] == -448.0
        assert scale[1, 0, 0] == torch.tensor(7.0) / 448
        assert scale[1, 1, 0] == 1.0 and cache[1, 1, 0, 0] == 448.0
        least = 2.0 ** -126
        for i, x in ((0, torch.finfo(dtype).tiny), (1, _least(dtype) * 2)):
            assert scale[2, i, 0] == max(torch.tensor(x) / 448, torch.tensor(least))
            back = cache[2, i, 0].double() * float(scale[2, i, 0])
            assert bool(((back - x).abs() <= max(2.0 ** -4 * x, least * 2.0 ** -10)).all())
        assert bool((cache[3] == 9.0).all()) and bool((scale[3] == 9.0).all())


READ = [  # tokens, sequences, page, heads, size of k, of v, heads first
    (1, 1, 1, 1, 1, 1, False), (7, 2, 4, 3, 5, 9, False), (300, 5, 16, 4, 96, 64, True), (65, 3, 7, 2, 130, 512, False),
    (2100, 4, 64, 8, 128, 128, False), (17000, 3, 16, 1, 64, 24, True), (40, 1, 5, 130, 8, 8, False)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("narrow", ["no", "one", "head", "row"])
@pytest.mark.parametrize("case", READ, ids=str)
def test_read(case, narrow, dtype):
    tokens, batch, page, heads, dim, v_dim, first = case
    c = Append(tokens, batch, page, heads, dim, v_dim, dtype, first)
    g = _gen(1)
    if narrow == "no":
        c.caches = [torch.randn(x.shape, generator=g).to(dtype) for x in c.caches]
    scales = {"no": [None, None], "one": [torch.rand(1, generator=g) for _ in range(2)],
              "head": [torch.rand(heads, generator=g) for _ in range(2)], "row": c.scales}[narrow]
    order = torch.randperm(tokens, generator=g)
    sequences, positions = c.sequences[order].to(torch.int32), c.positions[order]
    sequences[::7] = -1
    page_of = c.table[sequences.long().clamp(min=0), positions // page].long()
    wide = torch.full((tokens, 2 * heads, max(dim, v_dim) + 2), 5.0, dtype=dtype, device=DEV)
    outs = wide[:, :heads, 1:dim + 1], wide[:, heads:, 1:v_dim + 1]
    on = [None if s is None else c.on(s) if s.dim() == 3 else s.to(DEV) for s in scales]
    args = ([c.on(x) for x in c.caches], c.table.to(DEV), positions.to(DEV))
    named = dict(sequences=sequences.to(DEV), k_scale=on[0], v_scale=on[1], dtype=dtype)
    got = bm.cache_read(*args[0], *args[1:], **named)
    again = bm.cache_read(*args[0], *args[1:], **named, k_out=outs[0], v_out=outs[1])
    for i, x in enumerate(got):
        want = c.caches[i][page_of, positions % page].float()
        if scales[i] is not None:
            s = scales[i][page_of, positions % page] if narrow == "row" else scales[i].expand(heads)
            want = want * s[..., None]
        want = torch.where((sequences >= 0)[:, None, None], want, 0.0).to(dtype)
        assert torch.equal(x.cpu(), want)  # one product in 32 bits, rounded once
        assert torch.equal(again[i], x)
    wide[:, :heads, 1:dim + 1] = 5.0
    wide[:, heads:, 1:v_dim + 1] = 5.0
    assert bool((wide == 5).all())


def test_cache_attended_and_read_as_it_was_written():
    """Appended, attended and read back: a prompt in two chunks, then single tokens."""
    for dtype in (torch.bfloat16, torch.float16):
        for narrow in (False, True):
            _serve(dtype, narrow)


def _serve(dtype, narrow):
    heads, q_heads, dim, page, batch = 2, 8, 64, 16, 3
    lengths = [70, 5, 33]
    g = _gen(11)
    table = torch.randperm(24, generator=g).to(torch.int32).reshape(3, 8).to(DEV)
    kind = F8 if narrow else dtype
    caches = [torch.zeros(24, page, heads, dim, dtype=dtype).to(kind).to(DEV) for _ in range(2)]
    scales = [torch.zeros(24, page, heads, device=DEV) for _ in range(2)] if narrow else [None, None]
    q, k, v = (torch.randn(batch, 80, h, dim, generator=g).to(dtype).to(DEV) for h in (q_heads, heads, heads))
    freqs, done = _freqs(32).to(DEV), [0, 0, 0]
    turned_q, turned_k = bm.rotary((q, k), torch.arange(80, device=DEV).expand(3, 80).contiguous(), freqs)
    for step in [[n // 2 for n in lengths], [n - n // 2 for n in lengths], [1, 1, 1], [1, 1, 1]]:
        rows = [(s, done[s] + i) for s in range(batch) for i in range(step[s])]
        s, p = torch.tensor(rows, device=DEV).t().contiguous()
        ends = [done[b] + step[b] for b in range(batch)]
        args = dict(sequences=s.to(torch.int32), freqs=freqs, q=q[s, p])
        if narrow:
            mine = bm.cache_quantize(k[s, p], v[s, p], *caches, *scales, table, p, **args)
        else:
            mine = bm.cache_append(k[s, p], v[s, p], *caches, table, p, **args)
        starts = torch.tensor([0] + [sum(step[:b + 1]) for b in range(batch)], dtype=torch.int32, device=DEV)
        now = torch.tensor(ends, dtype=torch.int32, device=DEV)
        out = bm.cache_attention(mine, *caches, table, now, starts=starts, k_scale=scales[0], v_scale=scales[1])
        every = [(b, i) for b in range(batch) for i in range(ends[b])]
        es, ep = torch.tensor(every, device=DEV).t().contiguous()
        kr, vr = bm.cache_read(*caches, table, ep, sequences=es.to(torch.int32), k_scale=scales[0],
                               v_scale=scales[1], dtype=torch.float32 if narrow else dtype)
        step_of = 2.0 ** -4 if narrow else 0.0
        assert bool(((kr.double() - turned_k[es, ep].double()).abs() <=
                     step_of * kr.double().abs() * 1.1 + 2.0 ** -9 * narrow + 3 * _u(dtype) * kr.double().abs()).all())
        if not narrow:
            assert torch.equal(vr, v[es, ep])
        for t, (b, i) in enumerate(rows):
            at = (es == b) & (ep <= i)
            a = torch.einsum("hd,khd->hk", mine[t].double(), kr[at].double().repeat_interleave(4, 1))
            w = torch.softmax(a / dim ** 0.5, dim=1)
            values = vr[at].double().repeat_interleave(4, 1)
            want, size = torch.einsum("hk,khd->hd", w, values), torch.einsum("hk,khd->hd", w, values.abs())
            off = (out[t].double() - want).abs()
            # weights and result half a step each; chains of 64 and of 80 in 32 bits
            assert bool((off <= size * (_u(dtype) + 1000 * U32) + _u(dtype) * want.abs() + _least(dtype)).all())
        done = ends


# --------------------------------------------------------------------------
# The balance of a router
# --------------------------------------------------------------------------

def _balance_case(tokens, choices, experts, dtype, masked, seed=0):
    g = _gen(seed + tokens + experts)
    logits = (torch.randn(tokens, experts, generator=g) * 2).to(dtype)
    chosen = torch.randint(-1, experts + 1, (tokens, choices), generator=g)
    mask = torch.rand(tokens, generator=g) >= masked if masked else None
    return logits, chosen, mask


def _balance(logits, chosen, mask, grad=1.0):
    """Loss, counts and gradient from the definition, in 64 bits, and what the gradient may be off by."""
    x, e = logits.double(), logits.shape[1]
    on = torch.ones(len(x), dtype=torch.bool) if mask is None else mask
    n, kept = int(on.sum()), chosen[on].reshape(-1)
    counts = torch.bincount(kept[(kept >= 0) & (kept < e)], minlength=e)
    if n == 0:
        return 0.0, counts, torch.zeros_like(x), torch.zeros_like(x)
    p = torch.softmax(x, dim=1)
    slope = counts.double() * e / (n * n * chosen.shape[1])
    loss = float((slope * p[on].sum(0)).sum())
    dot = (p * slope).sum(1, keepdim=True)
    size = grad * p * (slope + dot)
    # exponents of magnitude x, their sums over the experts and the products
    room = (e + 20 + 2 * (x.abs() + x.abs().amax(1, keepdim=True))) * U32
    return loss, counts, torch.where(on[:, None], grad * p * (slope - dot), 0.0), \
        torch.where(on[:, None], size * 2 * room, 0.0)


BALANCE = [  # tokens, choices, experts, masked
    (1, 1, 1, 0.0), (1, 2, 3, 0.0), (5, 1, 7, 0.5), (33, 4, 8, 0.0), (257, 4, 60, 0.1), (100, 8, 64, 0.0), (63, 2, 65, 0.2),
    (300, 10, 256, 0.3), (77, 3, 257, 0.0), (50, 6, 1000, 0.1), (40, 8, 2048, 0.0), (19, 1024, 13, 0.0),
    (20000, 8, 128, 0.05), (9000, 2, 5, 0.0), (4097, 4, 513, 1.0), (3000, 7, 2041, 0.4),
    (1024, 3, 32, 0.1), (1025, 3, 31, 0.0), (16, 5, 2048, 0.0), (17, 5, 2048, 0.2), (1023, 1, 2, 0.3)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", BALANCE, ids=str)
def test_balance(case, dtype):
    logits, chosen, mask = _balance_case(*case[:3], dtype, case[3])
    loss, counts, grad, slack = _balance(logits, chosen, mask, 0.5)
    wide = torch.full((len(logits), logits.shape[1] + 3), NAN, dtype=dtype, device=DEV)
    x = wide[:, 1:logits.shape[1] + 1]
    x.copy_(logits)
    if mask is not None:  # what the mask leaves out does not matter
        x[(~mask).to(DEV)] = NAN
    on = None if mask is None else mask.to(DEV)
    got = bm.expert_balance(x, chosen.to(DEV), mask=on)
    assert torch.equal(got.counts.cpu(), counts.to(torch.int32))
    # sums of positive terms: a chain over a workgroup's tokens at most, exponents as above
    assert abs(float(got.loss) - loss) <= loss * (len(logits) + logits.shape[1] + 60) * U32
    again = bm.expert_balance(x, chosen.to(torch.int32).to(DEV), mask=on)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    one = torch.full((), 0.5, device=DEV)
    out = torch.full((len(logits), logits.shape[1] + 2), 5.0, dtype=dtype, device=DEV)
    bm.expert_balance_backward(one, x, got.slopes, mask=on, out=out[:, 1:-1])
    _within(out[:, 1:-1], grad, slack, dtype)
    assert bool((out[:, 0] == 5).all()) and bool((out[:, -1] == 5).all())
    assert torch.equal(bm.expert_balance_backward(one, x, got.slopes, mask=on), out[:, 1:-1])


def test_balance_of_nothing():
    got = bm.expert_balance(torch.zeros(0, 9, device=DEV), torch.zeros(0, 2, dtype=torch.int64, device=DEV))
    assert float(got.loss) == 0 and not bool(got.counts.any()) and not bool(got.slopes.any())
    even = bm.expert_balance(torch.zeros(8, 4, device=DEV), torch.arange(16, device=DEV).reshape(8, 2) % 4)
    assert float(even.loss) == 1.0 and even.counts.tolist() == [4] * 4
    far = torch.tensor([[1 << 32, -(1 << 32)], [(1 << 62) + 1, 1]], device=DEV)
    assert bm.expert_balance(torch.zeros(2, 2, device=DEV), far).counts.tolist() == [0, 1]


def test_balance_gradient():
    """Through autograd, against differences of the loss and the formula's own gradient."""
    logits, chosen, mask = _balance_case(60, 4, 24, torch.float32, 0.2)
    x = logits.to(DEV).requires_grad_()
    got = bm.expert_balance(x, chosen.to(DEV), mask=mask.to(DEV))
    assert not got.counts.requires_grad and not got.slopes.requires_grad
    (3.0 * got.loss).backward()
    _, _, grad, slack = _balance(logits, chosen, mask, 3.0)
    _within(x.grad, grad, slack, torch.float32)
    # the loss is smooth: a step h leaves (h^2 / 2) of its second derivative, at most 2 of the loss
    step = torch.randn(logits.shape, generator=_gen(4)) * 2.0 ** -8
    up, down = (float(bm.expert_balance((logits + s * step).to(DEV), chosen.to(DEV), mask=mask.to(DEV)).loss)
                for s in (1, -1))
    want = float((grad / 3.0 * step.double()).sum())
    third = float(step.abs().max()) ** 3 * 10 * float(got.loss)
    assert abs((up - down) / 2 - want) <= third + 200 * U32 * float(got.loss)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y = logits.to(DEV).requires_grad_()
        again = bm.expert_balance(y, chosen.to(DEV))
        again.slopes.zero_()
        again.loss.backward()


# --------------------------------------------------------------------------
# Streams and graphs
# --------------------------------------------------------------------------

def _inputs(seed, batch=40):
    g = _gen(seed)
    bf, n = torch.bfloat16, 2 * batch
    lengths = torch.randint(2, 200, (batch,), generator=g)
    s = torch.arange(batch).repeat_interleave(2)
    return dict(q=torch.randn(n, 8, 64, generator=g).to(bf).to(DEV), k=torch.randn(n, 2, 64, generator=g).to(bf).to(DEV),
                v=torch.randn(n, 2, 64, generator=g).to(bf).to(DEV),
                caches=[torch.ones(batch * 13, 16, 2, 64, dtype=bf).to(F8).to(DEV) for _ in range(2)],
                scales=[torch.ones(batch * 13, 16, 2, device=DEV) for _ in range(2)],
                table=torch.randperm(batch * 13, generator=g).reshape(batch, 13).to(torch.int32).to(DEV),
                positions=(lengths[s] - 2 + torch.arange(n) % 2).to(DEV), sequences=s.to(torch.int32).to(DEV),
                lengths=lengths.to(torch.int32).to(DEV),
                starts=(2 * torch.arange(batch + 1)).to(torch.int32).to(DEV), freqs=_freqs(32).to(DEV),
                logits=torch.randn(3000, 64, generator=g).to(DEV),
                chosen=torch.randint(-1, 64, (3000, 4), generator=g).to(DEV),
                mask=(torch.rand(3000, generator=g) > 0.2).to(DEV), one=torch.ones((), device=DEV))


def _step(q, k, v, caches, scales, table, positions, sequences, lengths, starts, freqs, logits, chosen, mask, one,
          stream=None):
    turned = bm.cache_quantize(k, v, *caches, *scales, table, positions, sequences=sequences, freqs=freqs, q=q,
                               stream=stream)
    kw = dict(k_scale=scales[0], v_scale=scales[1], stream=stream)
    out = bm.cache_attention(turned, *caches, table, lengths, starts=starts, **kw)
    read = bm.cache_read(*caches, table, positions, sequences=sequences, dtype=torch.bfloat16, **kw)
    balance = bm.expert_balance(logits, chosen, mask=mask, stream=stream)
    grad = bm.expert_balance_backward(one, logits, balance.slopes, mask=mask, stream=stream)
    return [turned, out, *read, *balance, grad, *caches, *scales]


def _same(a, b):
    return all(torch.equal(p.float(), q.float()) for p, q in zip(a, b))


def test_on_another_stream():
    """Inputs made on the current stream just before, results read on it just after."""
    want = [t.clone() for t in _step(**_inputs(70))]
    for how in (torch.cuda.Stream(), int(torch.cuda.Stream().cuda_stream)):
        a = _inputs(70)
        x = a["q"].clone().reshape(-1, 512)
        for _ in range(20):  # keep the current stream busy ahead of the inputs
            x = torch.tanh(x @ torch.ones(512, 512, dtype=x.dtype, device=DEV))
        a["q"] = a["q"] + 0 * x.nan_to_num().reshape(a["q"].shape)
        got = _step(**a, stream=how)
        assert _same([t.clone() for t in got], want)


def test_in_a_graph():
    """Captured once, replayed on other inputs, with eager work in between; two graphs at once."""
    a, other = _inputs(71), _inputs(90)
    for x in (a, other):
        _step(**x)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph, x in zip(graphs, (a, other)):
        with torch.cuda.graph(graph):
            outs.append(_step(**x))
    wanted = [t.clone() for t in _step(**_inputs(90))]
    for seed in (72, 73, 74, 75):
        b = _inputs(seed)
        want = [t.clone() for t in _step(**b)]
        fresh = _inputs(seed)
        for name, t in fresh.items():
            for to, x in zip(a[name], t) if isinstance(t, list) else [(a[name], t)]:
                to.copy_(x)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert _same(outs[0], want), seed
        assert _same(outs[1], wanted), seed


@pytest.mark.parametrize("tokens", [40, 3000])
def test_a_balance_step_in_a_graph(tokens):
    """Loss and gradient captured together, in one workgroup and in two launches, replayed on other
    inputs with eager steps in between; no eager graph of the leaves is alive while it is captured."""
    def inputs(seed):
        logits, chosen, mask = _balance_case(tokens, 4, 64, torch.bfloat16, 0.2, seed)
        return [logits.to(DEV).requires_grad_(), chosen.to(DEV), mask.to(DEV)]

    def step(x, chosen, mask):
        got = bm.expert_balance(x, chosen, mask=mask)
        return [got.loss, got.counts, got.slopes, *torch.autograd.grad(got.loss * 0.5, x)]
    a = inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(*a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*a)
    for seed in (2, 3, 4):
        b = inputs(seed)
        want = [t.detach().clone() for t in step(*b)]
        with torch.no_grad():
            for t, u in zip(a, b):
                t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), seed


def test_in_place_results_count_for_autograd():
    a = _inputs(5)
    w = torch.ones((), device=DEV, requires_grad=True)
    writes = {
        "out": (torch.zeros(80, 8, 64, dtype=torch.bfloat16, device=DEV), lambda t: bm.cache_attention(
            a["q"], *a["caches"], a["table"], a["lengths"], starts=a["starts"], k_scale=a["scales"][0],
            v_scale=a["scales"][1], out=t)),
        "scales": (a["scales"][0].clone(), lambda t: bm.cache_quantize(
            a["k"], a["v"], *a["caches"], t, a["scales"][1], a["table"], a["positions"], sequences=a["sequences"])),
        "read": (torch.zeros(80, 2, 64, device=DEV), lambda t: bm.cache_read(
            *a["caches"], a["table"], a["positions"], sequences=a["sequences"], k_scale=a["scales"][0],
            v_scale=a["scales"][1], dtype=torch.float32, v_out=t)),
        "gradient": (torch.zeros(3000, 64, device=DEV), lambda t: bm.expert_balance_backward(
            a["one"], a["logits"], torch.ones(64, device=DEV), out=t))}
    for name, (t, call) in writes.items():
        loss = (t * w).sum()
        call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


# --------------------------------------------------------------------------
# The example
# --------------------------------------------------------------------------

def test_the_example_from_8_bits():
    """A layer served from a cache in 8 bits: finite, and the router's balance gradient among those
    that the training step compares (it raises where shapes or gradients are missing)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "sparse_layer.py")
    spec = importlib.util.spec_from_file_location("sparse_layer", path)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    device = torch.device(DEV)
    with torch.no_grad():
        most, middle = layer.serve(device, torch.bfloat16, 70, 3, narrow=True)
    assert math.isfinite(most) and middle <= most
    # as in the serving test: sums of at most 512 terms, each off by one rounding in 32 bits
    assert layer.train(device, 33) <= 512 * U32
