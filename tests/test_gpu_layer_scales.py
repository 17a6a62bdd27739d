"""GPU tests of the scales of caches in 8 bits that attention reads: those of places that are not
seen, of no and of other signs than the usual one, and of all magnitudes.

Tolerances are those of test_gpu_layer: a rounding to a type is off by at most half a step, a chain
of n 32-bit operations by n 2^-24 times the sum of the terms' magnitudes."""
import math

import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402
from test_gpu_layer import DEV, F8, NAN, TYPES, U32, Case, _gen, _least, _u, _within  # noqa: E402

pytestmark = pytest.mark.gpu


def _seen(c):
    """The places that some token sees, as [pages, places]."""
    seen = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for s, n in enumerate(c.new):
        first = max(0, c.lengths[s] - n - c.window + 1) if c.window else 0
        at = torch.arange(first, c.lengths[s]) if n else torch.arange(0)
        seen[c.table[s, at // c.page].long(), at % c.page] = True
    return seen


def _attend(c, k_scale, v_scale, k=None, v=None, scale=None):
    args, named = c.args()
    named.update(k_scale=c.on(k_scale), v_scale=c.on(v_scale))
    return bm.cache_attention(args[0], args[1] if k is None else c.on(k), args[2] if v is None else c.on(v),
                              *args[3:], scale=scale, **named)


# new, lengths, window: few rows in shares, many rows a sequence, and both with a window's begin
# inside a tile of keys
ROWS = [([1, 1], [300, 17], 100), ([3, 1], [200, 90], 33), ([30, 1], [150, 300], 0), ([130, 70], [400, 75], 77),
        ([130], [290], 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_scales_of_places_that_nobody_sees(case, what, dtype):
    """Pages of nobody, places behind a sequence's end and in front of a window: their scales, as
    their keys and values, may be anything."""
    new, lengths, window = case
    c = Case(new, lengths, 16, 6, 2, 64, 80, dtype, "row", window=window)
    want, slack = c.want(64 ** -0.5)
    seen = _seen(c)[..., None]
    scales = [torch.where(seen, s, what) for s in c.scales]
    _within(_attend(c, *scales), want, slack, dtype)
    k, v = (torch.where(seen[..., None], x.float(), NAN).to(F8) for x in (c.k, c.v))
    _within(_attend(c, *scales, k=k, v=v), want, slack, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(4, 2, 64, 64, 3), (8, 2, 96, 72, 30), (4, 2, 128, 104, 150), (4, 2, 256, 200, 80)], ids=str)
def test_a_scale_that_is_none_reaches_only_those_that_see_it(shape, dtype):
    """A NaN or an infinity for a scale in the middle of a chunk shows in the rows that see its place
    and in no other, also where another value is a NaN."""
    q_heads, heads, dim, v_dim, n = shape
    group, length, page = q_heads // heads, 2 * n + 50, 16
    for window in (0, n // 2 + 1):
        c = Case([n], [length], page, q_heads, heads, dim, v_dim, dtype, "row", window=window, seed=3)
        want, slack = c.want(dim ** -0.5)
        place = torch.arange(length - n, length)
        for back, what, which in ((0, NAN, 1), (n // 2, math.inf, 1), (n + 3, -math.inf, 1), (n - 1, NAN, 0)):
            for odd_value in (False, True):
                at = length - 1 - back
                home = int(c.table[0, at // page]), at % page
                sees = (place >= at) & ((place < at + window) if window else True)
                none = torch.zeros_like(want, dtype=torch.bool)
                none[sees, :group] = True
                scales, v = [s.clone() for s in c.scales], c.v.float()
                scales[which][home][0] = what
                if odd_value:  # of the last token's place, which only that token sees
                    v[int(c.table[0, (length - 1) // page]), (length - 1) % page, 1, 5] = NAN
                    none[n - 1, group:, 5] = True
                got = _attend(c, *scales, v=v.to(F8)).cpu()
                assert torch.equal(~got.isfinite(), none)
                _within(torch.where(none, 0, got), torch.where(none, 0, want), slack, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("narrow", ["one", "head", "row"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_scales_of_no_and_of_both_signs(case, narrow, dtype):
    """Scales of 0 and below are scales as others are, for one token and for many."""
    new, lengths, window = case
    for signs in ([0.0, 1.0, -1.0], [-1.0, 0.0, 0.0], [0.0, 0.0, 0.0]):
        c = Case(new, lengths, 16, 6, 3, 64, 80, dtype, narrow, window=window)
        k, v = c.scales
        by = torch.tensor(signs if narrow == "head" else signs[0])
        if narrow == "row":
            by = torch.tensor(signs)[torch.randint(0, 3, k.shape, generator=_gen(1))]
        c.scales = k * by, v * by.flip(-1) if by.dim() else v * by
        c.check()
        c.scales = k * by, v
        c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_keys_scales_whose_product_with_the_scale_is_none(case, dtype):
    """A head's scale that is lost in 32 bits when multiplied by the scores' scale."""
    new, lengths, window = case
    c = Case(new, lengths, 16, 6, 2, 64, 80, dtype, "head", window=window)
    c.scales = torch.tensor([2.0 ** -120, 0.02]), c.scales[1]
    c.check(scale=2.0 ** -40)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [-1.0, -2.0 ** -7, 1.0])
def test_weights_that_a_scale_makes_minus_one(dtype, scale):
    """Equal weights times a scale below 0, beside a value that is no number and that only the last
    token sees: no key is left out."""
    n, length, page = 3, 60, 16
    c = Case([n], [length], page, 2, 1, 64, 64, dtype, "row")
    c.k = torch.where(c.k.float().isnan(), c.k.float(), 0.0).to(F8)
    c.scales = c.scales[0], torch.full_like(c.scales[1], scale)
    want, slack = c.want(0.125)
    v = c.v.float()
    v[int(c.table[0, (length - 1) // page]), (length - 1) % page, 0, 7] = NAN
    got = _attend(c, *c.scales, v=v.to(F8)).cpu()
    none = torch.zeros_like(want, dtype=torch.bool)
    none[n - 1, :, 7] = True
    assert torch.equal(~got.isfinite(), none)
    _within(torch.where(none, 0, got), torch.where(none, 0, want), slack, dtype)


def _without_loss(c, scale):
    """c.want, its slack without what weights of 5 exponent bits may lose: the weights' half step, twice
    the scores' worst, and both sums."""
    want, _ = c.want(scale)
    slack = torch.zeros_like(want)
    for s, n in enumerate(c.new):
        (k, there), (v, _) = c.rows(s, 0), c.rows(s, 1)
        length = c.lengths[s]
        see = (torch.arange(length) <= length - n + torch.arange(n)[:, None]) & there
        rows = slice(int(c.starts[s]), int(c.starts[s + 1]))
        x = c.q[rows].double()
        for h in range(x.shape[1]):
            kh, vh = k[:, h // c.group], v[:, h // c.group]
            a = (scale * (x[:, h] @ kh.t())).masked_fill(~see, -math.inf)
            off = scale * (x.shape[2] + 16) * U32 * (x[:, h].abs() @ kh.abs().t()) + 4 * U32
            worst = off.masked_fill(~see, 0.0).amax(1, keepdim=True)
            slack[rows, h] = torch.softmax(a, dim=1) @ vh.abs() * (
                _u(c.dtype) + 2 * worst + 2 * (length + 16) * U32) * 1.01
    return want, slack


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,length", [(1, 700), (3, 300), (130, 400)])
@pytest.mark.parametrize("low,high", [(-24, 10), (-24, -20), (5, 10), (-60, -30)])
def test_scales_of_values_of_all_magnitudes(low, high, new, length, dtype):
    """Row scales between two powers of two: what a weight times its scale is does not matter."""
    c = Case([new], [length], 16, 4, 2, 64, 72, dtype, "row")
    c.v = (c.v.float() / 64).to(F8)
    g = _gen(high)
    by = 2.0 ** (low + (high - low) * torch.rand(c.scales[1].shape, generator=g))
    c.scales = c.scales[0], by.float()
    want, slack = _without_loss(c, 0.125)
    _within(_attend(c, *c.scales), want, slack, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("most,first", [(1e-3, 1.0), (1e-3, 1e-3 / 448), (1e-2, 1.0), (1e-1, 1e-4)])
def test_small_values_behind_a_row_of_zeros(most, first, new, dtype):
    """One key of weight 1 whose values are zeros, with the scale 1 as a row of zeros is stored or
    another, and thousands of 2^-14 of its weight, of small values."""
    length, page = 8192, 64
    c = Case([new], [length], page, 4, 1, 64, 64, dtype, "row", seed=2)
    at = torch.arange(length)
    page_of, place = c.table[0, at // page].long(), at % page
    k, v = torch.zeros(*c.k.shape), torch.zeros(*c.v.shape)
    k[page_of, place, 0, 0] = -448.0
    k[page_of[0], place[0], 0, 0] = 0.0
    v[page_of, place, 0] = 448.0 * (0.5 + 0.5 * torch.rand(length, 64, generator=_gen(1)))
    v[page_of[0], place[0]] = 0.0
    c.k, c.v = k.to(F8), v.to(F8)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    scales = torch.full_like(c.scales[1], most / 448)
    scales[page_of[0], place[0]] = first
    c.scales = torch.full_like(scales, 14 * math.log(2.0) / 448), scales
    want, slack = _without_loss(c, 1.0)
    assert float(want[-1].abs().max()) > 0.1 * most
    _within(_attend(c, *c.scales, scale=1.0), want, slack, dtype)
