"""GPU tests of the calls on token rows against their definitions in 64 bits.

Tolerances.  A rounding to a type is off by at most half a step, u = eps / 2
relative to the value (plus half the smallest subnormal); a chain of n 32-bit
additions or fused multiply-adds is off by at most n 2^-24 times the sum of
the terms' magnitudes.  Moves without arithmetic are held to equality."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
U32 = 2.0 ** -24
F8 = torch.float8_e4m3fn


def _half_step(dtype):
    info = torch.finfo(dtype)
    return info.eps / 2, info.tiny * info.eps / 2  # relative, and of the subnormals


def _near(got, want, slack, dtype):
    """got within its type's rounding of want (64 bits), and `slack` more."""
    u, least = _half_step(dtype)
    off = (got.double().cpu() - want).abs()
    bound = slack * (1 + u) + u * want.abs() + least
    bad = ~(off <= bound)
    assert not bool(bad.any()), "%d values off, the worst by %g of %g" % (
        int(bad.sum()), float((off / bound)[bad].max()), 1.0)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------
# The order
# --------------------------------------------------------------------------

def _order_reference(experts, count, align):
    flat = np.asarray(experts).reshape(-1)
    n = flat.size
    capacity = n + min(n, count) * (align - 1)
    rows, slots = np.full(n, -1, np.int64), np.full(capacity, -1, np.int64)
    offsets, counts, at = [0], [], 0
    for e in range(count):
        mine = np.nonzero(flat == e)[0]
        rows[mine] = at + np.arange(mine.size)
        slots[at:at + mine.size] = mine
        counts.append(mine.size)
        at += -(-mine.size // align) * align
        offsets.append(at)
    return offsets, counts, rows, slots


def _check_order(experts, count, align=1, **kw):
    order = bm.expert_order(experts, count, align=align, **kw)
    torch.cuda.synchronize()
    offsets, counts, rows, slots = _order_reference(experts.cpu().numpy(), count, align)
    assert order.offsets.tolist() == list(offsets)
    assert order.counts.tolist() == counts
    assert np.array_equal(order.rows.cpu().numpy().reshape(-1), rows)
    assert np.array_equal(order.slots.cpu().numpy(), slots)
    return order


@pytest.mark.parametrize("count", [1, 2, 60, 64, 1024, 1025, 2048])
@pytest.mark.parametrize("shape", [(0, 4), (1, 1), (1, 8), (63, 1), (64, 1), (65, 3), (1024, 4),
                                   (1365, 3), (4097, 1), (2050, 2), (40001, 3)])
def test_order(shape, count):
    g = _gen(shape[0] * 7 + count)
    experts = torch.randint(-1, count, shape, generator=g)
    _check_order(experts.to(DEV), count)
    _check_order(experts.to(torch.int32).to(DEV), count, align=16)


@pytest.mark.parametrize("n", [5000, 3, 600000])
def test_order_of_skewed_choices(n):
    """All of one expert, all dropped, and one expert that is wanted by most."""
    for fill in (0, 7, -1, 8):
        _check_order(torch.full((n, 1), fill, dtype=torch.int64, device=DEV), 8, align=4)
    some = torch.randint(0, 50, (n, 1), generator=_gen(n))
    _check_order(torch.where(some < 8, some, 3).to(DEV), 8)


@pytest.mark.parametrize("n,count", [
    (256, 5), (257, 2048), (1024, 7), (1025, 7), (4096, 1024), (4097, 300), (8192, 64), (8193, 64), (9000, 2048), (16384, 9),
    (16384, 2048), (16385, 9), (30000, 1), (65536, 30), (65537, 30), (530000, 700), (4300000, 5), (4300000, 1500)])
def test_order_of_many_lengths(n, count):
    """One workgroup and several, choices held in registers and read twice."""
    experts = torch.randint(-1, count + 1, (n, 1), generator=_gen(n + count))
    _check_order(experts.to(torch.int32).to(DEV), count, align=3)


def test_order_with_wide_padding():
    for n, align in ((20000, 5000), (100, 30000), (5000, 200000)):
        experts = torch.randint(0, 7, (n, 1), generator=_gen(9))
        _check_order(experts.to(DEV), 7, align=align)


def test_order_drops_far_values():
    """Values that would be experts if their upper half were lost."""
    v = torch.tensor([1 << 32, (1 << 32) + 1, -(1 << 32), 2, (1 << 62) + 2, 0, -1, 3],
                     dtype=torch.int64, device=DEV)
    order = _check_order(v, 3)
    assert order.rows.shape == (8, 1) and order.counts.tolist() == [1, 0, 1]
    w = torch.tensor([2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device=DEV)
    assert bm.expert_order(w, 2).rows.reshape(-1).tolist() == [-1, -1, 0]


# --------------------------------------------------------------------------
# Gather, combine and their gradients
# --------------------------------------------------------------------------

def _make_order(tokens, choices, count, drop, align, seed):
    g = _gen(seed)
    scores = torch.rand(tokens, count, generator=g)
    experts = scores.topk(choices, dim=1).indices
    if drop:
        experts = torch.where(torch.rand(tokens, choices, generator=g) < drop, -1, experts)
    order = bm.expert_order(experts.contiguous().to(DEV), count, align=align)
    return order, order.rows.cpu().long(), order.slots.cpu().long()


MOVES = [  # tokens, choices, experts, width, drop, align
    (1, 1, 1, 1, 0.0, 1), (1, 8, 8, 2048, 0.0, 1), (2, 3, 5, 3, 0.3, 4), (5, 2, 4, 7, 0.0, 1),
    (9, 2, 4, 8, 0.5, 1), (33, 4, 16, 9, 0.2, 8), (64, 7, 9, 64, 0.0, 1), (65, 9, 17, 65, 0.1, 16),
    (130, 5, 8, 513, 0.5, 1), (257, 6, 60, 1001, 0.2, 32), (300, 8, 64, 2048, 0.0, 1),
    (128, 10, 40, 2880, 0.1, 1), (4099, 3, 8, 136, 0.3, 1), (5000, 8, 16, 40, 0.0, 64),
    (70, 17, 32, 1100, 0.9, 16), (20, 4, 8, 512, 1.0, 1), (40, 25, 64, 4100, 0.0, 1),
    (7, 8, 8, 256, 0.0, 1), (3, 3, 4, 700, 0.0, 1), (5, 8, 16, 1024, 0.2, 1), (11, 15, 16, 515, 0.1, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", MOVES, ids=str)
def test_gather_and_its_gradient(case, dtype):
    tokens, choices, count, width, drop, align = case
    order, rows, slots = _make_order(tokens, choices, count, drop, align, width)
    x = torch.randn(tokens, width, generator=_gen(1)).to(dtype)
    out = torch.full((slots.numel(), width), float("nan"), dtype=dtype, device=DEV)
    bm.expert_gather(x.to(DEV), order, out=out)
    want = torch.where(slots[:, None] >= 0, x[slots.clamp(min=0) // choices], torch.zeros(()).to(dtype))
    assert torch.equal(out.cpu(), want)

    grad = torch.randn(slots.numel(), width, generator=_gen(2)).to(dtype)
    got = bm.expert_gather_backward(grad.to(DEV), order)
    picked = torch.where(rows[..., None] >= 0, grad.double()[rows.clamp(min=0)],
                         torch.zeros((), dtype=torch.float64))
    _near(got, picked.sum(1), choices * U32 * picked.abs().sum(1), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", MOVES, ids=str)
def test_combine_and_its_gradients(case, dtype):
    tokens, choices, count, width, drop, align = case
    order, rows, slots = _make_order(tokens, choices, count, drop, align, width)
    x = torch.randn(slots.numel(), width, generator=_gen(3)).to(dtype)
    grad = torch.randn(tokens, width, generator=_gen(4)).to(dtype)
    held = rows[..., None] >= 0
    nothing = torch.zeros((), dtype=torch.float64)
    picked = torch.where(held, x.double()[rows.clamp(min=0)], nothing)
    for wtype in {torch.float32, dtype}:
        w = torch.rand(tokens, choices, generator=_gen(5)).to(wtype)
        got = bm.expert_combine(x.to(DEV), order, w.to(DEV))
        terms = picked * w.double()[..., None]
        _near(got, terms.sum(1), choices * U32 * terms.abs().sum(1), dtype)

        grad_x, grad_w = bm.expert_combine_backward(grad.to(DEV), x.to(DEV), order, w.to(DEV))
        at = slots.clamp(min=0)
        want = grad.double()[at // choices] * w.double().reshape(-1)[at][:, None]
        want = torch.where(slots[:, None] >= 0, want, nothing)
        _near(grad_x, want, U32 * want.abs(), dtype)
        assert not bool(grad_x.cpu()[slots < 0].any())
        dots = grad.double()[:, None] * picked
        # a lane adds at most width + 1 products, then 6 sums join lanes and 4 waves
        _near(grad_w, dots.sum(-1), (width + 10) * U32 * dots.abs().sum(-1), wtype)


def test_combine_ignores_what_is_not_held():
    """NaN and infinity in padding, in rows of no choice and in row 0 do not
    reach a token whose choice is dropped; a kept NaN does."""
    experts = torch.tensor([[0, -1], [-1, -1], [1, 0]], device=DEV)
    order = bm.expert_order(experts, 2, align=4)
    rows = order.rows.cpu()
    x = torch.full((order.slots.numel(), 600), float("nan"))
    x[int(rows[0, 0])] = float("inf")
    x[int(rows[2, 0])] = 2.0
    x[int(rows[2, 1])] = 3.0
    for dtype in TYPES:
        w = torch.tensor([[1.0, float("nan")], [float("inf"), 1.0], [0.5, 2.0]], device=DEV)
        got = bm.expert_combine(x.to(dtype).to(DEV), order, w).cpu().float()
        assert bool((got[0] == float("inf")).all())
        assert not bool(got[1].any()) and bool((got[2] == 7.0).all())
        grad_x, grad_w = bm.expert_combine_backward(torch.ones(3, 600, dtype=dtype, device=DEV),
                                                    x.to(dtype).to(DEV), order, w)
        assert grad_w.cpu().tolist()[1] == [0.0, 0.0] and grad_w[0, 1] == 0
        assert not bool(grad_x.cpu()[order.slots.cpu() < 0].any())
        assert bm.expert_combine(torch.full_like(x, float("nan")).to(dtype).to(DEV), order,
                                 w).isnan().cpu().any(1).tolist() == [True, False, True]


@pytest.mark.parametrize("case", [  # tokens, choices, width: rows by expert of 98 MiB and more
    (13000, 6, 4096), (13000, 6, 4095), (14000, 8, 1024), (30000, 2, 1024)], ids=str)
def test_moves_of_more_than_the_caches_hold(case):
    """Rows that are streamed, checked on the device: sums in 64 bits."""
    tokens, choices, width = case
    g = torch.Generator(device=DEV).manual_seed(width)
    experts = torch.rand(tokens, 24, device=DEV, generator=g).topk(choices, dim=1).indices
    experts = torch.where(torch.rand(tokens, choices, device=DEV, generator=g) < 0.1, -1, experts)
    order = bm.expert_order(experts.contiguous(), 24, align=16)
    rows, slots = order.rows.long(), order.slots.long()
    held, at = slots >= 0, slots.clamp(min=0)
    x = torch.randn(tokens, width, device=DEV, generator=g).to(torch.bfloat16)
    w = torch.rand(tokens, choices, device=DEV, generator=g)
    y = bm.expert_gather(x, order)
    assert torch.equal(y[held], x[at[held] // choices]) and not bool(y[~held].any())
    y = torch.randn(y.shape, device=DEV, generator=g).to(torch.bfloat16)
    got = bm.expert_combine(y, order, w)
    grad_y, grad_w = bm.expert_combine_backward(x, y, order, w)
    want, size = (torch.zeros(tokens, width, dtype=torch.float64, device=DEV) for _ in range(2))
    for k in range(choices):
        one = y[rows[:, k].clamp(min=0)].double() * (rows[:, k] >= 0)[:, None]
        term = one * w[:, k, None].double()
        want += term
        size += term.abs()
        dots = x.double() * one
        off = (grad_w[:, k].double() - dots.sum(1)).abs()
        assert bool((off <= (width + 10) * U32 * dots.abs().sum(1) + U32 * dots.sum(1).abs()).all())
    u = 2.0 ** -8
    assert bool(((got.double() - want).abs() <= choices * U32 * size * (1 + u) + u * want.abs()).all())
    want = x[at // choices].float() * w.reshape(-1)[at][:, None]
    assert torch.equal(grad_y[held], want.to(torch.bfloat16)[held]) and not bool(grad_y[~held].any())


def test_wrong_rows_are_skipped():
    """Rows of an order that point nowhere are skipped, not followed."""
    order, rows, slots = _make_order(40, 4, 8, 0.0, 1, 3)
    bad = order.rows.clone()
    bad[3, 1], bad[7, 0], bad[8, 2], bad[9, 3] = 160, 2 ** 31 - 1, -2 ** 31, -7
    wrong = order._replace(rows=bad)
    keep = ((bad >= 0) & (bad < 160)).cpu()
    x = torch.randn(160, 100, generator=_gen(6))
    got = bm.expert_combine(x.to(DEV), wrong)
    picked = torch.where(keep[..., None], x.double()[rows], torch.zeros((), dtype=torch.float64))
    _near(got, picked.sum(1), 4 * U32 * picked.abs().sum(1), torch.float32)
    y = torch.randn(40, 100, generator=_gen(7))
    out = bm.expert_gather(y.to(DEV), wrong, out=torch.zeros(160, 100, device=DEV)).cpu()
    for t in range(40):
        for k in range(4):
            assert torch.equal(out[rows[t, k]], y[t] if keep[t, k] else torch.zeros(100))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_with_strides(dtype):
    """Views with rows apart, and at odd elements; what lies between stays."""
    order, rows, slots = _make_order(50, 3, 7, 0.2, 1, 4)
    wide = torch.randn(50, 211, generator=_gen(8)).to(dtype).to(DEV)
    x = wide[:, 3:104]
    out = torch.full((150, 128), 5.0, dtype=dtype, device=DEV)
    got = bm.expert_gather(x, order, out=out[:, 1:102])
    assert torch.equal(got, bm.expert_gather(x.contiguous(), order))
    assert bool((out[:, 0] == 5).all()) and bool((out[:, 102:] == 5).all())
    w = torch.rand(50, 3, generator=_gen(9)).to(DEV)
    back = torch.full((50, 107), 5.0, dtype=dtype, device=DEV)
    bm.expert_combine(out[:, 1:102], order, w, out=back[:, 5:106])
    assert torch.equal(back[:, 5:106], bm.expert_combine(got.contiguous(), order, w))
    assert bool((back[:, :5] == 5).all()) and bool((back[:, 106:] == 5).all())
    same = wide[:1, :101].expand(50, 101)  # one row read for every token
    assert torch.equal(bm.expert_gather(same, order), bm.expert_gather(same.contiguous(), order))
    a = bm.expert_combine_backward(x, out[:, 1:102], order, w)
    b = bm.expert_combine_backward(x.contiguous(), got.contiguous(), order, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_sums_are_the_same_each_time():
    order, _, slots = _make_order(3000, 8, 64, 0.1, 1, 5)
    x = torch.randn(slots.numel(), 1000, generator=_gen(10)).to(torch.bfloat16).to(DEV)
    grad, w = torch.randn(3000, 1000, device=DEV).to(torch.bfloat16), torch.rand(3000, 8, device=DEV)
    first = (bm.expert_combine(x, order, w), *bm.expert_combine_backward(grad, x, order, w))
    for _ in range(3):
        again = (bm.expert_combine(x, order, w), *bm.expert_combine_backward(grad, x, order, w))
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_rows_past_32_bits():
    """Rows whose offsets in elements and in bytes pass 32 bits."""
    stride = (1 << 31) // 3 + 5
    order = bm.expert_order(torch.tensor([[3, 0], [1, 2]], device=DEV), 4)
    big = torch.empty(3 * stride + 64, dtype=torch.bfloat16, device=DEV)
    rows = big.as_strided((4, 64), (stride, 1))
    x = torch.randn(2, 64, generator=_gen(11)).to(torch.bfloat16).to(DEV)
    bm.expert_gather(x, order, out=rows)
    assert torch.equal(rows.cpu(), x[[0, 1, 1, 0]].cpu())
    assert torch.equal(bm.expert_combine(rows, order, torch.tensor([[1.0, 0.0], [0.0, 1.0]], device=DEV)), x)
    grad, _ = bm.expert_combine_backward(x, rows, order, torch.ones(2, 2, device=DEV))
    assert torch.equal(grad, rows.contiguous())


def test_empty_tokens():
    order = bm.expert_order(torch.zeros(0, 4, dtype=torch.int64, device=DEV), 8, align=16)
    assert order.offsets.tolist() == [0] * 9 and order.slots.numel() == 0
    x = torch.zeros(0, 32, device=DEV)
    assert bm.expert_gather(x, order).shape == (0, 32)
    assert bm.expert_combine(x, order, torch.zeros(0, 4, device=DEV)).shape == (0, 32)
    assert bm.expert_combine_backward(x, x, order, torch.zeros(0, 4, device=DEV))[1].shape == (0, 4)


def test_gradients_against_differences():
    """The moves are linear in each input, so that a difference of two calls,
    one input moved by a step, is the derivative times the step."""
    order, rows, slots = _make_order(6, 3, 5, 0.2, 2, 6)
    n, width = slots.numel(), 20
    x, dx = (torch.randn(n, width, generator=_gen(s)).to(DEV) for s in (12, 13))
    w, dw = (torch.randn(6, 3, generator=_gen(s)).to(DEV) for s in (14, 15))
    grad = torch.randn(6, width, generator=_gen(16)).to(DEV)
    grad_x, grad_w = bm.expert_combine_backward(grad, x, order, w)

    def loss(x, w):
        return float((bm.expert_combine(x, order, w).double() * grad.double()).sum())
    size = float((bm.expert_combine(x.abs() + dx.abs(), order, w.abs() + dw.abs()) * grad.abs()).sum())
    tol = 40 * U32 * size  # a sum of 20 products and 10 more, and a few roundings of each loss
    assert abs(loss(x + dx, w) - loss(x, w) - float((grad_x.double() * dx.double()).sum())) <= tol
    assert abs(loss(x, w + dw) - loss(x, w) - float((grad_w.double() * dw.double()).sum())) <= tol
    y, dy = (torch.randn(6, width, generator=_gen(s)).to(DEV) for s in (17, 18))
    g = torch.randn(n, width, generator=_gen(19)).to(DEV)
    diff = bm.expert_gather(y + dy, order).double() - bm.expert_gather(y, order).double()
    want = float((diff * g.double()).sum())
    got = float((bm.expert_gather_backward(g, order).double() * dy.double()).sum())
    assert abs(want - got) <= 16 * U32 * float(((y.abs() + dy.abs()).sum() * g.abs().max())) * 3


def test_autograd_of_the_moves():
    """A layer's way through its experts under autograd, against the same in 64 bits."""
    tokens, choices, count, width = 37, 3, 6, 48
    order, rows, slots = _make_order(tokens, choices, count, 0.2, 4, 7)
    x0 = torch.randn(tokens, width, generator=_gen(20))
    w0 = torch.rand(tokens, choices, generator=_gen(21))
    a0 = torch.randn(width, width, generator=_gen(22)) / 7

    def plain(x, w, a):
        held = (rows >= 0).double()
        y = torch.tanh(x.reshape(tokens, 1, width) @ a).expand(tokens, choices, width)
        return (y * (w * held)[..., None]).sum(1)
    x, w, a = (t.double().requires_grad_() for t in (x0, w0, a0))
    plain(x, w, a).square().sum().backward()
    xd, wd, ad = (t.to(DEV).requires_grad_() for t in (x0, w0, a0))
    out = bm.expert_combine(torch.tanh(bm.expert_gather(xd, order) @ ad), order, wd)
    out.square().sum().backward()
    for got, want in ((xd.grad, x.grad), (wd.grad, w.grad), (ad.grad, a.grad)):
        # 48- and 37-term sums in 32 bits, twice over
        assert float((got.double().cpu() - want).abs().max()) <= 400 * U32 * float(want.abs().max())
    y = torch.randn(slots.numel(), width, device=DEV, requires_grad=True)
    bm.expert_combine(y, order).sum().backward()
    assert torch.equal(y.grad[:, 0].cpu(), (slots >= 0).float())


# --------------------------------------------------------------------------
# Rotary positions
# --------------------------------------------------------------------------

def _turned(x, angle, interleaved, inverse=False, scale=1.0):
    """x [..., H, D] and angle [..., P], in 64 bits."""
    x, pairs = x.double(), angle.shape[-1]
    c, s = torch.cos(angle).unsqueeze(-2), torch.sin(angle).unsqueeze(-2)
    s = -s if inverse else s
    out = x.clone()
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out[..., lo] = scale * (x[..., lo] * c - x[..., hi] * s)
    out[..., hi] = scale * (x[..., hi] * c + x[..., lo] * s)
    return out


def _turn_slack(x, angle, interleaved, scale=1.0):
    """The reduced angle, at most pi / 4, is rounded three times and the series
    about three times more, which is below 6 2^-24 of cosine and sine; the
    scale and the two products round four times more.  The 64-bit angle is off
    by 4 2^-53 of itself on either side."""
    pairs = angle.shape[-1]
    a = x.double().abs()
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    both = (a[..., lo] + a[..., hi]) * abs(scale)
    slack = torch.zeros_like(a)
    each = both * (10 * U32 + 2.0 ** -50 * angle.abs().unsqueeze(-2))
    slack[..., lo], slack[..., hi] = each, each
    return slack


def _freqs(pairs, dtype=torch.float64):
    return (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).to(dtype)


ROTARY = [  # tokens, heads, size, pairs, axes, interleaved
    (1, 1, 2, 1, 1, False), (3, 2, 2, 1, 1, True), (2, 3, 7, 3, 2, False), (5, 1, 16, 8, 1, True),
    (9, 4, 64, 32, 3, False), (17, 5, 72, 36, 2, True), (33, 2, 80, 20, 1, False),
    (64, 8, 128, 64, 3, False), (65, 3, 128, 64, 1, True), (7, 2, 100, 50, 2, False),
    (11, 2, 100, 45, 8, True), (3, 9, 256, 128, 3, False), (4, 2, 512, 256, 2, False),
    (5, 2, 512, 256, 1, True), (6, 2, 510, 4, 1, False), (4500, 2, 64, 32, 2, False),
    (2100, 3, 34, 17, 1, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_rotary(case, dtype):
    tokens, heads, size, pairs, axes, interleaved = case
    g = _gen(size + tokens)
    x = torch.randn(tokens, heads, size, generator=g).to(dtype)
    positions = torch.randint(-50, 9000, (axes, tokens), generator=g)
    axis = torch.randint(0, axes, (pairs,), generator=g).to(torch.int32)
    freqs = _freqs(pairs)
    angle = positions.double()[axis.long()].t() * freqs
    args = (positions.to(DEV), freqs.to(DEV), axis.to(DEV), interleaved)
    xd = x.to(DEV)
    got = bm.rotary(xd, *args)
    slack = _turn_slack(x, angle, interleaved)
    _near(got, _turned(x, angle, interleaved), slack, dtype)
    assert torch.equal(got[..., 2 * pairs:], xd[..., 2 * pairs:])
    back = bm.rotary_backward(xd, *args)
    _near(back, _turned(x, angle, interleaved, inverse=True), slack, dtype)
    # in place, and two tensors at once, of other numbers of heads
    again = xd.clone()
    assert bm.rotary(again, *args, out=again) is again and torch.equal(again, got)
    pair = (torch.cat([xd, xd], 1), xd.clone())
    q, k = bm.rotary(pair, *args, out=pair)
    assert torch.equal(q, torch.cat([got, got], 1)) and torch.equal(k, got)
    p32, f32 = args[0].to(torch.int32), args[1].float()
    angle = positions.double()[axis.long()].t() * freqs.float().double()
    _near(bm.rotary(xd, p32, f32, args[2], interleaved), _turned(x, angle, interleaved),
          _turn_slack(x, angle, interleaved), dtype)


def test_rotary_layouts():
    """Batches, heads before tokens, and views of one projection give what
    their contiguous copies give."""
    g = _gen(30)
    positions, freqs = torch.randint(0, 5000, (3, 2, 50), generator=g).to(DEV), _freqs(16).to(DEV)
    axes = bm.rotary_axes([6, 5, 5], device=DEV)
    x = torch.randn(2, 6, 50, 40, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
    flat = bm.rotary(x.reshape(100, 6, 40), positions.reshape(3, 100), freqs, axes)
    got = bm.rotary(x, positions, freqs, axes)
    assert got.stride() == x.stride() and torch.equal(got.reshape(100, 6, 40), flat)
    both = torch.randn(100, 10 * 40, generator=g).to(torch.float16).to(DEV)
    q, k = both[:, :160].unflatten(1, (4, 40)), both[:, 160:240].unflatten(1, (2, 40))
    want = bm.rotary((q.contiguous(), k.contiguous()), positions.reshape(3, 100), freqs, axes)
    rest = both[:, 240:].clone()
    got = bm.rotary((q, k), positions.reshape(3, 100), freqs, axes, out=(q, k))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(both[:, 240:], rest)
    one = bm.rotary(x, positions[0], freqs)
    assert torch.equal(one, bm.rotary(x, positions[:1], freqs))
    assert bm.rotary(x[:0], positions[:, :0], freqs, axes).shape == (0, 50, 6, 40)


def test_turns_of_more_than_the_caches_hold():
    """Heads that are streamed give what parts of them give."""
    g = torch.Generator(device=DEV).manual_seed(34)
    both = torch.randn(12000, 28 * 128, device=DEV, generator=g).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, 128)) for t in both.split([20 * 128, 4 * 128, 4 * 128], dim=1))
    positions, freqs = torch.randint(0, 9000, (3, 12000), generator=_gen(35)).to(DEV), _freqs(50).to(DEV)
    axes = bm.rotary_axes([20, 15, 15], device=DEV)
    want = [bm.rotary((q[a:a + 1000], k[a:a + 1000]), positions[:, a:a + 1000].contiguous(), freqs, axes)
            for a in range(0, 12000, 1000)]
    got = bm.rotary((q, k), positions, freqs, axes)
    for i in range(2):
        assert torch.equal(got[i], torch.cat([w[i] for w in want]))
    caches = [torch.zeros(1500, 8, 4, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.randperm(1500, generator=_gen(36)).to(torch.int32).reshape(3, 500).to(DEV)
    place = torch.arange(12000, device=DEV)
    out = bm.cache_append(k, v, *caches, table, place % 4000, sequences=(place // 4000).to(torch.int32),
                          freqs=freqs, axes=axes, turns=positions, q=q)
    page = table[place // 4000, place % 4000 // 8].long()
    assert torch.equal(out, got[0]) and torch.equal(caches[0][page, place % 8], got[1])
    assert torch.equal(caches[1][page, place % 8], v)


def test_rotary_of_far_positions():
    """Angles whose 32-bit form has lost the turn: a position and its
    neighbour differ by the frequency's angle, wherever they are."""
    for base in (1 << 20, (1 << 31) - 2, 10 ** 12, -(1 << 40)):
        positions = torch.tensor([base, base + 1])
        freqs = _freqs(32)
        x = torch.randn(2, 3, 64, generator=_gen(31))
        got = bm.rotary(x.to(DEV), positions.to(DEV), freqs.to(DEV))
        angle = positions.double()[:, None] * freqs
        _near(got, _turned(x, angle, False), _turn_slack(x, angle, False), torch.float32)


def test_rotary_scale_axes_and_special_values():
    g = _gen(32)
    x = torch.randn(10, 2, 32, generator=g).to(DEV)
    positions = torch.randint(1, 100, (2, 10), generator=g)
    freqs = _freqs(16)
    axis = torch.tensor([0, 1, 2, -1] * 4, dtype=torch.int32)  # two of four have no axis
    angle = positions.double()[axis.long().clamp(0, 1)].t() * freqs
    angle[:, (axis < 0) | (axis > 1)] = 0.0
    got = bm.rotary(x, positions.to(DEV), freqs.to(DEV), axis.to(DEV), scale=1.25)
    _near(got, _turned(x.cpu(), angle, False, scale=1.25), _turn_slack(x.cpu(), angle, False, 1.25),
          torch.float32)
    zero = bm.rotary(x, torch.zeros(10, dtype=torch.int64, device=DEV), freqs.to(DEV))
    assert torch.equal(zero, x)
    x[3, 1, 5], x[4, 0, 31] = float("nan"), float("inf")
    got = bm.rotary(x, positions[0].to(DEV), freqs.to(DEV)).isfinite().cpu()
    assert torch.nonzero(~got).tolist() == [[3, 1, 5], [3, 1, 21], [4, 0, 15], [4, 0, 31]]


def test_rotary_gradient():
    """Against the formula's own gradient, against differences (the turn is
    linear) and through autograd."""
    g = _gen(33)
    positions, freqs = torch.randint(0, 9000, (3, 12), generator=g), _freqs(10)
    axis = bm.rotary_axes([4, 3, 3], interleaved=True)
    angle = positions.double()[axis.long()].t() * freqs
    args = (positions.to(DEV), freqs.to(DEV), axis.to(DEV), True, 0.75)
    x, dx, grad = (torch.randn(12, 3, 24, generator=g) for _ in range(3))
    ref = x.double().requires_grad_()
    (_turned(ref, angle, True, scale=0.75) * grad.double()).sum().backward()
    slack = _turn_slack(grad, angle, True, 0.75)
    _near(bm.rotary_backward(grad.to(DEV), *args), ref.grad, slack, torch.float32)
    diff = (bm.rotary((x + dx).to(DEV), *args).double() - bm.rotary(x.to(DEV), *args).double()).cpu()
    want = (bm.rotary_backward(grad.to(DEV), *args).double().cpu() * dx.double()).sum()
    size = 2 * float(grad.abs().sum() * (x.abs() + dx.abs()).max())
    assert abs(float((diff * grad.double()).sum() - want)) <= 40 * U32 * size
    q, k = x.to(DEV).requires_grad_(), dx.to(DEV).requires_grad_()
    a, b = bm.rotary((q, k), *args)
    ((a * grad.to(DEV)).sum() + b.sum()).backward()
    assert torch.equal(q.grad, bm.rotary_backward(grad.to(DEV), *args))
    assert torch.equal(k.grad, bm.rotary_backward(torch.ones_like(k), *args))


# --------------------------------------------------------------------------
# The paged cache
# --------------------------------------------------------------------------

def _append_case(tokens, batch, page, heads, dim, v_dim, dtype, seed, pages=None):
    """Sequences of several lengths, each with new tokens; pages in no order."""
    g = _gen(seed)
    owner = torch.cat([torch.arange(min(batch, tokens)),
                       torch.randint(0, batch, (max(tokens - batch, 0),), generator=g)])
    owner = owner.sort().values
    held = torch.randint(0, 3 * page, (batch,), generator=g)
    first = torch.searchsorted(owner, torch.arange(batch))
    place = held[owner] + torch.arange(tokens) - first[owner]
    width = int(place.max()) // page + 2
    pages = pages or batch * width + 3
    table = torch.randperm(pages, generator=g)[:batch * width].reshape(batch, width)
    return {"k": torch.randn(tokens, heads, dim, generator=g).to(dtype),
            "v": torch.randn(tokens, heads, v_dim, generator=g).to(dtype),
            "table": table.to(torch.int32), "sequences": owner.to(torch.int32),
            "positions": place, "pages": pages}


def _expected(cache, values, c, page):
    """Every token's values at its place, in order."""
    out = cache.clone()
    for t in range(values.shape[0]):
        s, p = int(c["sequences"][t]), int(c["positions"][t])
        out[int(c["table"][s, p // page]), p % page] = values[t]
    return out


APPENDS = [  # tokens, batch, page, heads, size of k, of v, pairs, interleaved, heads first
    (1, 1, 1, 1, 2, 1, 1, False, False), (5, 5, 16, 2, 64, 64, 32, False, False),
    (64, 64, 16, 8, 128, 128, 64, False, True), (100, 3, 7, 2, 96, 40, 24, True, False),
    (33, 4, 32, 3, 20, 7, 3, False, False), (50, 2, 48, 1, 100, 100, 50, False, True),
    (17, 2, 5, 2, 130, 512, 65, True, True), (3000, 6, 64, 2, 64, 64, 32, False, False),
    (40, 4, 16, 4, 192, 128, 96, False, False), (25, 1, 1, 2, 66, 9, 0, False, False),
    (4500, 9, 16, 1, 24, 24, 0, False, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append(case, dtype):
    tokens, batch, page, heads, dim, v_dim, pairs, interleaved, first = case
    c = _append_case(tokens, batch, page, heads, dim, v_dim, dtype, tokens + dim)

    def pool(d):
        fill = torch.randn(c["pages"], page, heads, d, generator=_gen(d)).to(dtype)
        if first:
            return fill, fill.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        return fill, fill.to(DEV)
    k0, kc = pool(dim)
    v0, vc = pool(v_dim)
    index = {"sequences": c["sequences"].to(DEV)}
    if batch == tokens:
        index = {}
    args = (c["k"].to(DEV), c["v"].to(DEV), kc, vc, c["table"].to(DEV), c["positions"].to(DEV))
    if pairs:
        freqs = _freqs(pairs)
        angle = c["positions"].double()[:, None] * freqs
        q = torch.randn(tokens, 3 * heads, dim, generator=_gen(40)).to(dtype)
        got = bm.cache_append(*args, freqs=freqs.to(DEV), interleaved=interleaved, q=q.to(DEV), **index)
        _near(got, _turned(q, angle, interleaved), _turn_slack(q, angle, interleaved), dtype)
        turned = _turned(c["k"], angle, interleaved)
        slack = _turn_slack(c["k"], angle, interleaved)
    else:
        assert bm.cache_append(*args, **index) is None
        turned, slack = c["k"].double(), torch.zeros_like(c["k"], dtype=torch.float64)
    torch.cuda.synchronize()
    assert torch.equal(vc.cpu(), _expected(v0, c["v"], c, page))
    mark = _expected(torch.zeros(c["pages"], page, heads, dim), torch.ones(tokens, heads, dim), c, page)
    want = _expected(k0.double(), turned, c, page)
    _near(kc, want, _expected(torch.zeros_like(want), slack, c, page), dtype)
    assert torch.equal(kc.cpu()[mark == 0], k0[mark == 0])  # nothing else was written


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("each", [True, False])
def test_append_in_8_bits(dtype, each):
    c = _append_case(70, 5, 16, 3, 48, 40, dtype, 50)
    special = torch.tensor([0.0, -0.0, 1e9, -1e9, float("inf"), -float("inf"), float("nan"), 448.0,
                            464.0, 465.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 17.0, 19.0, 0.013])
    c["v"][3, 1, :16] = special.to(dtype)
    scale = torch.rand(3, generator=_gen(51)) * 0.1 + 0.01
    scale[1] = 1.0
    if not each:
        scale = torch.ones(1)
    kc, vc = (torch.randn(c["pages"], 16, 3, d, generator=_gen(d)).to(F8) for d in (48, 40))
    freqs = _freqs(20)
    angle = c["positions"].double()[:, None] * freqs
    kd, vd = kc.to(DEV), vc.to(DEV)
    bm.cache_append(c["k"].to(DEV), c["v"].to(DEV), kd, vd, c["table"].to(DEV),
                    c["positions"].to(DEV), sequences=c["sequences"].to(DEV), freqs=freqs.to(DEV),
                    k_scale=scale.to(DEV), v_scale=scale.to(DEV))
    y = c["v"].float() / scale[:, None]
    y = torch.where(y.isnan(), y, y.clamp(-448.0, 448.0)).to(F8)
    want = _expected(vc.view(torch.uint8), y.view(torch.uint8), c, 16)
    got = vd.cpu().view(torch.uint8)
    nan = (want & 127) == 127
    assert torch.equal((got & 127) == 127, nan) and torch.equal(got[~nan], want[~nan])
    turned = _turned(c["k"], angle, False) / scale.double()[:, None]
    slack = _turn_slack(c["k"], angle, False) / scale.double()[:, None] + U32 * turned.abs()
    slack = _expected(torch.zeros(kc.shape, dtype=torch.float64), slack, c, 16)
    want = _expected(kc.double(), turned.clamp(-448.0, 448.0), c, 16)
    off = (kd.cpu().double() - want).abs()
    # half a step of 3 bits after the first, 2^-10 among the subnormals
    assert bool((off <= slack * (1 + 2.0 ** -4) + 2.0 ** -4 * want.abs() + 2.0 ** -10).all())


def test_append_skips_what_has_no_place():
    """Padding, sequences, positions and pages out of range store nothing, and
    queries are turned all the same."""
    tokens, page = 12, 4
    k = torch.randn(tokens, 2, 16, generator=_gen(60)).to(DEV)
    v, q = k + 1, k - 1
    table = torch.tensor([[0, 1, -1], [5, 6, 2 ** 31 - 1], [2, 3, 4]], dtype=torch.int32, device=DEV)
    sequences = torch.tensor([0, -1, 3, 2 ** 31 - 1, -2 ** 31, 0, 0, 1, 1, 2, 2, 2], dtype=torch.int32)
    positions = torch.tensor([3, 0, 0, 0, 0, 8, -1, 4, 8, 12, 11, 1 << 40])
    stored = {0: (0, 3), 10: (4, 3)}  # of table 1's pages, 5 and 6 are past the cache's 5
    caches = [torch.full((5, page, 2, 16), 9.0, device=DEV) for _ in range(2)]
    freqs = _freqs(8).to(DEV)
    for pos in (positions, positions.clamp(max=2 ** 31 - 1).to(torch.int32)):
        for c in caches:
            c.fill_(9.0)
        got = bm.cache_append(k, v, *caches, table, pos.to(DEV), sequences=sequences.to(DEV),
                              freqs=freqs, q=q)
        assert torch.equal(got, bm.rotary(q, pos.to(DEV), freqs))
        turned = bm.rotary(k, pos.to(DEV), freqs)
        for cache, values in zip(caches, (turned, v)):
            want = torch.full((5, page, 2, 16), 9.0)
            for t, at in stored.items():
                want[at] = values[t].cpu()
            assert torch.equal(cache.cpu(), want)
    none = torch.zeros(0, 3, dtype=torch.int32, device=DEV)  # a batch without sequences
    before = caches[0].clone()
    bm.cache_append(k, v, *caches, none, positions.to(DEV))
    bm.cache_append(k[:0], v[:0], *caches, table, positions[:0].to(DEV))
    assert torch.equal(caches[0], before)


def test_append_by_other_turns():
    """Places in the cache and positions on several axes are not the same."""
    c = _append_case(40, 4, 16, 2, 64, 64, torch.float32, 61)
    turns = torch.randint(0, 3000, (3, 40), generator=_gen(62)).to(torch.int32).to(DEV)
    axes, freqs = bm.rotary_axes([12, 10, 10], device=DEV), _freqs(32).to(DEV)
    caches = [torch.zeros(c["pages"], 16, 2, 64, device=DEV) for _ in range(2)]
    k, q = c["k"].to(DEV), torch.randn(40, 6, 64, generator=_gen(63)).to(DEV)
    want_q, want_k = bm.rotary((q, k), turns, freqs, axes, scale=0.5)
    got = bm.cache_append(k, c["v"].to(DEV), *caches, c["table"].to(DEV), c["positions"].to(DEV),
                          sequences=c["sequences"].to(DEV), freqs=freqs, axes=axes, turns=turns,
                          scale=0.5, q=q, q_out=q)
    assert got is q and torch.equal(q, want_q)
    want = _expected(torch.zeros(caches[0].shape), want_k.cpu(), c, 16)
    assert torch.equal(caches[0].cpu(), want)


def test_append_past_32_bits():
    """Pages whose offsets pass 32 bits, keys and values next to each other."""
    pages, page = 3, 4
    step = (1 << 31) // 2 + 8 * 1024
    big = torch.zeros(2 * step + 4096, dtype=torch.float16, device=DEV)
    big = torch.cat([big, torch.zeros(step, dtype=torch.float16, device=DEV)])
    kc = big.as_strided((pages, page, 2, 64), (step, 128, 64, 1))
    vc = big.as_strided((pages, page, 2, 64), (step, 128, 64, 1), page * 128)
    k = torch.randn(3, 2, 64, generator=_gen(64)).to(torch.float16).to(DEV)
    table = torch.tensor([[2], [0], [1]], dtype=torch.int32, device=DEV)
    bm.cache_append(k, k + 1, kc, vc, table, torch.tensor([1, 2, 3], device=DEV))
    for t, (p, i) in enumerate([(2, 1), (0, 2), (1, 3)]):
        assert torch.equal(kc[p, i], k[t]) and torch.equal(vc[p, i], (k + 1)[t])
    assert int(big.count_nonzero()) == int(k.count_nonzero()) + int((k + 1).count_nonzero())


# --------------------------------------------------------------------------
# Streams and graphs
# --------------------------------------------------------------------------

def _step(x, experts, w, q, k, v, caches, table, positions, freqs, stream=None):
    order = bm.expert_order(experts, 16, stream=stream)
    rows = bm.expert_gather(x, order, stream=stream)
    out = bm.expert_combine(rows, order, w, stream=stream)
    grads = bm.expert_combine_backward(x, rows, order, w, stream=stream)
    turned = bm.cache_append(k, v, *caches, table, positions, freqs=freqs, q=q, stream=stream)
    back = bm.rotary_backward(turned, positions, freqs, stream=stream)
    return [*order, rows, out, *grads, turned, back, *caches]


def _step_inputs(seed, tokens=600):
    g = _gen(seed)
    bf = torch.bfloat16
    return dict(x=torch.randn(tokens, 512, generator=g).to(bf).to(DEV),
                experts=torch.randint(0, 16, (tokens, 8), generator=g).to(DEV),
                w=torch.rand(tokens, 8, generator=g).to(DEV),
                q=torch.randn(tokens, 8, 64, generator=g).to(bf).to(DEV),
                k=torch.randn(tokens, 2, 64, generator=g).to(bf).to(DEV),
                v=torch.randn(tokens, 2, 64, generator=g).to(bf).to(DEV),
                caches=[torch.zeros(tokens, 8, 2, 64, dtype=bf, device=DEV) for _ in range(2)],
                table=torch.randperm(tokens, generator=g)[:, None].to(torch.int32).to(DEV),
                positions=torch.randint(0, 8, (tokens,), generator=g).to(DEV),
                freqs=_freqs(32).to(DEV))


def test_on_another_stream():
    """Inputs made on the current stream just before, results read on it just after."""
    want = [t.clone() for t in _step(**_step_inputs(70))]
    side = torch.cuda.Stream()
    for how in (side, int(side.cuda_stream)):
        a = _step_inputs(70)
        x = a["x"].clone()
        for _ in range(20):  # keep the current stream busy ahead of the inputs
            x = torch.tanh(x @ torch.ones(512, 512, dtype=x.dtype, device=DEV))
        a["x"] = a["x"] + 0 * x.nan_to_num()
        got = _step(**a, stream=how)
        assert all(torch.equal(p, q) for p, q in zip([t.clone() for t in got], want))


def test_in_a_graph():
    """Captured once, replayed on other inputs, with eager work in between."""
    a = _step_inputs(71, tokens=900)  # 7200 choices: the sort of several workgroups
    for _ in range(2):
        _step(**a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(**a)
    for seed in (72, 73, 74, 75):
        b = _step_inputs(seed, tokens=900)
        want = [t.clone() for t in _step(**b)]
        for name, t in b.items():
            if name == "caches":
                for p in a["caches"]:
                    p.zero_()
            else:
                a[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), seed


def _training_step(x, experts, w, y, positions, freqs):
    order = bm.expert_order(experts, 16, align=4)
    q, k = bm.rotary((x.unflatten(1, (8, 64)), x.unflatten(1, (8, 64))), positions, freqs)
    rows = torch.tanh(bm.expert_gather((q + 0.5 * k).flatten(1), order))
    out = bm.expert_combine(rows, order, w)
    return (out, *torch.autograd.grad((out * y).sum(), (x, w)))


def test_a_training_step_in_a_graph():
    """Forward and backward passes captured together, replayed on other inputs
    with eager steps in between; no eager graph of the leaves is alive while
    the capture runs."""
    def inputs(seed):
        g = _gen(seed)
        return [torch.randn(300, 512, generator=g).to(DEV).requires_grad_(),
                torch.randint(-1, 16, (300, 4), generator=g).to(DEV),
                torch.rand(300, 4, generator=g).to(DEV).requires_grad_(),
                torch.randn(300, 512, generator=g).to(DEV),
                torch.randint(0, 5000, (300,), generator=g).to(DEV), _freqs(32).to(DEV)]
    a = inputs(80)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _training_step(*a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _training_step(*a)
    for seed in (81, 82, 83):
        b = inputs(seed)
        want = [t.detach().clone() for t in _training_step(*b)]
        with torch.no_grad():
            for t, u in zip(a, b):
                t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), seed


# --------------------------------------------------------------------------
# The example
# --------------------------------------------------------------------------

def test_the_example():
    """A layer that serves and trains through these calls: sums of at most 512
    terms in 32 bits, off by at most 512 roundings of the largest value."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "sparse_layer.py")
    spec = importlib.util.spec_from_file_location("sparse_layer", path)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    device = torch.device(DEV)
    with torch.no_grad():
        assert layer.serve(device, torch.float32, 70, 3)[0] <= 512 * U32
    assert layer.train(device, 70) <= 512 * U32
