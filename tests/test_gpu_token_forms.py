"""GPU tests of the calls on token rows in forms that are compiled apart: 8-bit
caches by type, pairing and width, and the sums of the weights' gradient.

Tolerances.  A rounding to a type is off by at most half a step, eps / 2 relative
to the value; n dependent 32-bit additions or fused multiply-adds are off by at
most n 2^-24 (1 + n 2^-24) times the sum of the terms' magnitudes."""
import math

import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]
U32 = 2.0 ** -24
F8 = torch.float8_e4m3fn
E4M3_MAX = 448.0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# --------------------------------------------------------------------------
# 8-bit caches
# --------------------------------------------------------------------------

def _turned(x, angle, interleaved):
    """x [T, H, D] turned by angle [T, P], and what 32-bit arithmetic may be off by:
    cosine and sine by 6 roundings, two products and their sum by 4 more, and
    the 64-bit angle by 4 2^-53 of itself on either side."""
    x, pairs = x.double(), angle.shape[-1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out, slack = x.clone(), torch.zeros_like(x)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    each = (x[..., lo].abs() + x[..., hi].abs()) * (10 * U32 + 2.0 ** -50 * angle.abs()[:, None])
    slack[..., lo], slack[..., hi] = each, each
    return out, slack


NARROW = [  # tokens, heads, size of k, of v, pairs, interleaved, heads before places
    (9, 2, 2, 1, 1, False, False), (9, 2, 2, 2, 1, True, False), (13, 3, 3, 3, 1, True, True),
    (33, 3, 16, 7, 3, False, False), (33, 3, 16, 7, 3, True, False), (21, 5, 96, 9, 6, True, False),
    (21, 5, 96, 9, 6, False, True), (14, 2, 20, 5, 8, True, False), (40, 4, 64, 64, 32, True, False),
    (64, 1, 128, 128, 64, False, True), (70, 3, 48, 40, 20, True, True),
    (17, 2, 130, 512, 65, True, False), (19, 2, 130, 100, 65, False, False),
    (25, 2, 24, 12, 0, False, False), (12, 1, 3, 17, 0, False, True), (1500, 2, 64, 64, 16, True, False)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", NARROW, ids=str)
def test_8_bit_caches(case, dtype):
    """Values are the nearest of their quotients, keys nearest to the turned ones'."""
    tokens, heads, dim, v_dim, pairs, interleaved, first = case
    page, g = 7, _gen(tokens + dim)
    width = -(-tokens // page)
    pages = width + 2
    table = torch.randperm(pages, generator=g)[None, :width].to(torch.int32)
    place = torch.randperm(tokens, generator=g)
    at, inside = table[0, place // page].long(), place % page
    k, q = (torch.randn(tokens, n, dim, generator=g).to(dtype) for n in (heads, 2 * heads))
    v = torch.randn(tokens, heads, v_dim, generator=g).to(dtype)
    special = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e4, -1e4, 0.0, -0.0, 2.0 ** -9,
                            2.0 ** -10, 464.0, 465.0, 17.0, 19.0]).to(dtype)
    n = min(special.numel(), tokens)
    v[:n, heads - 1, v_dim - 1] = special[:n]
    k_scale = torch.rand(heads, generator=g) * 0.1 + 0.01
    v_scale = torch.ones(1)

    def pool(d, seed):
        fill = torch.randn(pages, page, heads, d, generator=_gen(seed)).to(F8)
        if first:
            return fill, fill.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        return fill, fill.to(DEV)
    (k0, kc), (v0, vc) = pool(dim, 1), pool(v_dim, 2)
    more, turned, slack = {}, k.double(), torch.zeros(tokens, heads, dim, dtype=torch.float64)
    if pairs:
        freqs = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        angle = place.double()[:, None] * freqs
        more = {"freqs": freqs.to(DEV), "interleaved": interleaved, "q": q.to(DEV)}
        turned, slack = _turned(k, angle, interleaved)
    got_q = bm.cache_append(k.to(DEV), v.to(DEV), kc, vc, table.to(DEV), place.to(DEV),
                            sequences=torch.zeros(tokens, dtype=torch.int32, device=DEV),
                            k_scale=k_scale.to(DEV), v_scale=v_scale.to(DEV), **more)
    torch.cuda.synchronize()
    if pairs:
        want, q_slack = _turned(q, angle, interleaved)
        u, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny
        off = (got_q.cpu().double() - want).abs()
        assert bool((off <= q_slack * (1 + u) + u * want.abs() + u * tiny).all())

    # values: one quotient in 32 bits (by one, exact), then one rounding
    y = v.float()
    want = v0.view(torch.uint8).clone()
    want[at, inside] = torch.where(y.isnan(), y, y.clamp(-E4M3_MAX, E4M3_MAX)).to(F8).view(torch.uint8)
    got = vc.cpu().view(torch.uint8)
    nan = (want & 127) == 127
    assert torch.equal((got & 127) == 127, nan) and torch.equal(got[~nan], want[~nan])

    # keys: the 32-bit slack and the quotient's rounding, then half a step of 3
    # bits after the first, or half of 2^-9 among the subnormals
    turned, slack = turned / k_scale.double()[:, None], slack / k_scale.double()[:, None]
    slack = slack + U32 * turned.abs()
    want, may = k0.double(), torch.zeros(k0.shape, dtype=torch.float64)
    want[at, inside] = turned.clamp(-E4M3_MAX, E4M3_MAX)
    may[at, inside] = slack * (1 + 2.0 ** -4) + 2.0 ** -4 * want[at, inside].abs() + 2.0 ** -10
    assert bool(((kc.cpu().double() - want).abs() <= may).all())


# --------------------------------------------------------------------------
# The weights' gradient
# --------------------------------------------------------------------------

def _roundings(width, dtype):
    """On the way of one product to its sum: a lane takes whole vectors in turn,
    as many lanes as a power of two of them has, at most a wave, and the lanes
    are joined two by two."""
    n = 128 // torch.finfo(dtype).bits
    n = n if width >= n else 1
    vectors = -(-width // n)
    lanes = min(64, 1 << (vectors.bit_length() - 1))
    return -(-vectors // lanes) * n + int(math.log2(lanes)) + 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 3, 7, 8, 9, 65, 127, 136, 513, 1001, 2048, 2880, 4100, 8192])
def test_sums_of_the_weights_gradient(width, dtype):
    tokens, choices = 60, 5
    g = _gen(width)
    experts = torch.rand(tokens, 9, generator=g).topk(choices, dim=1).indices
    experts = torch.where(torch.rand(tokens, choices, generator=g) < 0.1, -1, experts)
    order = bm.expert_order(experts.contiguous().to(DEV), 9, align=4)
    rows = order.rows.cpu().long()
    x = torch.randn(order.slots.numel(), width, generator=g).to(dtype)
    grad = torch.randn(tokens, width, generator=g).to(dtype)
    w = torch.rand(tokens, choices, generator=g)
    got = bm.expert_combine_backward(grad.to(DEV), x.to(DEV), order, w.to(DEV))[1].cpu().double()
    terms = grad.double()[:, None] * x.double()[rows.clamp(min=0)] * (rows >= 0)[..., None]
    bound = _roundings(width, dtype) * U32 * terms.abs().sum(-1)
    assert bool(((got - terms.sum(-1)).abs() <= bound).all())
    assert not bool(got[rows < 0].any())
