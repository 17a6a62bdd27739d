"""A decoder layer with experts, its token rows moved by this library.

    python examples/sparse_layer.py [--tokens 512] [--steps 4]

runs one layer as a serving program and a training program use it:

* a prefill of several sequences of different lengths: keys and values go to a
  paged cache, keys and queries turned by their positions on the way, every
  sequence attends over its pages, and each token's experts are reached by
  expert_order, expert_gather and expert_combine;
* decoding steps of one token a sequence through the same calls;
* a training step, whose gradients flow through the gather, the combine and the
  rotary positions (three axes, as for video).

Each part is compared with a plain computation in 64 bits, and the largest
difference is printed.  Products and attention are torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bmmc_affine_index_amd as bm  # noqa: E402

HEADS, KV_HEADS, HEAD_DIM, PAGE = 8, 2, 64, 16
DIM, HIDDEN, EXPERTS, CHOICES = 512, 256, 16, 4


class Layer:
    """Weights of one layer and its paged cache."""

    def __init__(self, dtype, device, sequences, pages_each, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, device=device, generator=g) / shape[-2] ** 0.5
            return w.to(dtype)
        self.qkv = weight(DIM, (HEADS + 2 * KV_HEADS) * HEAD_DIM)
        self.out = weight(HEADS * HEAD_DIM, DIM)
        self.router = weight(DIM, EXPERTS).float()
        self.up, self.down = weight(EXPERTS, DIM, HIDDEN), weight(EXPERTS, HIDDEN, DIM)
        self.freqs = 10000.0 ** (-torch.arange(HEAD_DIM // 2, device=device, dtype=torch.float64) /
                                 (HEAD_DIM // 2))
        pages = sequences * pages_each
        # keys and values of a page next to each other
        cache = torch.zeros(pages, 2, PAGE, KV_HEADS, HEAD_DIM, device=device, dtype=dtype)
        self.k_cache, self.v_cache = cache[:, 0], cache[:, 1]
        self.table = torch.randperm(pages, device=device, generator=g).to(torch.int32).reshape(
            sequences, pages_each)

    def heads(self, x):
        """Views of one projection: queries, keys, values."""
        both = x @ self.qkv
        q, k, v = both.split([HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM], dim=1)
        return (q.unflatten(1, (HEADS, HEAD_DIM)), k.unflatten(1, (KV_HEADS, HEAD_DIM)),
                v.unflatten(1, (KV_HEADS, HEAD_DIM)))

    def attend(self, x, sequences, positions):
        """Attention of tokens over their sequences' pages; the tokens' own keys and values are
        appended first."""
        q, k, v = self.heads(x)
        q = bm.cache_append(k, v, self.k_cache, self.v_cache, self.table, positions,
                            sequences=sequences, freqs=self.freqs, q=q)
        outs = torch.empty_like(q)
        for s in range(self.table.shape[0]):
            mine = (sequences == s).nonzero().reshape(-1)
            if mine.numel():
                pages = self.table[s].long()
                keys = self.k_cache[pages].flatten(0, 1).float()
                values = self.v_cache[pages].flatten(0, 1).float()
                outs[mine] = attention(q[mine].float(), keys, values, positions[mine]).to(q.dtype)
        return outs.flatten(1) @ self.out

    def route(self, x):
        top, experts = (x.float() @ self.router).topk(CHOICES, dim=1)
        return experts.contiguous(), torch.softmax(top, dim=1)

    def experts(self, x, up, down):
        """The experts' products, each on its own rows."""
        experts, weights = self.route(x)
        order = bm.expert_order(experts, EXPERTS, align=8)
        rows = bm.expert_gather(x, order)
        ends = order.offsets.tolist()
        parts = [torch.nn.functional.silu(rows[a:b] @ up[e]) @ down[e]
                 for e, (a, b) in enumerate(zip(ends, ends[1:]))]
        parts.append(rows[ends[-1]:])  # rows past the last expert's, all padding
        return bm.expert_combine(torch.cat(parts), order, weights)

    def __call__(self, x, sequences, positions):
        x = x + self.attend(x, sequences, positions)
        return x + self.experts(x, self.up, self.down)


def attention(q, keys, values, positions):
    """q [T, H, D] over [S, Hk, D], each token up to its own position."""
    group = q.shape[1] // keys.shape[1]
    keys, values = (t.repeat_interleave(group, 1).transpose(0, 1) for t in (keys, values))
    scores = q.transpose(0, 1) @ keys.transpose(1, 2).contiguous() / q.shape[2] ** 0.5
    hidden = torch.arange(keys.shape[1], device=q.device) > positions[:, None]
    weights = torch.softmax(scores.masked_fill(hidden, float("-inf")), dim=2)
    return (weights @ values.contiguous()).transpose(0, 1)


# ---------------------------------------------------------------------------
# The same in 64 bits
# ---------------------------------------------------------------------------

def turned(x, angle):
    """The two halves of each head as complex numbers, turned by angle [T, pairs]."""
    z = torch.polar(torch.ones_like(angle), angle)[:, None, :] * torch.complex(*x.chunk(2, dim=2))
    return torch.cat([z.real, z.imag], dim=2)


def plain_experts(layer, x, experts, weights, up, down):
    out = torch.zeros_like(x)
    for e in range(EXPERTS):
        t, j = (experts == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ up[e]) @ down[e]
        out = out.index_add(0, t, y * weights[t, j][:, None])
    return out


def plain_layer(layer, x, route):
    """One whole sequence, without a cache; `route` is the layer's, in 32 bits."""
    wide = {n: getattr(layer, n).double() for n in ("qkv", "out", "up", "down")}
    x = x.double()
    q, k, v = (x @ wide["qkv"]).split([HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM,
                                       KV_HEADS * HEAD_DIM], dim=1)
    place = torch.arange(x.shape[0], device=x.device)
    angle = place[:, None].double() * layer.freqs
    q = turned(q.unflatten(1, (HEADS, HEAD_DIM)), angle)
    k = turned(k.unflatten(1, (KV_HEADS, HEAD_DIM)), angle)
    a = attention(q, k, v.unflatten(1, (KV_HEADS, HEAD_DIM)), place)
    x = x + a.flatten(1) @ wide["out"]
    return x + plain_experts(layer, x, *route(x), wide["up"], wide["down"])


def serve(device, dtype, tokens, steps):
    """A ragged prefill and decoding steps; the differences of the tokens from 64 bits, relative
    to the largest value: (the largest of all tokens, the one in the middle)."""
    lengths = [tokens, max(1, tokens // 3), 1]
    layer = Layer(dtype, device, len(lengths), (tokens + steps + PAGE) // PAGE)
    g = torch.Generator(device=device).manual_seed(1)
    xs = [torch.randn(n + steps, DIM, device=device, generator=g).to(dtype) for n in lengths]
    each = [torch.arange(n, device=device) for n in lengths]
    sequences = torch.cat([torch.full_like(p, s) for s, p in enumerate(each)]).to(torch.int32)
    got = list(layer(torch.cat([x[:n] for x, n in zip(xs, lengths)]), sequences,
                     torch.cat(each)).split(lengths))
    all_sequences = torch.arange(len(lengths), device=device, dtype=torch.int32)
    for i in range(steps):
        places = torch.tensor(lengths, device=device) + i
        new = layer(torch.stack([x[n + i] for x, n in zip(xs, lengths)]), all_sequences, places)
        got = [torch.cat([a, b[None]]) for a, b in zip(got, new)]
    off = []
    for x, y in zip(xs, got):
        def route(z):
            experts, weights = layer.route(z)
            return experts, weights.double()
        want = plain_layer(layer, x, route)
        off.append((y.double() - want).abs().amax(1) / want.abs().max())
    off = torch.cat(off)
    return float(off.max()), float(off.median())


def train(device, tokens):
    """Gradients of a step through rotary positions on three axes and through the experts, in 32
    bits; the largest difference from 64 bits, relative to the largest value."""
    layer = Layer(torch.float32, device, 1, 1)
    g = torch.Generator(device=device).manual_seed(2)
    x0 = torch.randn(tokens, DIM, device=device, generator=g)
    side = max(1, round(tokens ** (1 / 3)))
    i = torch.arange(tokens, device=device)
    positions = torch.stack([i // (side * side), i // side % side, i % side])
    axes = bm.rotary_axes([12, 10, 10], device=device)
    experts, weights = layer.route(x0)

    x, up, down, w = (t.detach().clone().requires_grad_() for t in (x0, layer.up, layer.down, weights))
    q, k = bm.rotary((x.unflatten(1, (HEADS, HEAD_DIM)), x.unflatten(1, (HEADS, HEAD_DIM)) * 0.5),
                     positions, layer.freqs, axes=axes)
    order = bm.expert_order(experts, EXPERTS, align=8)
    rows = bm.expert_gather((q * 0.7 + k).flatten(1), order)
    ends = order.offsets.tolist()
    parts = [torch.nn.functional.silu(rows[a:b] @ up[e]) @ down[e] for e, (a, b) in enumerate(zip(ends, ends[1:]))]
    y = bm.expert_combine(torch.cat(parts + [rows[ends[-1]:]]), order, w)
    got = torch.autograd.grad((y * y).sum(), (x, up, down, w))

    x, up, down, w = (t.detach().double().requires_grad_() for t in (x0, layer.up, layer.down, weights))
    angle = positions.double()[axes.long()].t() * layer.freqs
    z = turned(x.unflatten(1, (HEADS, HEAD_DIM)) * 0.7, angle) + \
        turned(x.unflatten(1, (HEADS, HEAD_DIM)) * 0.5, angle)
    y = plain_experts(layer, z.flatten(1), experts, w, up, down)
    want = torch.autograd.grad((y * y).sum(), (x, up, down, w))
    return max(float((a.double() - b).abs().max() / b.abs().max()) for a, b in zip(got, want))


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    device = torch.device("cuda", torch.cuda.current_device())
    with torch.no_grad():
        for dtype in (torch.float32, torch.bfloat16):
            # where a rounding turns a router's choice, a token differs by an expert
            print("serving in %s: tokens off by %.1e of the largest value at most, by %.1e in "
                  "the middle" % (dtype, *serve(device, dtype, a.tokens, a.steps)))
    print("training in float32: gradients off by %.1e of the largest" % train(device, a.tokens))


if __name__ == "__main__":
    main()
