"""The operators on token rows, as cases to be timed and checked.

Three groups of operators move rows of a language model's tokens to places
that only the data tells:

  * tokens sorted by expert and back: the order of the choices, the rows
    gathered in that order, the rows combined back into their tokens with the
    router's weights, and the gradients of both moves;
  * rotary positions with several axes, and their gradient;
  * keys and values appended to a paged cache, rotated on the way.

Where `own` is false, run() computes them with elementary torch operations in
32 bits (the angles in 64); where it is true, with the library's calls.
"""
import math

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _experts(name, op, tokens, choices, experts, dim, dtype, drop=0.0, align=1):
    return {"name": name, "op": op, "tokens": tokens, "choices": choices, "experts": experts,
            "dim": dim, "dtype": dtype, "drop": drop, "align": align}


def _rotary(name, tokens, q_heads, k_heads, head_dim, pairs, axes, dtype, interleaved=False,
            alternate=False, backward=False, start=0):
    return {"name": name, "op": "rotary", "tokens": tokens, "q_heads": q_heads,
            "k_heads": k_heads, "head_dim": head_dim, "pairs": pairs, "axes": axes,
            "dtype": dtype, "interleaved": interleaved, "alternate": alternate,
            "backward": backward, "start": start}


def _append(name, tokens, batch, context, page, q_heads, k_heads, head_dim, pairs, dtype,
            e4m3=False, heads_first=False, padded=0, axes=1):
    return {"name": name, "op": "append", "tokens": tokens, "batch": batch, "context": context,
            "page": page, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "pairs": pairs, "dtype": dtype, "e4m3": e4m3, "heads_first": heads_first,
            "padded": padded, "axes": axes}


def listed():
    return [
        # one decoding step of a small batch: the order and its rows, latency counts
        _experts("dispatch decode", "dispatch", 32, 8, 64, 2048, "bfloat16"),
        # a long prefill's tokens, each to 8 of 128 experts: the largest dispatch
        _experts("dispatch prefill", "dispatch", 16384, 8, 128, 4096, "bfloat16"),
        # one rank's share of the experts (half the choices are another rank's), an odd width,
        # each expert's rows padded to a product's tile
        _experts("dispatch share", "dispatch", 4099, 3, 60, 1001, "float32", drop=0.5, align=16),
        # one decoding step's way back
        _experts("combine decode", "combine", 17, 8, 64, 2048, "float16"),
        # the prefill's way back
        _experts("combine prefill", "combine", 16384, 8, 128, 4096, "bfloat16"),
        # a training step: gradients of the rows and of the router's weights
        _experts("combine backward", "combine_backward", 8192, 8, 64, 2048, "bfloat16"),
        # a training step: the gradient of the tokens, a width of whole vectors and a ragged count
        _experts("gather backward", "gather_backward", 8191, 6, 96, 1536, "bfloat16", drop=0.1),
        # a video prompt's queries and keys, time, height and width, views of the one projection
        _rotary("rotary video", 32768, 32, 8, 128, 64, 3, "bfloat16"),
        # a training step of an image tower: two axes in turn, adjacent pairs, an odd token count
        _rotary("rotary image backward", 5329, 16, 16, 72, 36, 2, "float32", interleaved=True,
                alternate=True, backward=True),
        # one decoding step of 64 sequences at their own lengths, four places of it padding
        _append("append decode", 64, 60, 1024, 16, 32, 8, 128, 64, "bfloat16", padded=4),
        # a long prefill in chunks of a ragged batch
        _append("append prefill", 32768, 12, 4096, 64, 32, 8, 128, 64, "bfloat16"),
        # a chunk into an 8-bit cache whose heads come before its places, part of the head rotated
        _append("append 8-bit", 1001, 7, 700, 32, 24, 4, 96, 32, "float16", e4m3=True,
                heads_first=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch", "combine", "combine_backward", "gather_backward",
                     "rotary", "rotary", "append", "append"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    size = 4 if dtype == "float32" else 2
    if op == "rotary" or op == "append":
        head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(16, 128)])
        k_heads = rng.choice([1, 2, 4, 8, 16])
        q_heads = k_heads * rng.choice([1, 2, 4, 5, 8])
        pairs = head_dim // 2 if rng.random() < 0.7 else max(1, head_dim // rng.choice([4, 8]))
        most = (1 << 28) // ((q_heads + 2 * k_heads) * head_dim * size)
        tokens = _log(rng, 1, max(1, min(32768, most)))
        if op == "rotary":
            axes = rng.choice([1, 2, 3, 3])
            return _strip(_rotary("", tokens, q_heads, k_heads, head_dim, max(pairs, axes), axes,
                                  dtype, interleaved=rng.random() < 0.4,
                                  alternate=rng.random() < 0.4, backward=rng.random() < 0.4,
                                  start=rng.choice([0, 0, _log(rng, 1, 1 << 20)])))
        batch = _log(rng, 1, min(tokens, 256))
        return _strip(_append("", tokens, batch, _log(rng, 1, 2048), rng.choice([1, 16, 32, 64, 48]),
                              q_heads, k_heads, head_dim, pairs, dtype,
                              e4m3=dtype != "float32" and rng.random() < 0.3,
                              heads_first=rng.random() < 0.4,
                              padded=rng.choice([0, 0, min(tokens - batch, rng.randint(0, 9))]),
                              axes=rng.choice([1, 1, 3]) if pairs >= 3 else 1))
    experts = rng.choice([8, 16, 60, 64, 128, 256, rng.randint(2, 384)])
    choices = rng.randint(1, min(10, experts))
    dim = rng.choice([512, 1024, 2048, 2880, 4096, 7168, _log(rng, 64, 8192)])
    # the backward pass both reads and writes its rows
    most = (1 << (29 if op == "combine_backward" else 30)) // (choices * dim * size)
    tokens = _log(rng, 1, max(1, min(32768, most)))
    padding = min(tokens * choices, experts) * 64 * dim * size
    return _strip(_experts("", op, tokens, choices, experts, dim, dtype,
                           drop=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]),
                           align=rng.choice([1, 1, 16, 64]) if padding < 1 << 28 else 1))


def _strip(case):
    return {k: v for k, v in case.items() if k != "name"}


def _rows(case):
    """Rows of the sorted order: one for each choice, and each expert's padding at its most."""
    n = case["tokens"] * case["choices"]
    return n + min(n, case["experts"]) * (case["align"] - 1)


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    t = case["tokens"]
    if case["op"] == "rotary":
        each = t * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        turned = t * (case["q_heads"] + case["k_heads"]) * 2 * case["pairs"]
        return {"bytes": 2 * each * size + 8 * t * case["axes"] + 8 * case["pairs"],
                "flops": 3 * turned}
    if case["op"] == "append":
        q = t * case["q_heads"] * case["head_dim"]
        kv = (t - case["padded"]) * 2 * case["k_heads"] * case["head_dim"]
        turned = t * (case["q_heads"] + case["k_heads"]) * 2 * case["pairs"]
        return {"bytes": 2 * q * size + kv * (size + (1 if case["e4m3"] else size)) +
                t * (12 + 8 * case["axes"]), "flops": 3 * turned}
    n, r, d = t * case["choices"], _rows(case), case["dim"]
    held = int(n * (1 - case["drop"]))
    if case["op"] == "dispatch":
        return {"bytes": 8 * n + 4 * (n + r + 2 * case["experts"] + 1) + (t + r) * d * size,
                "flops": 0}
    if case["op"] == "combine":
        return {"bytes": 8 * n + (held + t) * d * size, "flops": 2 * held * d}
    if case["op"] == "gather_backward":
        return {"bytes": 4 * n + (held + t) * d * size, "flops": held * d}
    return {"bytes": 16 * n + (t + held + r) * d * size, "flops": 3 * held * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _choose(case, g):
    """The router's choices, most wanted first, with experts that are wanted unequally; the
    choices of another rank's experts are -1."""
    t, e = case["tokens"], case["experts"]
    scores = torch.randn(t, e, device="cuda", generator=g)
    scores += torch.randn(e, device="cuda", generator=g)
    top, experts = scores.topk(case["choices"], dim=1)
    weights = torch.softmax(top, dim=1)
    if case["drop"]:
        away = torch.rand(experts.shape, device="cuda", generator=g) < case["drop"]
        experts = torch.where(away, torch.full_like(experts, -1), experts)
    return experts.contiguous(), weights.contiguous()


def _frequencies(pairs):
    return 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)


def _axis_of_pair(pairs, axes, alternate):
    """Pair -> axis: in turn, or one run of pairs for each axis (what is over goes to the first)."""
    i = torch.arange(pairs, device="cuda", dtype=torch.int32)
    if alternate:
        return i % axes
    each = pairs // axes
    return ((i - (pairs - each * axes)).clamp(min=0) // max(each, 1)).to(torch.int32)


def _grid(tokens, axes, start):
    """Positions of tokens laid out as time, height, width (or fewer axes), int64 [axes, tokens]."""
    i = torch.arange(tokens, device="cuda", dtype=torch.int64)
    side = max(1, int(math.isqrt(tokens)) if axes == 2 else int(round(tokens ** (1 / 3))))
    parts = [i] if axes == 1 else [i // side, i % side] if axes == 2 else \
        [i // (side * side), i // side % side, i % side]
    return torch.stack(parts) + start


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32).to(dtype)

    s = {"case": case}
    t = case["tokens"]
    if case["op"] in ("rotary", "append"):
        hq, hk, d = case["q_heads"], case["k_heads"], case["head_dim"]
        # the queries, keys and values are views of one projection's output
        both = normal(t, (hq + 2 * hk) * d)
        s["q"] = both[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = both[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = both[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["freqs"] = _frequencies(case["pairs"])
        if case["op"] == "rotary":
            s["axis"] = _axis_of_pair(case["pairs"], case["axes"], case["alternate"])
            s["positions"] = _grid(t, case["axes"], case["start"])
            return s
        s["axis"] = _axis_of_pair(case["pairs"], case["axes"], True)
        batch, page = case["batch"], case["page"]
        # each sequence holds a length of its own and gets at least one of the new tokens
        new = t - case["padded"]
        more = torch.randint(0, batch, (new - batch,), device="cuda", generator=g)
        owner = torch.cat([torch.arange(batch, device="cuda"), more]).sort().values
        held = torch.randint(0, case["context"] + 1, (batch,), device="cuda", generator=g)
        first = torch.searchsorted(owner, torch.arange(batch, device="cuda"))
        place = held[owner] + torch.arange(new, device="cuda") - first[owner]
        pad = torch.full((case["padded"],), -1, device="cuda", dtype=torch.int64)
        s["sequences"] = torch.cat([owner, pad]).to(torch.int32)
        s["positions"] = torch.cat([place, torch.zeros_like(pad)]).to(torch.int32)
        # as long a table as the longest sequence can need, its pages in no order
        wide = (case["context"] + new - batch + 1 + page - 1) // page
        pages = (batch * case["context"] + new) // page + 2 * batch
        s["table"] = _table(held, owner, batch, wide, page, pages, g)
        shape = (pages, case["k_heads"], page, d) if case["heads_first"] else \
            (pages, page, case["k_heads"], d)
        kinds = torch.float8_e4m3fn if case["e4m3"] else dtype
        s["k_cache"], s["v_cache"] = normal(*shape).to(kinds), normal(*shape).to(kinds)
        if case["e4m3"]:
            s["k_scale"] = 0.01 + 0.02 * torch.rand(hk, device="cuda", generator=g)
            s["v_scale"] = 0.01 + 0.02 * torch.rand(hk, device="cuda", generator=g)
        if case["axes"] > 1:
            s["turns"] = torch.randint(0, 2048, (case["axes"], t), device="cuda", generator=g)
        return s
    s["experts"], s["weights"] = _choose(case, g)
    if case["op"] == "dispatch":
        s["x"] = normal(t, case["dim"])
        return s
    s["order"] = _order(s["experts"], case["experts"], case["align"])
    if case["op"] == "combine_backward":
        s["grad"] = normal(t, case["dim"])
    s["rows"] = normal(_rows(case), case["dim"])
    return s


def _table(held, owner, batch, wide, page, pages, g):
    """int32 [batch, wide]: pages handed out in a random order to the places that the sequences
    reach, -1 where a sequence has no page."""
    length = held + torch.zeros_like(held).index_add(0, owner, torch.ones_like(owner))
    need = (length + page - 1) // page
    before = need.cumsum(0) - need
    column = torch.arange(wide, device="cuda")
    shuffled = torch.randperm(pages, device="cuda", generator=g)
    at = (before[:, None] + column).clamp(max=pages - 1)
    return torch.where(column < need[:, None], shuffled[at], -1).to(torch.int32).contiguous()


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _order(experts, count, align):
    """Choices sorted by expert, stable: (offsets [E+1], counts [E], row of each choice [T, K],
    choice of each row [R]); -1 for a choice that is dropped and for a row of padding."""
    flat = experts.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < count), flat, count)
    inorder, choice = torch.sort(key, stable=True)
    starts = torch.searchsorted(inorder, torch.arange(count + 1, device=flat.device))
    counts = starts[1:] - starts[:-1]
    offsets = torch.zeros(count + 1, dtype=torch.long, device=flat.device)
    offsets[1:] = ((counts + align - 1) // align * align).cumsum(0)
    row = offsets[inorder] + torch.arange(n, device=flat.device) - starts[inorder]
    held = inorder < count
    capacity = n + min(n, count) * (align - 1)
    rows = torch.empty_like(flat)
    rows[choice] = torch.where(held, row, -1)
    slots = torch.full((capacity + 1,), -1, dtype=torch.long, device=flat.device)
    slots[torch.where(held, row, capacity)] = choice
    return (offsets.int(), counts.int(), rows.reshape(experts.shape).int(), slots[:capacity].int())


def _gather(x, slots, choices):
    moved = x[slots.clamp(min=0).long() // choices]
    return torch.where(slots[:, None] >= 0, moved, torch.zeros((), dtype=x.dtype, device=x.device))


def _picked(rows, where):
    """float32 [T, K, D]: the row of each choice, zeros for a dropped one."""
    got = rows[where.clamp(min=0).long()].float()
    return got.masked_fill_(where[..., None] < 0, 0.0)


def _turned(x, angle, interleaved, backward):
    """x [T, H, D] turned by angle [T, pairs] (64 bits); float32."""
    pairs = angle.shape[1]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s = -s if backward else s
    x = x.float()
    out = x.clone()
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    return out


def _plain_append(s):
    case = s["case"]
    turns = s["turns"] if "turns" in s else s["positions"][None]
    angle = turns.double()[s["axis"].long()].t() * s["freqs"]
    q = _turned(s["q"], angle, False, False).to(s["q"].dtype)
    k, v = _turned(s["k"], angle, False, False), s["v"].float()
    if case["e4m3"]:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    k, v = k.to(s["k_cache"].dtype), v.to(s["v_cache"].dtype)
    # a padded token repeats the write of the first token that is none
    t = torch.arange(case["tokens"], device="cuda")
    held = s["sequences"] >= 0
    t = torch.where(held, t, held.int().argmax())
    place = s["positions"][t].long()
    at = s["table"][s["sequences"][t].long(), place // case["page"]].long()
    inside = place % case["page"]
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[k.element_size()]
    kc, vc = s["k_cache"].view(bits), s["v_cache"].view(bits)
    if case["heads_first"]:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kc[at, inside] = k.view(bits)[t]
    vc[at, inside] = v.view(bits)[t]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        offsets, counts, rows, slots = _order(s["experts"], case["experts"], case["align"])
        return {"offsets": offsets, "counts": counts, "rows": rows, "slots": slots,
                "x": _gather(s["x"], slots, case["choices"])}
    if op == "combine":
        got = _picked(s["rows"], s["order"][2])
        return (got * s["weights"][..., None]).sum(1).to(s["rows"].dtype)
    if op == "gather_backward":
        return _picked(s["rows"], s["order"][2]).sum(1).to(s["rows"].dtype)
    if op == "combine_backward":
        slots, where = s["order"][3], s["order"][2]
        g = s["grad"].float()
        weighed = g[slots.clamp(min=0).long() // case["choices"]]
        weighed *= s["weights"].reshape(-1)[slots.clamp(min=0).long()][:, None]
        weighed.masked_fill_(slots[:, None] < 0, 0.0)
        dots = (_picked(s["rows"], where) * g[:, None]).sum(-1)
        return {"rows": weighed.to(s["rows"].dtype), "weights": dots}
    if op == "rotary":
        angle = s["positions"].double()[s["axis"].long()].t() * s["freqs"]
        kind = (case["interleaved"], case["backward"])
        return {"q": _turned(s["q"], angle, *kind).to(s["q"].dtype),
                "k": _turned(s["k"], angle, *kind).to(s["k"].dtype)}
    return _plain_append(s)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import bmmc_affine_index_amd as bm
    case, op = s["case"], s["case"]["op"]
    if op == "dispatch":
        order = bm.expert_order(s["experts"], case["experts"], align=case["align"])
        return {"offsets": order.offsets, "counts": order.counts, "rows": order.rows,
                "slots": order.slots, "x": bm.expert_gather(s["x"], order)}
    if op == "rotary":
        turn = bm.rotary_backward if case["backward"] else bm.rotary
        q, k = turn((s["q"], s["k"]), s["positions"], s["freqs"], axes=s["axis"],
                    interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "append":
        kc, vc = s["k_cache"], s["v_cache"]
        if case["heads_first"]:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        q = bm.cache_append(s["k"], s["v"], kc, vc, s["table"], s["positions"],
                            sequences=s["sequences"], freqs=s["freqs"], axes=s["axis"],
                            turns=s.get("turns"), q=s["q"], k_scale=s.get("k_scale"),
                            v_scale=s.get("v_scale"))
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    order = bm.ExpertOrder(*s["order"])
    if op == "combine":
        return bm.expert_combine(s["rows"], order, s["weights"])
    if op == "gather_backward":
        return bm.expert_gather_backward(s["rows"], order)
    rows, weights = bm.expert_combine_backward(s["grad"], s["rows"], order, s["weights"])
    return {"rows": rows, "weights": weights}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_order(experts, count, align):
    """Expert by expert: its choices in increasing order take the next rows."""
    flat = experts.reshape(-1)
    n = flat.numel()
    capacity = n + min(n, count) * (align - 1)
    rows = torch.full((n,), -1, dtype=torch.long, device=flat.device)
    slots = torch.full((capacity,), -1, dtype=torch.long, device=flat.device)
    offsets, counts, at = [0], [], 0
    for e in range(count):
        mine = (flat == e).nonzero().reshape(-1)
        rows[mine] = at + torch.arange(mine.numel(), device=flat.device)
        slots[at:at + mine.numel()] = mine
        counts.append(mine.numel())
        at += -(-mine.numel() // align) * align
        offsets.append(at)
    return offsets, counts, rows.reshape(experts.shape), slots


def _exact_turn(x, turns, s, case, back=1.0):
    """Each pair as one complex number times exp(i angle)."""
    x = x.double().clone()
    pairs = case["pairs"]
    angle = torch.stack([turns[int(a)].double() * f for a, f in
                         zip(s["axis"].tolist(), s["freqs"].tolist())], dim=-1) * back
    unit = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    head = x[..., :2 * pairs]
    if case.get("interleaved"):
        z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * unit
        x[..., :2 * pairs] = torch.stack([z.real, z.imag], -1).flatten(-2)
    else:
        z = torch.complex(head[..., :pairs].contiguous(), head[..., pairs:].contiguous()) * unit
        x[..., :2 * pairs] = torch.cat([z.real, z.imag], -1)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        back = -1.0 if case["backward"] else 1.0
        return {n: _exact_turn(s[n], s["positions"], s, case, back) for n in ("q", "k")}
    if op == "append":
        turns = s["turns"] if "turns" in s else s["positions"].unsqueeze(0)
        out = {"q": _exact_turn(s["q"], turns, s, case)}
        seqs, places, table = (s[n].tolist() for n in ("sequences", "positions", "table"))
        new = [t for t in range(case["tokens"]) if seqs[t] >= 0]
        pages = torch.tensor([table[seqs[t]][places[t] // case["page"]] for t in new],
                             device="cuda")
        inside = torch.tensor([places[t] % case["page"] for t in new], device="cuda")
        new = torch.tensor(new, device="cuda")
        for n, x in (("k", _exact_turn(s["k"], turns, s, case)), ("v", s["v"].double())):
            if case["e4m3"]:
                x = (x / s[n + "_scale"].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
            cache = s[n + "_cache"].double()
            if case["heads_first"]:
                cache[pages, :, inside] = x[new]
            else:
                cache[pages, inside] = x[new]
            out[n + "_cache"] = cache
        return out
    offsets, counts, rows, slots = _exact_order(s["experts"], case["experts"], case["align"])
    k = case["choices"]
    if op == "dispatch":
        x = torch.zeros(slots.numel(), case["dim"], dtype=torch.float64, device="cuda")
        held = (slots >= 0).nonzero().reshape(-1)
        x[held] = s["x"].double()[slots[held] // k]
        whole = {"offsets": torch.tensor(offsets), "counts": torch.tensor(counts), "rows": rows,
                 "slots": slots}
        return {**whole, "x": x}
    if op in ("combine", "gather_backward"):
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (rows[:, j] >= 0).nonzero().reshape(-1)
            w = s["weights"][t, j].double()[:, None] if op == "combine" else 1.0
            out[t] += s["rows"][rows[t, j]].double() * w
        return out
    g = s["grad"].double()
    grad_rows = torch.zeros(slots.numel(), case["dim"], dtype=torch.float64, device="cuda")
    grad_weights = torch.zeros(case["tokens"], k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (rows[:, j] >= 0).nonzero().reshape(-1)
        grad_rows[rows[t, j]] = g[t] * s["weights"][t, j].double()[:, None]
        grad_weights[t, j] = (g[t] * s["rows"][rows[t, j]].double()).sum(1)
    return {"rows": grad_rows, "weights": grad_weights}
