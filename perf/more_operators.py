"""What a decoder layer with experts over a paged cache needs next to its moved rows, as cases to
be timed and checked.

Three groups of operators:

  * attention of new tokens, one or a chunk for each sequence, over a paged cache;
  * a cache in 8 bits whose scales are made as it is written, and a cache read back;
  * the balance loss of a router with the counts of its experts, and its gradient.

Where `own` is false, run() computes them with elementary torch operations in 32 bits (the angles
in 64); where it is true, with the library's calls.
"""
import math

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attend(name, tokens, batch, context, page, q_heads, k_heads, head_dim, v_dim, dtype,
            narrow="no", window=0, heads_first=False, padded=0):
    return {"name": name, "op": "attend", "tokens": tokens, "batch": batch, "context": context,
            "page": page, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "v_dim": v_dim, "dtype": dtype, "narrow": narrow, "window": window,
            "heads_first": heads_first, "padded": padded}


def _quantize(name, tokens, batch, context, page, q_heads, k_heads, head_dim, v_dim, pairs, dtype,
              interleaved=False, heads_first=False, padded=0):
    return {"name": name, "op": "quantize", "tokens": tokens, "batch": batch, "context": context,
            "page": page, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "v_dim": v_dim, "pairs": pairs, "dtype": dtype, "interleaved": interleaved,
            "heads_first": heads_first, "padded": padded}


def _read(name, tokens, batch, page, k_heads, head_dim, v_dim, dtype, narrow, heads_first=False,
          padded=0):
    return {"name": name, "op": "read", "tokens": tokens, "batch": batch, "page": page,
            "k_heads": k_heads, "head_dim": head_dim, "v_dim": v_dim, "dtype": dtype,
            "narrow": narrow, "heads_first": heads_first, "padded": padded}


def _balance(name, tokens, choices, experts, dtype, masked=0.0):
    return {"name": name, "op": "balance", "tokens": tokens, "choices": choices,
            "experts": experts, "dtype": dtype, "masked": masked}


def listed():
    return [
        # a decoding step of a few short sequences
        _attend("attend decode small", 16, 16, 1024, 16, 32, 8, 128, 128, "bfloat16"),
        # a decoding step of a full batch at lengths from short to long
        _attend("attend decode", 64, 64, 8192, 64, 32, 8, 128, 128, "bfloat16"),
        # the same from an 8-bit cache with a scale for each row, heads before places
        _attend("attend decode 8-bit", 128, 128, 4096, 32, 24, 4, 96, 96, "float16", narrow="row",
                heads_first=True),
        # drafted tokens of each sequence checked in one step, over the last keys only; padding
        # behind the last sequence
        _attend("attend drafts", 156, 32, 3000, 16, 16, 2, 64, 64, "float16", window=1024,
                padded=4),
        # a prompt's chunks of several sequences, some of them far into their context
        _attend("attend prefill", 8192, 4, 2048, 64, 32, 8, 128, 128, "bfloat16"),
        # a chunk in 32 bits, a head for each head, an odd number of tokens and of elements
        _attend("attend chunk fp32", 777, 3, 1500, 48, 10, 10, 80, 72, "float32"),
        # one decoding step into an 8-bit cache, four places of it padding
        _quantize("quantize decode", 64, 60, 1024, 16, 32, 8, 128, 128, 64, "bfloat16", padded=4),
        # a long prefill in chunks, part of each head turned
        _quantize("quantize prefill", 16384, 12, 4096, 64, 24, 8, 128, 96, 32, "bfloat16"),
        # places of an 8-bit cache read back for a prefix that is used again
        _read("read prefix", 40001, 9, 64, 8, 128, 128, "bfloat16", "row"),
        # a short read from a cache of the inputs' type, with padding
        _read("read short", 300, 5, 16, 4, 96, 64, "float16", "no", heads_first=True, padded=12),
        # the router of a small batch, its padding not counted
        _balance("balance small", 257, 4, 60, "float32", masked=0.1),
        # the router of a training step
        _balance("balance training", 65536, 8, 256, "float32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "quantize", "quantize", "read",
                     "balance"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "balance":
        experts = rng.choice([8, 16, 60, 64, 128, 256, rng.randint(2, 512)])
        tokens = _log(rng, 1, min(65536, (1 << 24) // experts))
        return _strip(_balance("", tokens, rng.randint(1, min(10, experts)), experts, dtype,
                               masked=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.5), 2)])))
    page = rng.choice([1, 16, 32, 64, 48])
    first = rng.random() < 0.4
    k_heads = rng.choice([1, 2, 4, 8])
    head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256, rng.randint(17, 256)])
    v_dim = head_dim if rng.random() < 0.7 else rng.choice([64, 128, rng.randint(17, 256)])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "attend":
        context = _log(rng, 1, 8192)
        # a chunk for each sequence, or one token; the scores of all of them fit 2^28
        batch = _log(rng, 1, max(1, min(128, (1 << 19) // context)))
        most = (1 << 27) // (batch * k_heads * group * (context + 64))
        each = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(1024, most)))
        tokens = batch * each + (rng.randint(0, each - 1) if each > 1 else 0)
        return _strip(_attend("", tokens, batch, context, page, k_heads * group, k_heads, head_dim,
                              v_dim, dtype, narrow=rng.choice(["no", "no", "head", "row"]),
                              window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), heads_first=first,
                              padded=rng.choice([0, 0, rng.randint(1, 9)])))
    size = 4 if dtype == "float32" else 2
    if op == "quantize":
        most = (1 << 27) // ((k_heads * group + 2 * k_heads) * max(head_dim, v_dim) * size)
        tokens = _log(rng, 1, max(1, min(32768, most)))
        pairs = head_dim // 2 if rng.random() < 0.7 else max(1, head_dim // rng.choice([4, 8]))
        return _strip(_quantize("", tokens, _log(rng, 1, min(tokens, 256)), _log(rng, 1, 2048),
                                page, k_heads * group, k_heads, head_dim, v_dim, pairs, dtype,
                                interleaved=rng.random() < 0.4, heads_first=first,
                                padded=rng.choice([0, 0, rng.randint(1, 9)])))
    tokens = _log(rng, 1, max(1, min(65536, (1 << 27) // (2 * k_heads * max(head_dim, v_dim) * size))))
    return _strip(_read("", tokens, _log(rng, 1, min(tokens, 64)), page, k_heads, head_dim, v_dim,
                        dtype, rng.choice(["no", "head", "row", "row"]), heads_first=first,
                        padded=rng.choice([0, 0, rng.randint(1, 9)])))


def _strip(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """(new tokens, keys in the cache with them) of each sequence, fixed by the case: contexts from
    short to long, chunks of unequal size."""
    batch, tokens = case["batch"], case["tokens"]
    weights = [2 + 7 * b % 5 for b in range(batch)] if tokens > batch else [1] * batch
    new, left = [], tokens - batch
    for b in range(batch):
        share = left if b + 1 == batch else (tokens - batch) * weights[b] // sum(weights)
        new.append(1 + share)
        left -= share
    held = [case["context"] * (b + 1) // batch for b in range(batch)]
    return [(n, h + n) for n, h in zip(new, held)]


def _pairs(n, length, window):
    """Keys that the n last of `length` places see, summed."""
    if not window:
        return n * length - n * (n - 1) // 2
    first = length - n + 1
    if first >= window:
        return n * window
    short = min(length, window - 1)
    return (first + short) * (short - first + 1) // 2 + (length - short) * window


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    t = case["tokens"]
    if case["op"] == "balance":
        e = case["experts"]
        return {"bytes": 3 * t * e * size + 8 * t * case["choices"] + 2 * t + 12 * e,
                "flops": 12 * t * e}
    hk, dk, dv = case["k_heads"], case["head_dim"], case["v_dim"]
    if case["op"] == "attend":
        hq, window = case["q_heads"], case["window"]
        pairs, keys = 0, 0
        for n, length in _lengths(case):
            pairs += _pairs(n, length, window)
            keys += min(length, window + n - 1) if window else length
        one = 1 if case["narrow"] != "no" else size
        more = 8 * keys * hk if case["narrow"] == "row" else 0
        return {"bytes": keys * hk * (dk + dv) * one + more + t * hq * (dk + dv) * size,
                "flops": 2 * pairs * hq * (dk + dv)}
    if case["op"] == "quantize":
        hq = case["q_heads"]
        return {"bytes": 2 * t * hq * dk * size + t * hk * ((dk + dv) * (size + 1) + 8) + 20 * t,
                "flops": 6 * t * (hq + hk) * case["pairs"] + 2 * t * hk * (dk + dv)}
    one = 1 if case["narrow"] != "no" else size
    more = 8 * t * hk if case["narrow"] == "row" else 0
    return {"bytes": t * hk * (dk + dv) * (size + one) + more + 12 * t,
            "flops": t * hk * (dk + dv) if case["narrow"] != "no" else 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(g, dtype, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32).to(dtype)


def _table(lengths, wide, page, g):
    """int32 [batch, wide]: pages handed out in a random order to the places that the sequences
    reach, -1 where a sequence has no page; and the number of pages, a few of them nobody's."""
    need = (lengths + page - 1) // page
    pages = int(need.sum()) + 3
    before = need.cumsum(0) - need
    column = torch.arange(wide, device="cuda")
    shuffled = torch.randperm(pages, device="cuda", generator=g)
    at = (before[:, None] + column).clamp(max=pages - 1)
    return torch.where(column < need[:, None], shuffled[at], -1).to(torch.int32), pages


def _pool(case, pages, dim, kind, g):
    """A cache's storage as [pages, places, heads, dim], its heads before its places in memory
    where the case says so."""
    shape = (pages, case["k_heads"], case["page"], dim) if case["heads_first"] else \
        (pages, case["page"], case["k_heads"], dim)
    pool = _normal(g, torch.float32, *shape)
    if kind == E4M3:
        pool = (pool * 100.0).clamp_(-E4M3_MAX, E4M3_MAX)
    pool = pool.to(kind)
    return pool.transpose(1, 2) if case["heads_first"] else pool


def _scales(case, pages, g):
    """None, a scale for each head, or one for each row of the cache."""
    if case["narrow"] == "no":
        return None
    shape = (case["k_heads"],) if case["narrow"] == "head" else \
        (pages, case["page"], case["k_heads"])
    return 0.005 + 0.01 * torch.rand(*shape, device="cuda", generator=g)


def _sequences(case, g):
    """The case's sequences in an order of the seed: new tokens and lengths [batch], int64."""
    both = torch.tensor(_lengths(case), device="cuda")
    return both[torch.randperm(case["batch"], device="cuda", generator=g)].unbind(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "balance":
        t, e = case["tokens"], case["experts"]
        # experts that are wanted unequally
        logits = _normal(g, torch.float32, t, e) + _normal(g, torch.float32, e)
        s["logits"] = logits.to(dtype)
        s["choices"] = logits.topk(case["choices"], dim=1).indices.contiguous()
        s["mask"] = torch.rand(t, device="cuda", generator=g) >= case["masked"] \
            if case["masked"] else None
        s["grad"] = torch.full((), 0.01, device="cuda")
        return s
    hk, dk, dv = case["k_heads"], case["head_dim"], case["v_dim"]
    if case["op"] == "read":
        # every place once, of sequences that hold as many places each
        each = (case["tokens"] + case["batch"] - 1) // case["batch"]
        lengths = torch.full((case["batch"],), each, device="cuda")
    else:
        new, lengths = _sequences(case, g)
    wide = (max(n for _, n in _lengths(case)) if case["op"] != "read" else each) // case["page"] + 2
    s["table"], pages = _table(lengths, wide, case["page"], g)
    narrow = case["op"] == "quantize" or case["narrow"] != "no"
    s["k_cache"] = _pool(case, pages, dk, E4M3 if narrow else dtype, g)
    s["v_cache"] = _pool(case, pages, dv, E4M3 if narrow else dtype, g)
    pad = case["padded"]
    if case["op"] == "attend":
        s["k_scale"], s["v_scale"] = _scales(case, pages, g), _scales(case, pages, g)
        # the queries are a view of one projection's output
        both = _normal(g, dtype, case["tokens"] + pad, (case["q_heads"] + 2) * dk)
        s["q"] = both[:, :case["q_heads"] * dk].unflatten(1, (case["q_heads"], dk))
        s["starts"] = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)]).to(torch.int32)
        s["lengths"] = lengths.to(torch.int32)
        # what a program that plans its steps knows of them
        s["longest"] = max(n for _, n in _lengths(case))
        s["most"] = max(n for n, _ in _lengths(case))
        return s
    t = case["tokens"]
    if case["op"] == "read":
        at = torch.arange(t, device="cuda")
        sequences, positions = at // each, at % each
        s["k_scale"], s["v_scale"] = _scales(case, pages, g), _scales(case, pages, g)
    else:
        sequences = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), new,
                                            output_size=t)
        ends = new.cumsum(0)
        positions = (lengths - ends)[sequences] + torch.arange(t, device="cuda")
        hq = case["q_heads"]
        both = _normal(g, dtype, t + pad, (hq + hk) * dk + hk * dv)
        s["q"] = both[:, :hq * dk].unflatten(1, (hq, dk))
        s["k"] = both[:, hq * dk:(hq + hk) * dk].unflatten(1, (hk, dk))
        s["v"] = both[:, (hq + hk) * dk:].unflatten(1, (hk, dv))
        s["freqs"] = 10000.0 ** (-torch.arange(case["pairs"], device="cuda", dtype=torch.float64) /
                                 case["pairs"])
        s["k_scale"], s["v_scale"] = (0.5 + torch.rand(pages, case["page"], hk, device="cuda",
                                                       generator=g) for _ in range(2))
    nowhere = torch.full((pad,), -1, device="cuda")
    s["sequences"] = torch.cat([sequences, nowhere]).to(torch.int32)
    s["positions"] = torch.cat([positions, torch.zeros_like(nowhere)]).to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _wide(rows, scale, page, place):
    """Rows of a cache in 32 bits, by their scales; page and place of any shape."""
    rows = rows.float()
    if scale is None:
        return rows
    return rows * (scale[page, place] if scale.dim() == 3 else scale)[..., None]


def _plain_attend(s):
    """All sequences next to each other, each padded to the longest."""
    case, q = s["case"], s["q"]
    batch, hk = case["batch"], case["k_heads"]
    group, most, longest = case["q_heads"] // hk, s["most"], s["longest"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    new = starts[1:] - starts[:-1]
    key = torch.arange(longest, device=q.device)
    page = s["table"][:, key // case["page"]].long().clamp(min=0)
    place = (key % case["page"]).expand(batch, -1)
    k = _wide(s["k_cache"][page, place], s["k_scale"], page, place).permute(0, 2, 3, 1).contiguous()
    v = _wide(s["v_cache"][page, place], s["v_scale"], page, place).transpose(1, 2).contiguous()
    i = torch.arange(most, device=q.device)
    rows = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    mine = q[rows].float().unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).reshape(
        batch, hk, most * group, -1)
    scores = torch.matmul(mine, k).mul_(case["head_dim"] ** -0.5).unflatten(2, (most, group))
    position = (lengths - new)[:, None] + i
    hidden = key > position[..., None]
    if case["window"]:
        hidden |= key <= position[..., None] - case["window"]
    scores.masked_fill_(hidden[:, None, :, None], float("-inf"))
    scores -= scores.amax(-1, keepdim=True)
    scores = scores.exp_().flatten(2, 3)
    got = torch.matmul(scores, v) / scores.sum(-1, keepdim=True)
    got = got.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    out = torch.zeros(q.shape[0], case["q_heads"], case["v_dim"], dtype=q.dtype, device=q.device)
    held = i < new[:, None]
    out[rows[held]] = got[held].to(q.dtype)
    return out


def _turned(x, angle, interleaved):
    """x [T, H, D] turned by angle [T, pairs] (64 bits); float32."""
    pairs = angle.shape[1]
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = x.float()
    out = x.clone()
    lo = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    hi = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    return out


def _homes(s):
    """Page and place of each token that has one; those tokens."""
    held = (s["sequences"] >= 0).nonzero().reshape(-1)
    positions = s["positions"][held].long()
    page = s["table"][s["sequences"][held].long(), positions // s["case"]["page"]].long()
    return held, page, positions % s["case"]["page"]


def _put(cache, scales, x, page, place):
    scale = x.abs().amax(-1) / E4M3_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    x = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    cache.view(torch.uint8)[page, place] = x.view(torch.uint8)
    scales[page, place] = scale


def _plain_quantize(s):
    angle = s["positions"].double()[:, None] * s["freqs"]
    q = _turned(s["q"], angle, s["case"]["interleaved"]).to(s["q"].dtype)
    k = _turned(s["k"], angle, s["case"]["interleaved"])
    held, page, place = _homes(s)
    _put(s["k_cache"], s["k_scale"], k[held], page, place)
    _put(s["v_cache"], s["v_scale"], s["v"][held].float(), page, place)
    return q


def _plain_read(s):
    dtype, case = TYPES[s["case"]["dtype"]], s["case"]
    held, page, place = _homes(s)
    t = s["sequences"].shape[0]
    k = torch.zeros(t, case["k_heads"], case["head_dim"], dtype=dtype, device=held.device)
    v = torch.zeros(t, case["k_heads"], case["v_dim"], dtype=dtype, device=held.device)
    k[held] = _wide(s["k_cache"][page, place], s["k_scale"], page, place).to(dtype)
    v[held] = _wide(s["v_cache"][page, place], s["v_scale"], page, place).to(dtype)
    return k, v


def _plain_balance(s):
    x, choices, mask = s["logits"].float(), s["choices"], s["mask"]
    t, e = x.shape
    p = (x - x.amax(1, keepdim=True)).exp_()
    p /= p.sum(1, keepdim=True)
    one = torch.ones(t, device=x.device) if mask is None else mask.float()
    counted = one.sum()
    hits = torch.zeros_like(x).scatter_add_(1, choices, one[:, None].expand(choices.shape))
    counts = hits.sum(0, dtype=torch.float64)
    slope = (counts * e / (counted.double() ** 2 * choices.shape[1])).float()
    mean = (p * one[:, None]).sum(0)
    loss = (slope * mean).sum()
    grad = s["grad"] * one[:, None] * p * (slope - (p * slope).sum(1, keepdim=True))
    return loss, counts.to(torch.int32), grad.to(s["logits"].dtype)


def run(s):
    got = _run_own(s) if own else {"attend": _plain_attend, "quantize": _plain_quantize,
                                   "read": _plain_read, "balance": _plain_balance}[s["case"]["op"]](s)
    op = s["case"]["op"]
    if op == "attend":
        return got
    if op == "read":
        return {"k": got[0], "v": got[1]}
    if op == "balance":
        return {"loss": got[0], "counts": got[1], "grad": got[2]}
    return {"q": got, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import bmmc_affine_index_amd as bm
    op = s["case"]["op"]
    if op == "attend":
        return bm.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                  starts=s["starts"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                  window=s["case"]["window"])
    if op == "quantize":
        return bm.cache_quantize(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                                 s["v_scale"], s["table"], s["positions"],
                                 sequences=s["sequences"], freqs=s["freqs"],
                                 interleaved=s["case"]["interleaved"], q=s["q"])
    if op == "read":
        return bm.cache_read(s["k_cache"], s["v_cache"], s["table"], s["positions"],
                             sequences=s["sequences"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], dtype=TYPES[s["case"]["dtype"]])
    balance = bm.expert_balance(s["logits"], s["choices"], mask=s["mask"])
    grad = bm.expert_balance_backward(s["grad"], s["logits"], balance.slopes, mask=s["mask"])
    return balance.loss, balance.counts, grad


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, name, page, place):
    rows = s[name + "_cache"][page, place].double()
    scale = s[name + "_scale"]
    if scale is None:
        return rows
    scale = scale.double()
    return rows * (scale[page, place].unsqueeze(-1) if scale.dim() == 3 else scale.reshape(1, -1, 1))


def _exact_attend(s):
    """Sequence by sequence, some tokens and one key head at a time."""
    case = s["case"]
    out = torch.zeros(s["q"].shape[0], case["q_heads"], case["v_dim"], dtype=torch.float64,
                      device="cuda")
    group = case["q_heads"] // case["k_heads"]
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    for b, length in enumerate(lengths):
        at = torch.arange(length, device="cuda")
        page = s["table"][b].long()[at // case["page"]]
        k, v = (_exact_rows(s, n, page, at % case["page"]) for n in ("k", "v"))
        for first in range(starts[b], starts[b + 1], 512):
            end = min(first + 512, starts[b + 1])
            place = length - starts[b + 1] + torch.arange(first, end, device="cuda")
            last = int(place[-1]) + 1
            seen = (at[:last] <= place[:, None]) if not case["window"] else \
                (at[:last] <= place[:, None]) & (at[:last] > place[:, None] - case["window"])
            for h in range(case["q_heads"]):
                a = (s["q"][first:end, h].double() @ k[:last, h // group].t().contiguous()) / \
                    math.sqrt(case["head_dim"])
                a = torch.softmax(a.masked_fill(~seen, float("-inf")), dim=1)
                out[first:end, h] = a @ v[:last, h // group]
    return out


def _exact_turn(x, s):
    """Each pair as one complex number times exp(i angle)."""
    x, pairs = x.double().clone(), s["case"]["pairs"]
    angle = torch.outer(s["positions"].double(), s["freqs"])
    unit = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    head = x[..., :2 * pairs]
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:2], pairs, 2).contiguous()) * unit
        x[..., :2 * pairs] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :pairs].contiguous(), head[..., pairs:].contiguous()) * unit
        x[..., :2 * pairs] = torch.cat([z.real, z.imag], -1)
    return x


def _exact_balance(s):
    x, e = s["logits"].double(), s["logits"].shape[1]
    counted = torch.ones(x.shape[0], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    n = int(counted.sum())
    grad = torch.zeros_like(x)
    counts = torch.bincount(s["choices"][counted].reshape(-1), minlength=e)
    if n == 0:
        return {"loss": torch.zeros((), dtype=torch.float64), "counts": counts, "grad": grad}
    p = torch.softmax(x[counted], dim=1)
    share = counts.double() / (n * s["choices"].shape[1])
    grad[counted] = float(s["grad"]) * e / n * p * (share - (p @ share)[:, None])
    return {"loss": e * (share * p.mean(0)).sum(), "counts": counts, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "balance":
        return _exact_balance(s)
    seqs, places, table = (s[n].tolist() for n in ("sequences", "positions", "table"))
    held = [t for t in range(len(seqs)) if seqs[t] >= 0]
    page = torch.tensor([table[seqs[t]][places[t] // case["page"]] for t in held], device="cuda")
    place = torch.tensor([places[t] % case["page"] for t in held], device="cuda")
    held = torch.tensor(held, device="cuda")
    out = {}
    if case["op"] == "read":
        for n in ("k", "v"):
            rows = _exact_rows(s, n, page, place)
            out[n] = torch.zeros(len(seqs), *rows.shape[1:], dtype=torch.float64, device="cuda")
            out[n][held] = rows
        return out
    out["q"] = _exact_turn(s["q"], s)
    for n, x in (("k", _exact_turn(s["k"], s)), ("v", s["v"].double())):
        x = x[held]
        scale = x.abs().max(dim=-1).values / E4M3_MAX
        cache, scales = s[n + "_cache"].double(), s[n + "_scale"].double()
        cache[page, place] = x / scale.unsqueeze(-1)
        scales[page, place] = scale
        out[n + "_cache"], out[n + "_scale"] = cache, scales
    return out
