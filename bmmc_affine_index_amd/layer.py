"""What a layer with experts over a paged cache needs next to its moved rows
(include/bmmc_layer.h).

Three groups of calls over the same library:

* ``cache_attention``: attention of new tokens, one or a chunk for each
  sequence, over the cache that ``cache_append`` or ``cache_quantize`` wrote;
* ``cache_quantize`` appends to a cache in 8 bits whose scales it makes on the
  way, ``cache_read`` brings rows of a cache back;
* ``expert_balance``: the balance loss of a router with the counts of its
  experts; ``expert_balance_backward`` is its gradient.

Their rules are those of the calls on token rows (``tokens``): device tensors,
asynchronous on torch's current stream or on ``stream``, ValueError for what the
kernels do not take, BmmcError for what the library refuses.  Index tensors are
data: what is out of range is skipped on the device.  Only ``expert_balance``
has a gradient, and none has a second or a forward-mode one.
"""
from __future__ import annotations

import collections
import ctypes

from .tokens import (_calls, _constant, _need, _run, bmmc_heads, bmmc_rotation, tokens_lib)

LAYER_EXPORTED = ("bmmc_cache_attention_workspace", "bmmc_cache_attention", "bmmc_cache_quantize",
                  "bmmc_cache_read", "bmmc_expert_balance_workspace", "bmmc_expert_balance",
                  "bmmc_expert_balance_backward")


class bmmc_scaled_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("place_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("scale_page", ctypes.c_int64),
                ("scale_place", ctypes.c_int64), ("scale_head", ctypes.c_int64),
                ("type", ctypes.c_int)]


class bmmc_attention(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("out_token", ctypes.c_int64),
                ("out_head", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("q_heads", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("batch", ctypes.c_int64),
                ("table_width", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("window", ctypes.c_int64), ("scale", ctypes.c_float), ("k_dim", ctypes.c_int),
                ("v_dim", ctypes.c_int), ("type", ctypes.c_int), ("clear_rest", ctypes.c_int)]


_bound = None


def layer_lib():
    """The loaded libbmmc.so with this module's entry points declared."""
    global _bound
    if _bound is not None:
        return _bound
    L = tokens_lib()
    p, i, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    heads, rotation = ctypes.POINTER(bmmc_heads), ctypes.POINTER(bmmc_rotation)
    cache, attention = ctypes.POINTER(bmmc_scaled_cache), ctypes.POINTER(bmmc_attention)
    L.bmmc_cache_attention_workspace.argtypes = [attention]
    L.bmmc_cache_attention.argtypes = [attention, cache, cache, p, n, p]
    L.bmmc_cache_quantize.argtypes = [heads, heads, heads, cache, cache, n, n, p, n, n, n, p, p, i,
                                      rotation, n, i, i, i, p]
    L.bmmc_cache_read.argtypes = [heads, heads, cache, cache, n, n, p, n, n, n, p, p, i, n, i, i, i,
                                  p]
    L.bmmc_expert_balance_workspace.argtypes = [n, i]
    L.bmmc_expert_balance.argtypes = [p, n, i, i, p, i, n, i, p, p, p, p, p, n, p]
    L.bmmc_expert_balance_backward.argtypes = [p, p, n, i, i, p, n, p, p, n, p]
    for name in LAYER_EXPORTED:
        getattr(L, name).restype = n if name.endswith("workspace") else i
    _bound = L
    return L


# ---------------------------------------------------------------------------
# Paged cache
# ---------------------------------------------------------------------------

def cache_attention(q, k_cache, v_cache, page_table, lengths, starts=None, k_scale=None,
                    v_scale=None, scale=None, window: int = 0, out=None, stream=None):
    """Attention of new tokens over a paged cache that holds their own keys and
    values already: [T, Hq, Dv] from q [T, Hq, D], which may be a view, and
    caches [pages, places, H, D or Dv] with any strides between places and
    heads; Hq is a multiple of H, and neighbouring heads of q share a key head.
    D and Dv are 8 to 512.

    The new tokens of sequence s are rows starts[s] to starts[s + 1] - 1 of q
    (int32 [B + 1], not falling; None: token s alone), the last of them at place
    lengths[s] - 1 (int32 [B]); page_table is int32 [B, pages a sequence].  A
    token sees the places up to its own, with a `window` the last `window` of
    them, on pages that are in range; what the others hold does not matter, be it
    NaN.  A token that sees none, or none of any weight, gives zeros.  `scale`
    is 1 / sqrt(D) or a positive number.

    float8_e4m3fn caches have k_scale and v_scale, float32: one value, one for
    each head, or [pages, places, H], one for each row, as cache_quantize
    makes.  Scales may be any numbers; what a row does not see has none.  Rows
    of q that belong to no sequence give zeros in a new tensor and leave a given
    `out` as it is.  Scores and sums are in 32 bits; weights, times v_scale
    where that is one for each row, are rounded to q's type before they meet the
    values, and so that 2^-16 of one is left out at most where q is float16 and
    v_scale is one for each row.  Otherwise float16 loses bits of weights below
    2^-21 of a row's largest, and those below 2^-32.  There is no gradient."""
    return _run(_calls().attention, (q, k_cache, v_cache, page_table, lengths, starts, k_scale,
                                     v_scale, scale, window, out), stream)[0]


def cache_quantize(k, v, k_cache, v_cache, k_scale, v_scale, page_table, positions,
                   sequences=None, freqs=None, axes=None, turns=None, interleaved: bool = False,
                   scale: float = 1.0, q=None, q_out=None, stream=None):
    """Append keys and values to a paged cache in 8 bits with a scale for each
    head of each token, made on the way: its largest finite magnitude / 448.
    The caches are float8_e4m3fn, k_scale and v_scale float32 [pages, places,
    H] with any strides; both are written in place.  What is stored is value /
    scale to the nearest; infinities become the type's largest value, NaN stays
    NaN.  Tokens of one call go to places of their own: where two go to the
    same, its scale may be one's and its values the other's.  Everything else
    is as in ``cache_append``."""
    return _run(_calls().quantize,
                (k, v, k_cache, v_cache, k_scale, v_scale, page_table, positions, sequences, freqs,
                 axes, turns, interleaved, scale, q, q_out), stream)


def cache_read(k_cache, v_cache, page_table, positions, sequences=None, k_scale=None,
               v_scale=None, dtype=None, k_out=None, v_out=None, stream=None):
    """Rows of a paged cache brought back: (keys [T, H, D], values [T, H, Dv]),
    those at positions[t] of sequence sequences[t] (None: sequence t), by the
    rules of ``cache_append``; zeros where there is no such place.  8-bit
    caches have k_scale and v_scale as in ``cache_attention`` and come back in
    `dtype`, each value times its scale rounded once; other caches come back
    as they are.  There is no gradient."""
    return _run(_calls().read, (k_cache, v_cache, page_table, positions, sequences, k_scale, v_scale,
                                dtype, k_out, v_out), stream)


# ---------------------------------------------------------------------------
# Balance of a router
# ---------------------------------------------------------------------------

ExpertBalance = collections.namedtuple("ExpertBalance", ["loss", "counts", "slopes"])
ExpertBalance.__doc__ = """A router's balance, device tensors: loss, one float32;
counts int32 [E], the choices of each expert; slopes float32 [E], the loss's
derivative by each counted token's probability of an expert."""


def expert_balance(logits, experts, mask=None, stream=None) -> ExpertBalance:
    """The balance loss of a router over E experts: E times the sum over the
    experts of their share of the choices times their mean probability, which
    is 1 where both are even.  logits [T, E] are turned to probabilities by a
    softmax; experts [T, K], int32 or int64, are the choices, of which one
    outside [0, E) is not counted; `mask`, bool [T], leaves tokens out (padding).
    The loss has a gradient by the logits; the shares have none.  Without a
    token that counts all is zero."""
    calls = _calls()
    if calls.asks(logits):
        return ExpertBalance(*_functions()["balance"].apply(logits, experts, mask, stream))
    return ExpertBalance(*_run(calls.balance, (logits, experts, mask), stream)[:3])


def expert_balance_backward(grad, logits, slopes, mask=None, out=None, stream=None):
    """Gradient of expert_balance's logits, [T, E] of their type, from that of
    its loss (one float32 on the device) and its slopes; zeros for tokens that
    the mask leaves out.  It has no gradient of its own."""
    calls = _calls()
    _constant(calls, "grad", grad)
    _constant(calls, "slopes", slopes)
    _need(out is None or not calls.asks(logits), "out cannot be given where a gradient is asked for")
    return _run(calls.balance_backward, (grad, logits, slopes, mask, out), stream)


_made = {}


def _functions() -> dict:
    """The autograd function, made on first use (it needs torch)."""
    if _made:
        return _made
    import torch
    from torch.autograd.function import once_differentiable
    call = _calls()

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, experts, mask, stream):
            loss, counts, slopes, _ = _run(call.balance, (logits, experts, mask), stream)
            ctx.save_for_backward(logits, slopes, mask)
            ctx.mark_non_differentiable(counts, slopes)
            return loss, counts, slopes

        @staticmethod
        @once_differentiable
        def backward(ctx, grad, *_):
            logits, slopes, mask = ctx.saved_tensors
            return _run(call.balance_backward, (grad, logits, slopes, mask, None), None), None, None, None

    _made["balance"] = Balance
    return _made
