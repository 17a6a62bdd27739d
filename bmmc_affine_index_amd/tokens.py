"""Rows of tokens moved to where the data says (include/bmmc_tokens.h).

Three groups of calls over the same library:

* ``expert_order`` sorts the choices of a router by expert, ``expert_gather``
  brings the tokens' rows into that order, ``expert_combine`` brings them back
  with the router's weights; ``expert_gather_backward`` and
  ``expert_combine_backward`` are their gradients;
* ``rotary`` turns heads by positions on one or several axes,
  ``rotary_backward`` turns their gradient back;
* ``cache_append`` puts keys and values into a paged cache, rotating keys (and
  queries) on the way.

Each takes device tensors and runs asynchronously on torch's current stream,
or on ``stream``, ordered after the work queued on the current stream and
before the work queued on it afterwards.  Shapes, types and strides that the
kernels do not take raise ValueError; what the library refuses raises
BmmcError.  The gathers, combines and ``rotary`` take part in autograd when an
input asks for a gradient, and what a call writes into a tensor that it is given
(``out``, ``q_out``, the caches) counts as a change in place.  There are no
second and no forward-mode derivatives: a tensor that asks for one raises
ValueError.  Index tensors are data: an expert, a row, a sequence, a position or
a page out of range is skipped on the device.
"""
from __future__ import annotations

import collections
import ctypes

from . import BmmcError, _ordered
from . import lib as _library

F32, F16, BF16, E4M3 = 0, 1, 2, 3
I32, I64 = 0, 1
MAX_EXPERTS = 2048
MAX_CHOICES = 1024
MAX_HEAD_DIM = 512
MAX_AXES = 8

TOKENS_EXPORTED = ("bmmc_expert_rows", "bmmc_expert_order_workspace", "bmmc_expert_order",
                   "bmmc_expert_gather", "bmmc_expert_combine", "bmmc_expert_combine_backward",
                   "bmmc_rotary", "bmmc_cache_append")


class bmmc_heads(ctypes.Structure):
    _fields_ = [("in", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("in_batch", ctypes.c_int64), ("in_token", ctypes.c_int64),
                ("in_head", ctypes.c_int64), ("out_batch", ctypes.c_int64),
                ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64)]


class bmmc_rotation(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
                ("axis_of_pair", ctypes.c_void_p), ("axis_stride", ctypes.c_int64),
                ("position_type", ctypes.c_int), ("freqs_are_64", ctypes.c_int),
                ("axes", ctypes.c_int), ("pairs", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("scale", ctypes.c_float)]


class bmmc_paged_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("place_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int),
                ("type", ctypes.c_int)]


_bound = None


def tokens_lib():
    """The loaded libbmmc.so with this module's entry points declared."""
    global _bound
    if _bound is not None:
        return _bound
    L = _library()
    p, i, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    heads, cache = ctypes.POINTER(bmmc_heads), ctypes.POINTER(bmmc_paged_cache)
    rotation = ctypes.POINTER(bmmc_rotation)
    L.bmmc_expert_rows.argtypes = [n, i, n]
    L.bmmc_expert_rows.restype = n
    L.bmmc_expert_order_workspace.argtypes = [n, i]
    L.bmmc_expert_order_workspace.restype = n
    L.bmmc_expert_order.argtypes = [p, i, n, i, n, p, p, p, p, p, n, p]
    L.bmmc_expert_gather.argtypes = [p, n, p, p, n, i, n, n, i, p, n, p]
    L.bmmc_expert_combine.argtypes = [p, n, p, p, i, n, i, n, n, i, p, n, p]
    L.bmmc_expert_combine_backward.argtypes = [p, n, p, n, p, p, p, i, n, i, n, n, i, p, n, p, p]
    L.bmmc_rotary.argtypes = [heads, i, n, n, i, i, rotation, p]
    L.bmmc_cache_append.argtypes = [heads, heads, heads, cache, cache, n, n, p, n, n, n, p, p, i,
                                    rotation, n, i, i, i, p]
    for name in TOKENS_EXPORTED[2:]:
        getattr(L, name).restype = i
    _bound = L
    return L


# ---------------------------------------------------------------------------
# Calls
# ---------------------------------------------------------------------------

_torch = None
_native = None


def _calls():
    """The native calls (csrc/binding), bound to the loaded library on first use."""
    global _torch, _native
    if _native is None:
        import torch
        try:
            from . import _calls as native
        except ImportError as e:
            raise RuntimeError("_calls.so is missing or does not load: build it with "
                               "`python -m bmmc_affine_index_amd.build` (there is no fallback "
                               "path)") from e
        native.load(tokens_lib()._name, BmmcError)
        _torch, _native = torch, native
    return _native


def _run(call, args: tuple, stream):
    """call(*args, stream): on torch's current stream, or in order on `stream`."""
    if stream is None:
        return call(*args, None)
    used = [t for a in args for t in (a if isinstance(a, tuple) else (a,))
            if isinstance(t, _torch.Tensor)]
    got = []

    def run(handle):
        got.append(call(*args, handle))
        made = got[0] if isinstance(got[0], tuple) else got
        used.extend(t for t in made if t is not None)
    if not all(t.is_cuda for t in used):
        raise ValueError("tensors must be device tensors")
    _ordered(run, used, stream)
    return got[0]


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _constant(calls, what: str, *tensors) -> None:
    """Refuse an input whose gradient no call makes; asking for it would lose it."""
    _need(not calls.asks(*tensors), what + " has no gradient: detach it, or call under no_grad")


# ---------------------------------------------------------------------------
# Tokens by expert
# ---------------------------------------------------------------------------

ExpertOrder = collections.namedtuple("ExpertOrder", ["offsets", "counts", "rows", "slots"])
ExpertOrder.__doc__ = """Choices sorted by expert, all int32 device tensors:
offsets [E + 1], the first row of each expert and the end of all rows;
counts [E], the choices of each expert; rows [T, K], the row of each choice or
-1 where it is dropped; slots [R], the choice t * K + k at each row or -1
where the row is padding.  The moves take both as expert_order made them: a row
whose choice has been changed in `rows` alone is not written."""


def expert_order(experts, num_experts: int, align: int = 1, stream=None) -> ExpertOrder:
    """Sort a router's choices by expert, stable.  experts is int32 or int64
    [T, K], the experts of each token (any other shape is taken flat, one
    choice a token); a value outside [0, num_experts) drops the choice.  With
    `align` every expert's rows start at a multiple of it.  The order has
    R = T K + min(T K, num_experts) (align - 1) rows, which depends on sizes
    alone, so that no call waits for the device."""
    got = _run(_calls().order, (experts, num_experts, align), stream)
    return ExpertOrder(*got[:4])


def _check_order(order) -> None:
    if not isinstance(order, ExpertOrder):
        raise ValueError("order must be an ExpertOrder")


def expert_gather(x, order: ExpertOrder, out=None, stream=None):
    """The tokens' rows in the order of their experts: [R, D] from x [T, D],
    each token's row once for each choice, zeros where a row is padding."""
    calls = _calls()
    _check_order(order)
    if calls.asks(x):
        _need(out is None, "out cannot be given where a gradient is asked for")
        return _functions()["gather"].apply(x, order, stream)
    return _run(calls.gather, (x, order.rows, order.slots, out), stream)


def expert_gather_backward(grad, order: ExpertOrder, out=None, stream=None):
    """Gradient of expert_gather's x: [T, D], the sum of each token's rows of
    grad [R, D], in 32 bits.  It has no gradient of its own."""
    calls = _calls()
    _check_order(order)
    _constant(calls, "grad", grad)
    return _run(calls.combine, (grad, order.rows, order.slots, None, out), stream)


def expert_combine(rows, order: ExpertOrder, weights=None, out=None, stream=None):
    """The rows by expert, [R, D], back as one row for each token, [T, D]: the
    sum over its choices of weight times row, in 32 bits and in order of the
    choices, rounded once.  weights is [T, K], float32 or of the rows' type
    (None: ones); dropped choices add nothing, whatever their weight."""
    calls = _calls()
    _check_order(order)
    if calls.asks(rows, weights):
        _need(out is None, "out cannot be given where a gradient is asked for")
        return _functions()["combine"].apply(rows, order, weights, stream)
    return _run(calls.combine, (rows, order.rows, order.slots, weights, out), stream)


def expert_combine_backward(grad, rows, order: ExpertOrder, weights, stream=None):
    """Gradients of expert_combine: (of the rows [R, D], of the weights
    [T, K]) from grad [T, D].  They have no gradients of their own; rows and
    weights may be the forward pass's, which ask for one."""
    calls = _calls()
    _check_order(order)
    _constant(calls, "grad", grad)
    return _run(calls.combine_backward, (grad, rows, order.rows, order.slots, weights), stream)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def _turned(calls, many, xs, positions, freqs, axes, interleaved, scale, out, inverse, stream):
    outs = None if out is None else tuple(out) if many else (out,)
    got = _run(calls.rotary, (xs, positions, freqs, axes, interleaved, scale, outs, inverse),
               stream)
    return got if many else got[0]


def rotary(x, positions, freqs, axes=None, interleaved: bool = False, scale: float = 1.0,
           out=None, stream=None):
    """Turn heads by their positions.  x is [T, H, D] or [B, S, H, D] with any
    strides between heads, or a pair of such tensors (queries and keys) that
    are turned in one launch.  Pair i of a head, its elements i and P + i (2i
    and 2i + 1 with `interleaved`) for P = len(freqs) <= D / 2, is turned by
    positions[axes[i]] * freqs[i] and multiplied by `scale`; elements past the
    pairs are copied.  positions is int32 or int64, of the tokens' shape for
    one axis, or [A, ...] for A axes; axes is int32 [P], None for the first
    axis; a pair of an axis that is not there is not turned.  freqs is float32
    or float64 and has no gradient; angles are held in 64 bits.  `out` may be x
    itself; of a pair, a tensor that is turned in place shares no elements with
    the other."""
    calls = _calls()
    many = isinstance(x, (tuple, list))
    xs = tuple(x) if many else (x,)
    if calls.asks(xs):
        _need(out is None, "out cannot be given where a gradient is asked for")
        _constant(calls, "freqs", freqs)
        how = positions, freqs, axes, interleaved, scale
        got = _functions()["rotary"].apply(how, stream, *xs)
        return got if many else got[0]
    return _turned(calls, many, xs, positions, freqs, axes, interleaved, scale, out, False, stream)


def rotary_backward(grad, positions, freqs, axes=None, interleaved: bool = False,
                    scale: float = 1.0, out=None, stream=None):
    """Gradient of rotary's x from that of its result: turned the other way.  It
    has no gradient of its own."""
    calls = _calls()
    many = isinstance(grad, (tuple, list))
    grads = tuple(grad) if many else (grad,)
    _constant(calls, "grad", grads)
    return _turned(calls, many, grads, positions, freqs, axes, interleaved, scale, out, True, stream)


def rotary_axes(sections, interleaved: bool = False, device=None):
    """int32 [sum(sections)] for rotary's `axes`: sections[a] pairs of each
    axis a, one axis after the other or, interleaved, in turn for as long as an
    axis has pairs left."""
    import torch
    left = [int(n) for n in sections]
    _need(left and min(left) >= 0 and sum(left) > 0, "sections are counts of pairs")
    if not interleaved:
        axes = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        axes = [a for i in range(max(left)) for a, n in enumerate(left) if i < n]
    return torch.tensor(axes, dtype=torch.int32, device=device)


# ---------------------------------------------------------------------------
# Paged cache
# ---------------------------------------------------------------------------

def cache_append(k, v, k_cache, v_cache, page_table, positions, sequences=None, freqs=None,
                 axes=None, turns=None, interleaved: bool = False, scale: float = 1.0, q=None,
                 q_out=None, k_scale=None, v_scale=None, stream=None):
    """Append the keys and values of T tokens to a paged cache, in place, in
    one launch.  k [T, H, D] and v [T, H, Dv] may be views; k_cache and v_cache
    are [pages, places, H, D or Dv] with any strides between places and heads,
    and may be views of one array that share no elements.
    Token t is at positions[t] (int32 or int64 [T]) of sequence sequences[t]
    (int32 [T]; None: token t is sequence t's): page page_table[sequence,
    position // places] (int32 [B, pages a sequence]), place position % places.
    A token with a sequence, a position or a page out of range (-1 for padding)
    stores nothing.

    With freqs, keys are turned on the way as by ``rotary``, by `turns` ([T] or
    [A, T]) or, None, by `positions`; queries q [T, Hq, D], where given, are
    turned into q_out (None: a new tensor; q itself: in place, where q shares no
    elements with k and v), which is returned.  float8_e4m3fn caches store value / scale, k_scale and v_scale
    being float32, one value or one for each head; larger values become the
    type's largest.  There is no gradient."""
    return _run(_calls().append,
                (k, v, k_cache, v_cache, page_table, positions, sequences, freqs, axes, turns,
                 interleaved, scale, q, q_out, k_scale, v_scale), stream)


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

_made = {}


def _functions() -> dict:
    """The autograd functions, made on first use (they need torch)."""
    if _made:
        return _made
    torch, call = _torch, _calls()
    from torch.autograd.function import once_differentiable

    def adjacent(g):
        return g if g.dim() < 1 or g.stride(-1) == 1 else g.contiguous()

    # Index tensors are saved as the inputs are: refilled before the backward
    # pass they would give the gradient of another map, and torch raises.
    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, order, stream):
            out = _run(call.gather, (x, order.rows, order.slots, None), stream)
            ctx.save_for_backward(order.rows, order.slots)
            return out

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            return _run(call.combine, (adjacent(grad), *ctx.saved_tensors, None, None), None), None, None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, order, weights, stream):
            out = _run(call.combine, (rows, order.rows, order.slots, weights, None), stream)
            # the largest array of a layer, kept where the weights' gradient needs it
            ctx.save_for_backward(order.rows, order.slots, weights,
                                  rows if ctx.needs_input_grad[2] else None)
            return out

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            at, slots, weights, rows = ctx.saved_tensors
            grad = adjacent(grad)
            if weights is None:
                return _run(call.gather, (grad, at, slots, None), None), None, None, None
            if rows is None:  # any row will do: the weights' gradient is not wanted
                rows = grad.new_empty(1, grad.shape[1]).expand(slots.shape[0], -1)
            got = _run(call.combine_backward, (grad, rows, at, slots, weights), None)
            wanted = [g if n else None for g, n in zip(got, ctx.needs_input_grad[::2])]
            return wanted[0], None, wanted[1], None

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, how, stream, *xs):
            positions, freqs, axes, *kind = how
            got = _turned(call, True, xs, positions, freqs, axes, *kind, None, False, stream)
            ctx.save_for_backward(positions, freqs, axes)
            ctx.kind = kind
            return got

        @staticmethod
        @once_differentiable
        def backward(ctx, *grads):
            got = _turned(call, True, tuple(adjacent(g) for g in grads), *ctx.saved_tensors, *ctx.kind,
                          None, True, None)
            return (None, None, *got)

    _made.update(gather=Gather, combine=Combine, rotary=Rotary)
    return _made
