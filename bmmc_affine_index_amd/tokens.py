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
input asks for a gradient.  Index tensors are data: an expert, a row, a
sequence, a position or a page out of range is skipped on the device.
"""
from __future__ import annotations

import collections
import ctypes

from . import BmmcError, OK, _ordered
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
# Arguments
# ---------------------------------------------------------------------------

_torch = None
_types = {}
_index_types = {}


def _t():
    """torch, and the tables of its types, on first use."""
    global _torch
    if _torch is None:
        import torch
        _types.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        _index_types.update({torch.int32: I32, torch.int64: I64})
        _torch = torch
    return _torch


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _run(call, tensors, stream, what: str) -> None:
    """call(stream handle) in order on the stream, on the tensors' device,
    which is torch's current one."""
    torch = _t()
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("tensors must be device tensors")
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensors must be on the current device")
    if stream is None:
        st = call(torch.cuda.current_stream().cuda_stream)
        if st != OK:
            raise BmmcError(st, what)
        return

    def run(h):
        st = call(h)
        if st != OK:
            raise BmmcError(st, what)
    _ordered(run, tensors, stream)


def _asks_gradient(*tensors) -> bool:
    return _t().is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _matrix(x, what: str) -> None:
    _need(x.dim() == 2 and x.dtype in _types, "%s must be [rows, width] of float32, float16 or "
          "bfloat16" % what)
    _need(x.shape[1] > 0, "%s has rows of no elements" % what)
    _need(x.stride(1) == 1 or x.shape[1] == 1, "the elements of a row of %s must be adjacent" % what)


def _index(x, what: str) -> None:
    _need(x.dtype in _index_types and x.is_contiguous(),
          "%s must be contiguous int32 or int64" % what)


def _int32(x, what: str) -> None:
    _need(x.dtype is _t().int32 and x.is_contiguous(), "%s must be contiguous int32" % what)


def _ptr(x):
    return None if x is None else x.data_ptr()


# ---------------------------------------------------------------------------
# Tokens by expert
# ---------------------------------------------------------------------------

ExpertOrder = collections.namedtuple("ExpertOrder", ["offsets", "counts", "rows", "slots"])
ExpertOrder.__doc__ = """Choices sorted by expert, all int32 device tensors:
offsets [E + 1], the first row of each expert and the end of all rows;
counts [E], the choices of each expert; rows [T, K], the row of each choice or
-1 where it is dropped; slots [R], the choice t * K + k at each row or -1
where the row is padding."""


def expert_order(experts, num_experts: int, align: int = 1, stream=None) -> ExpertOrder:
    """Sort a router's choices by expert, stable.  experts is int32 or int64
    [T, K], the experts of each token (any other shape is taken flat, one
    choice a token); a value outside [0, num_experts) drops the choice.  With
    `align` every expert's rows start at a multiple of it.  The order has
    R = T K + min(T K, num_experts) (align - 1) rows, which depends on sizes
    alone, so that no call waits for the device."""
    torch = _t()
    _index(experts, "experts")
    n = experts.numel()
    shape = experts.shape if experts.dim() == 2 else (n, 1)
    L = tokens_lib()
    capacity = L.bmmc_expert_rows(n, int(num_experts), int(align))
    _need(capacity >= 0, "the number of experts, the alignment or the order's rows are out of range")
    need = L.bmmc_expert_order_workspace(n, int(num_experts))
    like = {"dtype": torch.int32, "device": experts.device}
    order = ExpertOrder(torch.empty(num_experts + 1, **like), torch.empty(num_experts, **like),
                        torch.empty(shape, **like), torch.empty(capacity, **like))
    work = torch.empty(need // 4, **like) if need else None
    kind = _index_types[experts.dtype]
    _run(lambda h: L.bmmc_expert_order(experts.data_ptr(), kind, n, num_experts, align,
                                       order.offsets.data_ptr(), order.counts.data_ptr(),
                                       order.rows.data_ptr(), order.slots.data_ptr(), _ptr(work),
                                       need, h),
         [experts, *order] + ([work] if need else []), stream, "expert_order")
    return order


def _check_order(order) -> tuple:
    """(tokens, choices, capacity)"""
    _need(isinstance(order, ExpertOrder), "order must be an ExpertOrder")
    rows, slots = order.rows, order.slots
    _int32(rows, "order.rows")
    _int32(slots, "order.slots")
    _need(rows.dim() == 2 and slots.dim() == 1 and 1 <= rows.shape[1] <= MAX_CHOICES,
          "order.rows must be [tokens, choices] and order.slots [rows]")
    _need(slots.shape[0] >= rows.numel(), "the order has fewer rows than choices")
    return rows.shape[0], rows.shape[1], slots.shape[0]


def _out(out, rows: int, like, what: str):
    if out is None:
        return like.new_empty((rows, like.shape[1]))
    _matrix(out, what)
    _need(out.dtype is like.dtype and tuple(out.shape) == (rows, like.shape[1]),
          "%s must be [%d, %d] of the input's type" % (what, rows, like.shape[1]))
    _need(not (out.requires_grad and _t().is_grad_enabled()),
          "%s must not ask for a gradient" % what)
    return out


def _gather(x, order, out, stream):
    tokens, choices, capacity = _check_order(order)
    _matrix(x, "x")
    _need(x.shape[0] == tokens, "x must have one row for each token of the order")
    out = _out(out, capacity, x, "out")
    if capacity:
        L = tokens_lib()
        _run(lambda h: L.bmmc_expert_gather(x.data_ptr(), x.stride(0), order.rows.data_ptr(),
                                            order.slots.data_ptr(), tokens, choices, capacity,
                                            x.shape[1], _types[x.dtype], out.data_ptr(),
                                            out.stride(0), h),
             [x, order.rows, order.slots, out], stream, "expert_gather")
    return out


def _check_weights(weights, order, dtype) -> None:
    _need(tuple(weights.shape) == tuple(order.rows.shape) and weights.is_contiguous(),
          "weights must be contiguous [tokens, choices]")
    _need(weights.dtype is _torch.float32 or weights.dtype is dtype,
          "weights must be float32 or of the rows' type")


def _combine(rows, order, weights, out, stream):
    tokens, choices, capacity = _check_order(order)
    _matrix(rows, "rows")
    _need(rows.shape[0] == capacity, "rows must have the order's rows")
    if weights is not None:
        _check_weights(weights, order, rows.dtype)
    out = _out(out, tokens, rows, "out")
    if tokens:
        L = tokens_lib()
        kind = F32 if weights is None else _types[weights.dtype]
        used = [rows, order.rows, out] + ([weights] if weights is not None else [])
        _run(lambda h: L.bmmc_expert_combine(rows.data_ptr(), rows.stride(0),
                                             order.rows.data_ptr(), _ptr(weights), kind, tokens,
                                             choices, capacity, rows.shape[1],
                                             _types[rows.dtype], out.data_ptr(), out.stride(0), h),
             used, stream, "expert_combine")
    return out


def expert_gather(x, order: ExpertOrder, out=None, stream=None):
    """The tokens' rows in the order of their experts: [R, D] from x [T, D],
    each token's row once for each choice, zeros where a row is padding."""
    _t()
    if _asks_gradient(x):
        _need(out is None, "out cannot be given where a gradient is asked for")
        return _functions()["gather"].apply(x, order, stream)
    return _gather(x, order, out, stream)


def expert_gather_backward(grad, order: ExpertOrder, out=None, stream=None):
    """Gradient of expert_gather's x: [T, D], the sum of each token's rows of
    grad [R, D], in 32 bits."""
    _t()
    return _combine(grad, order, None, out, stream)


def expert_combine(rows, order: ExpertOrder, weights=None, out=None, stream=None):
    """The rows by expert, [R, D], back as one row for each token, [T, D]: the
    sum over its choices of weight times row, in 32 bits and in order of the
    choices, rounded once.  weights is [T, K], float32 or of the rows' type
    (None: ones); dropped choices add nothing, whatever their weight."""
    _t()
    if _asks_gradient(rows, weights):
        _need(out is None, "out cannot be given where a gradient is asked for")
        return _functions()["combine"].apply(rows, order, weights, stream)
    return _combine(rows, order, weights, out, stream)


def expert_combine_backward(grad, rows, order: ExpertOrder, weights, stream=None):
    """Gradients of expert_combine: (of the rows [R, D], of the weights
    [T, K]) from grad [T, D]."""
    torch = _t()
    tokens, choices, capacity = _check_order(order)
    _matrix(grad, "grad")
    _matrix(rows, "rows")
    _need(rows.shape[0] == capacity, "rows must have the order's rows")
    _need(grad.dtype is rows.dtype and tuple(grad.shape) == (tokens, rows.shape[1]),
          "grad must be [tokens, width] of the rows' type")
    _check_weights(weights, order, rows.dtype)
    grad_rows = torch.empty((capacity, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    grad_weights = torch.empty_like(weights)
    if capacity:
        L = tokens_lib()
        _run(lambda h: L.bmmc_expert_combine_backward(
            grad.data_ptr(), grad.stride(0), rows.data_ptr(), rows.stride(0),
            order.rows.data_ptr(), order.slots.data_ptr(), weights.data_ptr(),
            _types[weights.dtype], tokens, choices, capacity, rows.shape[1], _types[rows.dtype],
            grad_rows.data_ptr(), grad_rows.stride(0), grad_weights.data_ptr(), h),
            [grad, rows, order.rows, order.slots, weights, grad_rows, grad_weights], stream,
            "expert_combine_backward")
    return grad_rows, grad_weights


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def _heads(x, out, what: str) -> bmmc_heads:
    """x [T, H, D] or [B, S, H, D]; out likewise or None."""
    _need(x.stride(-1) == 1 or x.shape[-1] == 1,
          "the elements of a head of %s must be adjacent" % what)
    s = x.stride()
    batch = s[0] if len(s) == 4 else 0
    if out is None:
        return bmmc_heads(x.data_ptr(), None, x.shape[-2], batch, s[-3], s[-2], 0, 0, 0)
    _need(out.shape == x.shape and out.dtype is x.dtype,
          "the output of %s must have its shape and type" % what)
    _need(out.stride(-1) == 1 or out.shape[-1] == 1,
          "the elements of a head of %s's output must be adjacent" % what)
    o = out.stride()
    return bmmc_heads(x.data_ptr(), out.data_ptr(), x.shape[-2], batch, s[-3], s[-2],
                      o[0] if len(o) == 4 else 0, o[-3], o[-2])


def _rotation(positions, tokens, freqs, axes, interleaved, inverse, scale) -> tuple:
    """(bmmc_rotation, the tensors it uses); `tokens` is the shape that the
    positions of one axis have."""
    torch = _t()
    _need(freqs.dim() == 1 and freqs.dtype in (torch.float32, torch.float64) and
          freqs.is_contiguous() and freqs.shape[0] > 0,
          "freqs must be [pairs], contiguous, of float32 or float64")
    used = [freqs]
    count, stride, kind, address = 1, 0, I32, None
    if positions is not None:
        _need(positions.dtype in _index_types, "positions must be int32 or int64")
        shape = tuple(positions.shape)
        if shape == tokens:
            one = positions
        else:
            _need(shape[1:] == tokens and len(shape) == len(tokens) + 1,
                  "positions must have the tokens' shape, or that of axes before it")
            count, stride = shape[0], positions.stride(0)
            _need(1 <= count <= MAX_AXES, "there must be 1 to %d axes" % MAX_AXES)
            one = positions[0]
        _need(one.is_contiguous(), "the positions of an axis must be contiguous")
        kind, address = _index_types[positions.dtype], positions.data_ptr()
        used.append(positions)
    if axes is not None:
        _int32(axes, "axes")
        _need(axes.shape == freqs.shape, "axes must have one entry for each pair")
        used.append(axes)
    return bmmc_rotation(address, freqs.data_ptr(), _ptr(axes), stride, kind,
                         int(freqs.dtype is torch.float64), count, freqs.shape[0],
                         int(bool(interleaved)), int(inverse), scale), used


def _rotary(xs, positions, freqs, axes, interleaved, inverse, scale, outs, stream) -> list:
    torch = _t()
    _need(1 <= len(xs) <= 2 and len(outs) == len(xs), "one or two tensors of heads are turned")
    x = xs[0]
    lead, dim, dtype = tuple(x.shape[:-2]), x.shape[-1], x.dtype
    _need(len(lead) in (1, 2) and dtype in _types,
          "heads must be [tokens, heads, size] or [batch, tokens, heads, size] of float32, "
          "float16 or bfloat16")
    _need(0 < dim <= MAX_HEAD_DIM and min(y.shape[-2] for y in xs) > 0,
          "there must be heads, of up to %d elements" % MAX_HEAD_DIM)
    _need(all(y.dtype is dtype and y.dim() == x.dim() and y.shape[-1] == dim and
              tuple(y.shape[:-2]) == lead for y in xs), "the tensors must have the same tokens, "
          "size of heads and type")
    _need(2 * freqs.shape[0] <= dim if freqs.dim() == 1 else False,
          "freqs must be [pairs] with at most half as many pairs as a head has elements")
    outs = [torch.empty_like(y) if o is None else o for y, o in zip(xs, outs)]
    used = list(xs) + outs
    count = len(xs)
    heads = (bmmc_heads * count)(*[_heads(y, o, "x") for y, o in zip(xs, outs)])
    rotation, more = _rotation(positions, lead, freqs, axes, interleaved, inverse, scale)
    _need(positions is not None, "positions are needed")
    if x.numel():
        L = tokens_lib()
        batch, tokens = lead if len(lead) == 2 else (1, lead[0])
        kind = _types[dtype]
        _run(lambda h: L.bmmc_rotary(heads, count, batch, tokens, dim, kind,
                                     ctypes.byref(rotation), h), used + more, stream, "rotary")
    return outs


def _listed(x, out):
    many = isinstance(x, (tuple, list))
    xs = list(x) if many else [x]
    outs = [None] * len(xs) if out is None else list(out) if many else [out]
    return many, xs, outs


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
    or float64; angles are held in 64 bits.  `out` may be x itself."""
    _t()
    many, xs, outs = _listed(x, out)
    if _asks_gradient(*xs):
        _need(out is None, "out cannot be given where a gradient is asked for")
        got = _functions()["rotary"].apply((positions, freqs, axes, interleaved, scale, stream),
                                           *xs)
    else:
        got = _rotary(xs, positions, freqs, axes, interleaved, 0, scale, outs, stream)
    return tuple(got) if many else got[0]


def rotary_backward(grad, positions, freqs, axes=None, interleaved: bool = False,
                    scale: float = 1.0, out=None, stream=None):
    """Gradient of rotary's x from that of its result: turned the other way."""
    many, xs, outs = _listed(grad, out)
    got = _rotary(xs, positions, freqs, axes, interleaved, 1, scale, outs, stream)
    return tuple(got) if many else got[0]


def rotary_axes(sections, interleaved: bool = False, device=None):
    """int32 [sum(sections)] for rotary's `axes`: sections[a] pairs of each
    axis a, one axis after the other or, interleaved, in turn for as long as an
    axis has pairs left."""
    torch = _t()
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

def _paged(cache, x, scale, heads: int, what: str) -> bmmc_paged_cache:
    torch = _t()
    _need(cache.dim() == 4 and cache.shape[2] == heads and cache.shape[3] == x.shape[2],
          "%s must be [pages, places, heads, size]" % what)
    _need(cache.stride(3) == 1 or cache.shape[3] == 1,
          "the elements of a head of %s must be adjacent" % what)
    narrow = cache.dtype is torch.float8_e4m3fn
    _need(narrow or cache.dtype is x.dtype, "%s must be of the inputs' type or float8_e4m3fn" % what)
    _need(narrow == (scale is not None), "an 8-bit %s has a scale, no other has" % what)
    step = 0
    if narrow:
        _need(scale.dtype is torch.float32 and scale.is_contiguous() and
              scale.numel() in (1, heads), "a scale of %s is float32, one value or one for each "
              "head" % what)
        step = int(scale.numel() > 1)
    s = cache.stride()
    return bmmc_paged_cache(cache.data_ptr(), _ptr(scale), s[0], s[1], s[2], step,
                            E4M3 if narrow else _types[x.dtype])


def cache_append(k, v, k_cache, v_cache, page_table, positions, sequences=None, freqs=None,
                 axes=None, turns=None, interleaved: bool = False, scale: float = 1.0, q=None,
                 q_out=None, k_scale=None, v_scale=None, stream=None):
    """Append the keys and values of T tokens to a paged cache, in place, in
    one launch.  k [T, H, D] and v [T, H, Dv] may be views; k_cache and v_cache
    are [pages, places, H, D or Dv] with any strides between places and heads.
    Token t is at positions[t] (int32 or int64 [T]) of sequence sequences[t]
    (int32 [T]; None: token t is sequence t's): page page_table[sequence,
    position // places] (int32 [B, pages a sequence]), place position % places.
    A token with a sequence, a position or a page out of range (-1 for padding)
    stores nothing.

    With freqs, keys are turned on the way as by ``rotary``, by `turns` ([T] or
    [A, T]) or, None, by `positions`; queries q [T, Hq, D], where given, are
    turned into q_out (None: a new tensor; q itself: in place), which is
    returned.  float8_e4m3fn caches store value / scale, k_scale and v_scale
    being float32, one value or one for each head; larger values become the
    type's largest.  There is no gradient."""
    torch = _t()
    _need(k.dim() == 3 and v.dim() == 3 and k.dtype in _types and v.dtype is k.dtype and
          k.shape[:2] == v.shape[:2] and k.shape[1] > 0,
          "k and v must be [tokens, heads, size] of one type: float32, float16 or bfloat16")
    tokens, heads, dim = k.shape
    _need(0 < dim <= MAX_HEAD_DIM and 0 < v.shape[2] <= MAX_HEAD_DIM,
          "heads may have up to %d elements" % MAX_HEAD_DIM)
    _need(not _asks_gradient(k, v, q), "cache_append has no gradient: call it under no_grad")
    kc = _paged(k_cache, k, k_scale, heads, "k_cache")
    vc = _paged(v_cache, v, v_scale, heads, "v_cache")
    _need(k_cache.shape[:2] == v_cache.shape[:2] and k_cache.dtype is v_cache.dtype,
          "the two caches must have the same pages, places and type")
    _need(k_cache.shape[1] > 0, "pages have no places")
    _need(page_table.dim() == 2 and page_table.dtype is torch.int32 and
          (page_table.stride(1) == 1 or page_table.shape[1] <= 1),
          "page_table must be int32 [sequences, pages], the pages of a sequence adjacent")
    _index(positions, "positions")
    _need(tuple(positions.shape) == (tokens,), "positions must be [tokens]")
    used = [k, v, k_cache, v_cache, page_table, positions]
    if sequences is not None:
        _int32(sequences, "sequences")
        _need(tuple(sequences.shape) == (tokens,), "sequences must be [tokens]")
        used.append(sequences)
    for s in (k_scale, v_scale):
        if s is not None:
            used.append(s)
    rotation = None
    if freqs is None:
        _need(q is None and q_out is None and turns is None and axes is None,
              "queries, turns and axes go with freqs")
    else:
        rotation, more = _rotation(turns, (tokens,), freqs, axes, interleaved, 0, scale)
        _need(2 * freqs.shape[0] <= dim,
              "freqs must be [pairs] with at most half as many pairs as a head has elements")
        used += more
    qh = None
    if q is not None:
        _need(q.dim() == 3 and q.dtype is k.dtype and q.shape[0] == tokens and
              q.shape[1] > 0 and q.shape[2] == dim, "q must be [tokens, heads, size] as k")
        q_out = torch.empty_like(q) if q_out is None else q_out
        qh = _heads(q, q_out, "q")
        used += [q, q_out]
    else:
        _need(q_out is None, "q_out goes with q")
    if tokens:
        L = tokens_lib()
        kh, vh = _heads(k, None, "k"), _heads(v, None, "v")
        batch, width = page_table.shape
        _run(lambda h: L.bmmc_cache_append(
            qh, kh, vh, kc, vc, k_cache.shape[0], k_cache.shape[1], page_table.data_ptr(), batch,
            width, page_table.stride(0), _ptr(sequences), positions.data_ptr(),
            _index_types[positions.dtype], rotation, tokens, dim, v.shape[2], _types[k.dtype], h),
            used, stream, "cache_append")
    return q_out


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------

_made = {}


def _functions() -> dict:
    """The autograd functions, made on first use (they need torch)."""
    if _made:
        return _made
    torch = _t()
    from torch.autograd.function import once_differentiable

    def adjacent(g):
        return g if g.dim() < 1 or g.stride(-1) == 1 else g.contiguous()

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, order, stream):
            ctx.order = order
            return _gather(x, order, None, stream)

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            return expert_gather_backward(adjacent(grad), ctx.order), None, None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, order, weights, stream):
            ctx.order = order
            ctx.weighed = weights is not None
            if ctx.weighed:
                ctx.save_for_backward(rows, weights)
            return _combine(rows, order, weights, None, stream)

        @staticmethod
        @once_differentiable
        def backward(ctx, grad):
            grad = adjacent(grad)
            if not ctx.weighed:
                return _gather(grad, ctx.order, None, None), None, None, None
            rows, weights = ctx.saved_tensors
            grad_rows, grad_weights = expert_combine_backward(grad, rows, ctx.order, weights)
            return grad_rows, None, grad_weights, None

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, how, *xs):
            positions, freqs, axes, interleaved, scale, stream = how
            ctx.how = how
            got = _rotary(list(xs), positions, freqs, axes, interleaved, 0, scale,
                          [None] * len(xs), stream)
            return tuple(got)

        @staticmethod
        @once_differentiable
        def backward(ctx, *grads):
            positions, freqs, axes, interleaved, scale, _ = ctx.how
            got = _rotary([adjacent(g) for g in grads], positions, freqs, axes, interleaved, 1,
                          scale, [None] * len(grads), None)
            return (None, *got)

    _made.update(gather=Gather, combine=Combine, rotary=Rotary)
    return _made
