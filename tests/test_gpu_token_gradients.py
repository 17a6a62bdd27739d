"""GPU tests of the calls on token rows next to torch's autograd: what is written
in place and what a backward pass needs later are known to it."""
import pytest

torch = pytest.importorskip("torch")

import bmmc_affine_index_amd as bm  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=_gen(seed)).to(DEV)


def _order(tokens=6, choices=2):
    experts = torch.randint(-1, 5, (tokens, choices), generator=_gen(1))
    return bm.expert_order(experts.to(DEV), 5, align=2)


def _turns(tokens=6, pairs=4):
    positions = torch.randint(0, 900, (2, tokens), generator=_gen(2)).to(DEV)
    freqs = (10.0 ** -torch.arange(pairs, dtype=torch.float64)).to(DEV)
    return positions, freqs, torch.tensor([0, 1] * (pairs // 2), dtype=torch.int32, device=DEV)


def _append(k_cache, v_cache, q, q_out, stream=None):
    positions, freqs, _ = _turns()
    table = torch.arange(6, dtype=torch.int32, device=DEV)[:, None]
    bm.cache_append(_randn(6, 2, 8), _randn(6, 2, 8), k_cache, v_cache, table, positions[0] % 4,
                    freqs=freqs, q=q, q_out=q_out, stream=stream)


# --------------------------------------------------------------------------
# Results written in place
# --------------------------------------------------------------------------

def _rows():
    return _order().slots.numel()


WRITES = {  # name: (shapes of what is written, the call)
    "gather": (lambda: [(_rows(), 8)],
               lambda o, s: bm.expert_gather(_randn(6, 8), _order(), out=o[0], stream=s)),
    "combine": (lambda: [(6, 8)],
                lambda o, s: bm.expert_combine(_randn(_rows(), 8), _order(), out=o[0], stream=s)),
    "gather backward": (lambda: [(6, 8)], lambda o, s: bm.expert_gather_backward(
        _randn(_rows(), 8), _order(), out=o[0], stream=s)),
    "rotary": (lambda: [(6, 2, 8)], lambda o, s: bm.rotary(
        _randn(6, 2, 8), *_turns(), out=o[0], stream=s)),
    "rotary in place": (lambda: [(6, 2, 8)], lambda o, s: bm.rotary(
        o[0], *_turns(), out=o[0], stream=s)),
    "rotary of two in place": (lambda: [(6, 2, 8), (6, 3, 8)], lambda o, s: bm.rotary(
        tuple(o), *_turns(), out=tuple(o), stream=s)),
    "rotary backward in place": (lambda: [(6, 2, 8)], lambda o, s: bm.rotary_backward(
        o[0], *_turns(), out=o[0], stream=s)),
    "append": (lambda: [(6, 4, 2, 8), (6, 4, 2, 8), (6, 2, 8)],
               lambda o, s: _append(o[0], o[1], _randn(6, 2, 8), o[2], stream=s)),
    "append, queries in place": (lambda: [(6, 4, 2, 8), (6, 4, 2, 8), (6, 2, 8)],
                                 lambda o, s: _append(o[0], o[1], o[2], o[2], stream=s)),
}


@pytest.mark.parametrize("name", WRITES)
def test_a_saved_tensor_that_is_written_is_noticed(name):
    """A product keeps its factor for the gradient of the other one."""
    shapes, call = WRITES[name]
    for i in range(len(shapes())):
        for stream in (None, torch.cuda.Stream()):
            outs = [_randn(*shape, seed=3) for shape in shapes()]
            w = torch.ones((), device=DEV, requires_grad=True)
            loss = (outs[i] * w).sum()
            call(outs, stream)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
            # a view of a larger tensor counts for the whole
            big = [torch.cat([o, o]) for o in outs]
            loss = (big[i] * w).sum()
            call([b[:o.shape[0]] for b, o in zip(big, outs)], stream)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()


@pytest.mark.parametrize("name", WRITES)
def test_results_in_inference_tensors(name):
    """Inference tensors have no version to count."""
    shapes, call = WRITES[name]
    want = [_randn(*shape, seed=3) for shape in shapes()]
    call(want, None)
    with torch.inference_mode():
        outs = [_randn(*shape, seed=3) for shape in shapes()]
        call(outs, None)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_what_is_only_read_is_not_written():
    order, (positions, freqs, axes) = _order(), _turns()
    x, rows, w, q = _randn(6, 8), _randn(_rows(), 8), _randn(6, 2), _randn(6, 2, 8)
    read = [x, rows, w, q, positions, freqs, axes, *order]
    before = [t._version for t in read]
    bm.expert_gather(x, order)
    bm.expert_combine(rows, order, w)
    bm.expert_combine_backward(x, rows, order, w)
    bm.rotary((q, q), positions, freqs, axes)
    assert [t._version for t in read] == before


# --------------------------------------------------------------------------
# What a backward pass needs
# --------------------------------------------------------------------------

def _graph(name):
    """(the loss of a call, the tensors that its gradient is made of)."""
    order, (positions, freqs, axes) = _order(), _turns()
    if name == "gather":
        x = _randn(6, 8).requires_grad_()
        return bm.expert_gather(x, order).square().sum(), [order.rows, order.slots]
    rows = _randn(_rows(), 8).requires_grad_()
    if name == "combine":
        w = _randn(6, 2).requires_grad_()
        return bm.expert_combine(rows, order, w).square().sum(), [order.rows, order.slots, rows, w]
    if name == "combine without weights":
        return bm.expert_combine(rows, order).square().sum(), [order.rows, order.slots]
    q = _randn(6, 2, 8).requires_grad_()
    pair = bm.rotary((q, q * 2), positions, freqs, axes)
    return sum(t.square().sum() for t in pair), [positions, freqs, axes]


@pytest.mark.parametrize("name,count", [("gather", 2), ("combine", 4), ("combine without weights", 2),
                                        ("rotary", 3)])
def test_a_backward_pass_notices_changed_inputs(name, count):
    """An order, positions, frequencies or axes that are refilled before the
    backward pass would give the gradient of another map."""
    loss, _ = _graph(name)
    loss.backward()
    for i in range(count):
        loss, needed = _graph(name)
        assert len(needed) == count
        with torch.no_grad():
            needed[i].add_(0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_a_graph_is_let_go_with_what_it_kept():
    """Nothing that a backward pass needs outlives the graph, and a second pass
    over a graph that was not retained raises, as torch's operations do."""
    import weakref
    loss, needed = _graph("rotary")
    loss.backward(retain_graph=True)
    loss.backward()
    with pytest.raises(RuntimeError, match="second time"):
        loss.backward()
    kept = [weakref.ref(t) for t in needed]
    del needed
    assert all(r() is None for r in kept)


def test_gradients_of_no_tokens():
    """A rank without tokens: the gradient of a sum comes with strides of zero."""
    order = bm.expert_order(torch.zeros(0, 2, dtype=torch.int64, device=DEV), 5)
    positions, freqs, axes = _turns()
    x, w, q = (_randn(0, *shape).requires_grad_() for shape in ((8,), (2,), (2, 8)))
    bm.expert_combine(bm.expert_gather(x, order), order, w).sum().backward()
    assert x.grad.shape == (0, 8) and w.grad.shape == (0, 2)
    bm.expert_combine(x, order).sum().backward()
    sum(t.sum() for t in bm.rotary((q, q), positions[:, :0], freqs, axes)).backward()
    assert q.grad.shape == (0, 2, 8)


def test_combine_keeps_rows_only_for_the_weights():
    """The rows by expert, the largest array of a layer, are kept for the
    weights' gradient alone; the gradients are the same whoever asks."""
    import weakref
    order, w = _order(), _randn(6, 2)
    leaf, grad = _randn(_rows(), 8), _randn(6, 8)
    want_rows, want_w = bm.expert_combine_backward(grad, leaf, order, w)
    for weights_ask in (False, True):
        x, wx = leaf.clone().requires_grad_(), w.clone().requires_grad_(weights_ask)
        rows = x * 1.0
        out = bm.expert_combine(rows, order, wx)
        kept = weakref.ref(rows)
        del rows
        assert (kept() is not None) == weights_ask
        out.backward(grad)
        assert torch.equal(x.grad, want_rows)
        assert torch.equal(wx.grad, want_w) if weights_ask else wx.grad is None
    wx = w.clone().requires_grad_()
    bm.expert_combine(leaf, order, wx).backward(grad)
    assert torch.equal(wx.grad, want_w)
