"""How the tensor helpers call the library, on the CPU: the library's part is
replaced, what is looked at is the Python around it."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from monarch_block_diagonal_amd import torch_api as T  # noqa: E402


class Streams:
    """Stands in for torch.cuda's streams: a handle that is 0 makes a new stream of a raw one, as in torch."""

    def __init__(self, monkeypatch):
        self.current = [0]
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle if handle else 0xbad)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
        monkeypatch.setattr(torch.cuda, "stream", self.enter)

    @contextlib.contextmanager
    def enter(self, stream):
        self.current.append(stream)
        yield
        self.current.pop()


@pytest.mark.parametrize("handle", [0, 0x7f0040])
def test_a_raw_stream_is_the_one_named(monkeypatch, handle):
    streams = Streams(monkeypatch)
    streams.current = [0x1234]   # the caller's current stream is another one
    assert T._on_stream(handle, lambda: streams.current[-1]) == handle


def _without_kernels(monkeypatch):
    """Stand-ins for the library's calls: the right shapes, any values."""
    def forward(h, y=None, *par, **how):
        return (h if y is None else h.detach() + y.detach()), h.detach().clone(), torch.zeros(len(h), 4)

    def backward(dh_out, dn, h_out, y, stats, *par, **how):
        like = lambda t: None if t is None else torch.ones_like(t)  # noqa: E731
        return T.SandwichGrads(like(h_out), like(y), *map(like, par))

    monkeypatch.setattr(T, "sandwich_forward", forward)
    monkeypatch.setattr(T, "sandwich_backward", backward)
    monkeypatch.setattr(T, "distill_forward", lambda z, *a, **how: (z.detach().sum(1), torch.zeros(len(z), 4)))
    monkeypatch.setattr(T, "distill_backward", lambda dloss, z, *a, **how: torch.ones_like(z))


def _sandwich(x):
    w = torch.nn.Parameter(torch.ones(x.shape[1]))
    return T.SandwichFunction.apply(x, x * x, w, None, None, w, None,
                                    dict(post_norm=1, pre_norm=1, skip_scale=1.0, branch_scale=1.0, eps=1e-5))[1]


def _distill(x):
    return T.DistillLossFunction.apply(x, torch.zeros(len(x), 2), torch.zeros(len(x), 2, dtype=torch.int64), None)


@pytest.mark.parametrize("call", [_sandwich, _distill])
@pytest.mark.parametrize("weighted", [False, True])
def test_second_derivatives_are_refused(monkeypatch, call, weighted):
    """A penalty on a gradient must not lose the part that goes through a kernel, whatever else is in it."""
    _without_kernels(monkeypatch)
    x = torch.randn(3, 4, requires_grad=True)
    out = call(x)
    s = (out * x.sum()).sum() if weighted else out.sum() + (x ** 3).sum()
    g, = torch.autograd.grad(s, x, create_graph=True)
    with pytest.raises(RuntimeError, match="second"):
        (g * g).sum().backward()
    # the first derivative is there, with and without a graph of its own
    assert torch.equal(g.detach(), torch.autograd.grad((call(x) * x.sum()).sum() if weighted else call(x).sum() + (x ** 3).sum(), x)[0])


def test_gradients_with_a_graph_can_be_scaled_and_cleared(monkeypatch):
    """backward(create_graph=True) leaves gradients that clipping and zero_grad may write to."""
    _without_kernels(monkeypatch)
    x = torch.randn(3, 4, requires_grad=True)
    for _ in range(2):
        out = _sandwich(x)
        out.sum().backward(create_graph=True)
        torch.nn.utils.clip_grad_norm_([x], 0.5)
        with torch.no_grad():
            x.grad.mul_(2.0)
        x.grad.detach_().zero_()
        assert x.grad is not None and not x.grad.any()


def test_second_derivatives_of_the_layers_are_refused(monkeypatch):
    zeros = lambda *a, **k: (torch.zeros(3, 4), torch.zeros(3, 4))  # noqa: E731
    ones = lambda *ts: tuple(torch.ones_like(t) for t in ts)  # noqa: E731
    monkeypatch.setattr(T, "monarch_forward", zeros)
    monkeypatch.setattr(T, "monarch_forward_ex", zeros)
    monkeypatch.setattr(T, "monarch_backward", lambda dy, x, w1, w2, z, *a: ones(x, w1, w2))
    monkeypatch.setattr(T, "monarch_backward_ex", lambda dy, x, w1, w2, z, *a: (*ones(x, w1, w2), None))
    w = torch.nn.Parameter(torch.ones(2, 2, 2))
    for call in (lambda x: T.MonarchLinearFunction.apply(x, w, w),
                 lambda x: T.MonarchLinearExFunction.apply(x, w, w, None, 4)):
        x = torch.randn(3, 4, requires_grad=True)
        g, = torch.autograd.grad(call(x).sum() + (x ** 3).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="second"):
            (g * g).sum().backward()


@pytest.mark.parametrize("kind", ["step", "backward"])
def test_overwritten_logits_are_seen_by_autograd(monkeypatch, kind):
    """out=logits replaces values that a backward pass may have saved: that pass raises, as after any write in place."""
    monkeypatch.setattr(T, "_distill_shapes", lambda z, *a: (*z.shape, 2, z.shape[1], -1))
    monkeypatch.setattr(T, "_saved", lambda *a: None)
    monkeypatch.setattr(T.B, "monarch_distill_step", lambda *a: None)
    monkeypatch.setattr(T.B, "monarch_distill_bwd", lambda *a: None)
    t, ids, stats = torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 4)

    def write(z, out):
        if kind == "step":
            return T.distill_step(z, t, ids, out=out)[1]
        return T.distill_backward(torch.ones(3), z, t, ids, None, stats, out=out)

    x = torch.randn(3, 5, requires_grad=True)
    z = torch.tanh(x)   # tanh saves its result for its backward pass
    dz = write(z.detach(), z.detach())
    assert dz.data_ptr() == z.data_ptr()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward(dz)
    z = x * 2.0         # a product by a number saves nothing of its result
    z.backward(write(z.detach(), z.detach()))
    z = torch.tanh(x)   # memory of its own, or the library's: nothing to see
    z.backward(write(z.detach(), torch.empty(3, 5)))
    z = torch.tanh(x)
    z.backward(write(z.detach(), None))
    with torch.inference_mode():   # tensors without a version
        a = torch.ones(3, 5)
        write(a, a)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_of_rows_far_apart_are_stored_close(dtype):
    """dlogits takes the memory of the gradient, not that of the tensor whose rows the logits are."""
    per = 16 // dtype.itemsize
    for logits in (torch.zeros(16, 20, 501, dtype=dtype)[:, -1], torch.zeros(40, 1001, dtype=dtype)[::3], torch.zeros(9, 700, dtype=dtype)[:, :300],
                   torch.zeros(9, 304, dtype=dtype)[:, :300], torch.zeros(9, 301, dtype=dtype), torch.zeros(5, 7, dtype=dtype)[:, :2]):
        rows, vocab = logits.shape
        ld = T._rows_apart(logits, rows, vocab, "logits")
        dz, dld = T._distill_out(logits, rows, vocab, ld, -1, None)
        assert dz.shape == logits.shape and dz.dtype == dtype and dz.stride() == (dld, 1)
        room = dz.untyped_storage().nbytes() // dtype.itemsize
        assert room <= rows * (vocab + max(vocab // 8, per))
        # rows of the gradient start where rows of the logits do between two 16-byte boundaries
        assert (dld - ld) % per == 0
    padded = torch.zeros(4, 50304, dtype=dtype)[:, :50257]   # a little padding stays: rows start at cache lines
    assert T._distill_out(padded, 4, 50257, 50304, -1, None)[1] == 50304


def _off(*shape):
    """A contiguous tensor that starts between two 16-byte boundaries, as a slice of odd rows does."""
    n = 1
    for s in shape:
        n *= s
    t = torch.randn(n + 1)[1:].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


def test_sandwich_function_takes_slices(monkeypatch):
    """x[1:] of odd rows, and the gradients that cat hands back, start anywhere; the library's tensors may not."""
    def aligned(*ts):
        assert all(t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0) for t in ts)

    _without_kernels(monkeypatch)
    forward, backward = T.sandwich_forward, T.sandwich_backward
    monkeypatch.setattr(T, "sandwich_forward", lambda h, y, *par, **how: (aligned(h, y, *par), forward(h, y, *par, **how))[1])
    monkeypatch.setattr(T, "sandwich_backward", lambda *a, **how: (aligned(*a), backward(*a, **how))[1])
    how = dict(post_norm=1, pre_norm=1, skip_scale=1.0, branch_scale=1.0, eps=1e-5)
    h, y, gate = (t.requires_grad_() for t in (_off(3, 5), _off(3, 5), _off(3, 5)))
    w, b = _off(5), _off(5)
    h_out, n = T.SandwichFunction.apply(h, y, w, b, gate, w, b, how)
    torch.cat([torch.ones(1, 5), h_out, n]).square().sum().backward()
    assert h.grad is not None and gate.grad.shape == gate.shape
    T.SandwichFunction.apply(h, None, None, None, None, w, b, how).sum().backward()


def test_layer_functions_take_slices(monkeypatch):
    def aligned(*ts):
        assert all(t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0) for t in ts if t is None or torch.is_tensor(t))

    def fwd(x, w1, w2, *a):
        aligned(x, w1, w2, *a)
        return torch.zeros(3, 5), torch.zeros(3, 6)

    def bwd(dy, x, w1, w2, *a):
        aligned(dy, x, w1, w2, *a)
        return tuple(torch.ones_like(t) for t in (x, w1, w2))

    monkeypatch.setattr(T, "monarch_forward", fwd)
    monkeypatch.setattr(T, "monarch_forward_ex", lambda x, w1, w2, out, bias, act: fwd(x, w1, w2, bias))
    monkeypatch.setattr(T, "monarch_backward", bwd)
    monkeypatch.setattr(T, "monarch_backward_ex", lambda *a: (*bwd(*a), torch.ones(5)))
    x, w, b = (t.requires_grad_() for t in (_off(3, 5), _off(2, 3, 3), _off(5)))
    for out in (T.MonarchLinearFunction.apply(x, w, w), T.MonarchLinearExFunction.apply(x, w, w, b, 5)):
        torch.cat([torch.ones(1, 5), out]).square().sum().backward()


def test_a_gate_a_row_of_no_rows(monkeypatch):
    """An empty batch has no gate rows either; a batch with rows needs some."""
    monkeypatch.setattr(T.B, "current_device", lambda: -1)   # a CPU tensor's device
    shapes = lambda h, y, gate: T._sandwich_shapes(h, y, None, None, gate, None, None, 1, 1.0)[:3]  # noqa: E731
    none = torch.empty(0, 64)
    assert shapes(none, none, torch.empty(0, 64)) == (0, 64, 0)
    assert shapes(none, none, torch.ones(3, 64)) == (0, 64, 3)
    for h, gate in ((torch.ones(2, 64), torch.empty(0, 64)), (none, torch.empty(0, 63)), (none, torch.empty(0)), (none, torch.empty(64))):
        with pytest.raises(ValueError):
            shapes(h, h.clone(), gate)


def test_distill_function_takes_batches_of_sequences_and_slices(monkeypatch):
    """[batch, tokens, vocab] logits, a slice of a stored teacher, a transposed label: rows reach the library as it takes them."""
    def rows(z, t, ids, labels):
        assert z.dim() == t.dim() == ids.dim() == 2 and len(z) == len(t) == len(ids) and z.stride(1) == 1 and z.stride(0) >= z.shape[1]
        assert t.is_contiguous() and ids.is_contiguous() and (labels is None or (labels.dim() == 1 and labels.is_contiguous()))

    def forward(z, t, ids, labels, **how):
        rows(z, t, ids, labels)
        return z.sum(1) + t.sum(1) + (0 if labels is None else labels), torch.zeros(len(z), 4)

    def backward(dloss, z, t, ids, labels, stats, **how):
        rows(z, t, ids, labels)
        assert dloss.dim() == 1 and dloss.is_contiguous() and len(dloss) == len(z)
        return dloss[:, None] * z

    monkeypatch.setattr(T, "distill_forward", forward)
    monkeypatch.setattr(T, "distill_backward", backward)
    for lead in ((6,), (2, 3), (2, 1, 3), (), (0, 3)):
        z = torch.randn(*lead, 5).requires_grad_()
        t, ids = torch.randn(*lead, 4)[..., :2], torch.zeros(*lead, 4, dtype=torch.int64)[..., :2]
        labels = torch.zeros(lead[::-1], dtype=torch.int64)
        labels = labels.permute(tuple(range(len(lead)))[::-1])
        w = torch.rand(lead)
        for given in (z, torch.cat([z, z], -1)[..., 5:], z.detach().transpose(0, -1).contiguous().transpose(0, -1).requires_grad_()):
            loss = T.DistillLossFunction.apply(given, t, ids, labels)
            assert loss.shape == torch.Size(lead)
            g, = torch.autograd.grad((loss * w).sum(), given)
            assert torch.equal(g, w[..., None] * given)
        loss = T.DistillLossFunction.apply(z, t[..., :0], ids[..., :0], None, 2.0, 0.5)
        assert loss.shape == torch.Size(lead)
    z, t, ids = torch.randn(2, 3, 5), torch.randn(3, 2, 4), torch.zeros(2, 3, 4, dtype=torch.int64)
    for args in ((z, t, ids, None), (z, t.view(2, 3, 4), ids.view(3, 2, 4), None), (z, t.view(2, 3, 4), ids, torch.zeros(3, 2, dtype=torch.int64)),
                 (z, t.view(2, 3, 4), ids, torch.zeros(6, dtype=torch.int64)), (z, t.view(6, 4), ids.view(6, 4), None)):
        with pytest.raises(ValueError):
            T.DistillLossFunction.apply(*args)
