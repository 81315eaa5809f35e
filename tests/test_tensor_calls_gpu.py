"""The tensor helpers and autograd functions of the sandwich norm and the
distillation loss as programs call them: streams, memory, views, gradients of
gradients."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def test_raw_streams_are_the_ones_named(api):
    """Handle 0 is the default stream, also where the current one is another."""
    side = torch.cuda.Stream()
    now = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    with torch.cuda.stream(torch.cuda.Stream()):
        assert api._on_stream(0, now) == 0
        assert api._on_stream(side.cuda_stream, now) == side.cuda_stream
        assert api._on_stream(side, now) == side.cuda_stream


def test_default_stream_by_its_handle(api):
    """stream=0 follows the work queued on the default stream and comes before what is queued next."""
    h, y = torch.randn(4096, 768, device="cuda"), torch.randn(4096, 768, device="cuda")
    z, t = torch.randn(4096, 2000, device="cuda"), torch.randn(4096, 8, device="cuda")
    ids = torch.randint(0, 2000, (4096, 8), device="cuda")
    want = [*api.sandwich_forward(h * 2.0, y), *api.distill_step(z * 2.0, t, ids)]
    torch.cuda.synchronize()
    a = torch.randn(2048, 2048, device="cuda")
    for _ in range(8):
        a = a @ a * 1e-3
    h2, z2 = h * 2.0, z * 2.0   # queued behind the products
    got = [x.clone() for x in (*api.sandwich_forward(h2, y, stream=0), *api.distill_step(z2, t, ids, stream=0))]
    torch.cuda.synchronize()
    for i, (x, w) in enumerate(zip(got, want)):
        assert torch.equal(x, w), i


def test_second_derivatives_are_refused(api):
    """The first derivative with create_graph=True is the one without; its own derivative raises."""
    torch.manual_seed(1)
    x = torch.randn(6, 40, device="cuda", requires_grad=True)
    m = api.SandwichNorm(40, device="cuda")
    t, ids = torch.randn(6, 3, device="cuda"), torch.randint(0, 40, (6, 3), device="cuda")
    for call in (lambda: m(x, x * 2.0)[1].square().sum() + (x ** 3).sum(),
                 lambda: api.DistillLossFunction.apply(x, t, ids, None).sum() + (x ** 3).sum()):
        g, = torch.autograd.grad(call(), x, create_graph=True)
        assert torch.equal(g.detach(), torch.autograd.grad(call(), x)[0])
        with pytest.raises(RuntimeError, match="second"):
            g.square().sum().backward()


def test_overwritten_logits_are_seen_by_autograd(api):
    torch.manual_seed(2)
    x = torch.randn(5, 64, device="cuda", requires_grad=True)
    t, ids = torch.randn(5, 3, device="cuda"), torch.randint(0, 64, (5, 3), device="cuda")
    z = 8.0 * x
    _, want = api.distill_step(z.detach().clone(), t, ids)
    _, dz = api.distill_step(z.detach(), t, ids, out=z.detach())
    z.backward(dz)
    assert torch.equal(x.grad, 8.0 * want)
    z = torch.tanh(x)
    _, dz = api.distill_step(z.detach(), t, ids, out=z.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward(dz)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_a_sequence_s_last_position(api, dtype):
    """Rows far apart: the gradient of the same rows side by side, in memory of its own size."""
    torch.manual_seed(3)
    full = torch.randn(16, 30, 501, device="cuda").to(dtype)
    t, ids = torch.randn(16, 4, device="cuda"), torch.randint(0, 501, (16, 4), device="cuda")
    loss, dz = api.distill_step(full[:, -1], t, ids, temperature=2.0)
    want = api.distill_step(full[:, -1].contiguous(), t, ids, temperature=2.0)
    for got, w in ((loss, want[0]), (dz, want[1])):
        torch.testing.assert_close(got, w, rtol=2.0 ** -7 if dtype == torch.bfloat16 else 1e-5, atol=1e-6)
    assert dz.untyped_storage().nbytes() < 16 * 520 * dtype.itemsize
    x = full.clone().requires_grad_()
    api.DistillLossFunction.apply(x[:, -1], t, ids, None, 2.0).sum().backward()
    assert torch.equal(x.grad[:, -1], dz) and not x.grad[:, :-1].any()


@pytest.mark.parametrize("d", [625, 33])
def test_sandwich_norm_between_slices_of_odd_rows(api, d):
    """h[1:] and what cat hands back lie off every 16-byte boundary: results and gradients of the aligned copies."""
    torch.manual_seed(4)
    m = api.SandwichNorm(d, bias=True, device="cuda")
    h, y = torch.randn(8, d, device="cuda", requires_grad=True), torch.randn(8, d, device="cuda", requires_grad=True)
    head = torch.randn(1, d, device="cuda")
    h_out, n = m(h[1:], y[1:])
    torch.cat([head, h_out, n]).square().sum().backward()
    got = [h_out, n, h.grad, y.grad]
    h2, y2 = (t.detach()[1:].clone().requires_grad_() for t in (h, y))
    h_out, n = m(h2, y2)
    (h_out.square().sum() + n.square().sum()).backward()
    assert torch.equal(got[0], h_out) and torch.equal(got[1], n)
    assert torch.equal(got[2][1:], h2.grad) and torch.equal(got[3][1:], y2.grad)
    assert not got[2][0].any() and not got[3][0].any()


def test_layer_between_slices_of_odd_rows(api):
    torch.manual_seed(5)
    m = api.MonarchLinear(33, 65, 4, device="cuda")
    x = torch.randn(9, 33, device="cuda", requires_grad=True)
    y = m(x[1:])
    torch.cat([torch.ones(1, 65, device="cuda"), y]).square().sum().backward()
    x2 = x.detach()[1:].clone().requires_grad_()
    y2 = m(x2)
    y2.square().sum().backward()
    assert torch.equal(y, y2) and torch.equal(x.grad[1:], x2.grad) and not x.grad[0].any()


def test_no_rows_with_a_gate(api):
    """An empty batch: with a gate a row, with one that every row shares, through the module."""
    none, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    for gate in (torch.empty(0, 64, device="cuda"), torch.ones(1, 64, device="cuda"), torch.ones(3, 64, device="cuda")):
        h_out, n, stats = api.sandwich_forward(none, none.clone(), w, None, gate, w, None)
        g = api.sandwich_backward(none, none, h_out, none, stats, w, None, gate, w, None)
        assert h_out.shape == n.shape == (0, 64) and g.dgate.shape == gate.shape and not g.dgate.any()
        assert not g.dpost_weight.any() and not g.dpre_weight.any()
    m = api.SandwichNorm(64, device="cuda")
    h = torch.empty(2, 0, 64, device="cuda", requires_grad=True)
    h_out, n = m(h, h * 1.0, gate=torch.empty(0, 64, device="cuda"))
    (h_out.sum() + n.sum()).backward()
    assert h.grad.shape == h.shape and not m.pre_weight.grad.any()


def test_distill_function_of_sequences(api):
    """[batch, tokens, vocab] logits without their last position, the first entries of a stored teacher."""
    torch.manual_seed(6)
    z = torch.randn(3, 8, 333, device="cuda", requires_grad=True)
    t, ids = torch.randn(3, 7, 20, device="cuda"), torch.randint(0, 333, (3, 7, 20), device="cuda")
    labels, w = torch.randint(0, 333, (3, 8), device="cuda"), torch.rand(3, 7, device="cuda")
    loss = api.DistillLossFunction.apply(z[:, :-1], t[..., :5], ids[..., :5], labels[:, 1:], 2.0, 0.5)
    (loss * w).sum().backward()
    rows = lambda x: x.reshape(21, *x.shape[2:]).contiguous()  # noqa: E731
    zr = rows(z.detach()[:, :-1])
    want, stats = api.distill_forward(zr, rows(t[..., :5]), rows(ids[..., :5]), rows(labels[:, 1:]), temperature=2.0, mix=0.5)
    dz = api.distill_backward(rows(w), zr, rows(t[..., :5]), rows(ids[..., :5]), rows(labels[:, 1:]), stats, temperature=2.0, mix=0.5)
    assert torch.equal(loss, want.view(3, 7))
    assert torch.equal(z.grad[:, :-1], dz.view(3, 7, 333)) and not z.grad[:, -1].any()
