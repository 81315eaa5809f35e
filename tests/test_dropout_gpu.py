"""GPU parity of dropout against oracle/dropout.py: the same elements are kept, values
are off by the rounding of the product and one of the result (2^-24 of each term, 2^-8 of the result in bf16)."""
import numpy as np
import pytest

from oracle import dropout as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def draw(shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    return [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(3)]


def check(got, x, p, seed, offset, residual):
    num = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    y, keep = O.dropout(num(x), p, seed, offset, num(residual))
    a = num(got).astype(np.float64)
    terms = np.abs(y) + (0 if residual is None else 2 * np.abs(num(residual).astype(np.float64)))
    # the factor, the product and the sum are rounded to fp32, the result to its type
    assert (np.abs(a - y) <= 3 * 2.0 ** -24 * terms + HALF[x.dtype] * np.abs(y) * (1 + 2.0 ** -20)).all()
    dropped = ~keep
    assert (a[dropped] == (0.0 if residual is None else num(residual)[dropped])).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (1, 768), (17, 625), (2, 3, 1001), (300, 4096)])
def test_parity(api, shape, dtype):
    x, res, dy = draw(shape, dtype)
    for p, seed, offset, r in ((0.1, 5, 0, res), (0.5, (1 << 63) + 9, 1, None), (0.013, (1 << 64) - 1, (1 << 64) - 2, res),
                               (0.0, 1, 2, res), (1.0, 1, 2, res), (1.0, 1, 2, None)):
        check(api.dropout_forward(x, p, seed, offset, r), x, p, seed, offset, r)
        check(api.dropout_backward(dy, p, seed, offset), dy, p, seed, offset, None)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_large(api, dtype):
    """Past 2^22 elements: several units a thread, an odd end."""
    x, res, _ = draw((4099, 1027), dtype)
    check(api.dropout_forward(x, 0.3, 11, 12, res), x, 0.3, 11, 12, res)


def test_past_32_bits(api):
    """Elements past 2^32 are their own draws."""
    n = (1 << 32) + 4097
    x = torch.ones((n,), dtype=BF16, device="cuda")
    y = api.dropout_forward(x, 0.5, 21, 3)
    for first in (0, (1 << 31) - 100, (1 << 32) - 1000, n - 4000):
        want = O.draws(4000, 21, 3, first=first) >= 32768
        assert np.array_equal(y[first:first + 4000].float().cpu().numpy(), 2.0 * want)
    del x, y
    torch.cuda.empty_cache()


def test_what_is_dropped_holds_anything(api):
    x, res, _ = draw((64, 100), F32)
    keep = torch.from_numpy(O.draws(6400, 3, 4).reshape(64, 100) >= 32768).cuda()
    clean = api.dropout_forward(x, 0.5, 3, 4, res)
    x[~keep] = float("nan")
    x[0][~keep[0]] = float("inf")
    assert torch.equal(api.dropout_forward(x, 0.5, 3, 4, res), clean)


def test_state_stream_and_capture(api):
    x, res, dy = draw((33, 129), BF16)
    state = torch.tensor([41, 7], dtype=torch.int64, device="cuda")
    want = api.dropout_forward(x, 0.2, 41, 7, res)
    assert torch.equal(api.dropout_forward(x, 0.2, residual=res, state=state), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.dropout_forward(x, 0.2, 41, 7, res, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.dropout_forward(x, 0.2, residual=res, state=state)
        dx = api.dropout_backward(dy, 0.2, state=state)
    for k in range(4):
        state[1] = 100 + k
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, api.dropout_forward(x, 0.2, 41, 100 + k, res))
        assert torch.equal(dx, api.dropout_backward(dy, 0.2, 41, 100 + k))


def test_function_and_module(api):
    x, res, dy = draw((6, 5, 33), F32)
    for shift in (0, 1):   # off a 16-byte boundary
        a = torch.empty((6 * 5 * 33 + 1,), device="cuda")[shift:shift + 6 * 5 * 33].view(6, 5, 33).copy_(x).requires_grad_()
        b = res.clone().requires_grad_()
        y = api.DropoutFunction.apply(a, 0.4, 9, 10, b, None)
        y.backward(dy)
        assert torch.equal(y, api.dropout_forward(x, 0.4, 9, 10, res))
        assert torch.equal(a.grad, api.dropout_backward(dy, 0.4, 9, 10)) and torch.equal(b.grad, dy)
    drop = api.Dropout(0.5, seed=3)
    one, two = drop(x), drop(x)
    assert torch.equal(one, api.dropout_forward(x, 0.5, 3, 0)) and torch.equal(two, api.dropout_forward(x, 0.5, 3, 1))
    state = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    a = x.clone().requires_grad_()
    y = drop(a, res, state=state)
    state[1] = 5   # after the forward pass: the backward pass draws what that drew
    y.backward(dy)
    assert torch.equal(a.grad, api.dropout_backward(dy, 0.5, 1, 2))
    with pytest.raises(RuntimeError, match="second derivatives"):
        a = x.clone().requires_grad_()
        g, = torch.autograd.grad(drop(a).sum(), a, create_graph=True)
        g.sum().backward()


def test_refusals(api):
    x, res, _ = draw((4, 6), F32)
    for kw in (dict(residual=res[:3]), dict(x=x.t()), dict(x=x.cpu()), dict(residual=res.cpu()), dict(seed=None), dict(seed=-1), dict(offset=1 << 64),
               dict(state=torch.zeros((3,), dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            api.dropout_forward(**{**dict(x=x, p=0.5, seed=1, residual=res), **kw})
    for kw in (dict(residual=res.bfloat16()), dict(x=x.half(), residual=None), dict(state=torch.zeros((2,), device="cuda"))):
        with pytest.raises(TypeError):
            api.dropout_forward(**{**dict(x=x, p=0.5, seed=1, residual=res), **kw})
    with pytest.raises(RuntimeError):
        api.dropout_forward(x, 1.5, 1)
