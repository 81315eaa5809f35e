"""Dropout as a module: recomputed forward passes, copies, and training that is taken up again. On the CPU
the kernel's place is taken by oracle/dropout.py; the GPU tests are the same with the kernel."""
import copy

import numpy as np
import pytest

from oracle import dropout as O

torch = pytest.importorskip("torch")
from monarch_block_diagonal_amd import torch_api as T  # noqa: E402


def stated(x, p, seed=None, offset=0, residual=None, *, state=None, stream=None):
    """dropout_forward by the oracle."""
    if state is not None:
        seed, offset = (int(v) for v in state)
    num = lambda t: None if t is None else t.detach().cpu().numpy()  # noqa: E731
    y, _ = O.dropout(num(x), p, seed, offset, num(residual))
    return torch.from_numpy(np.asarray(y)).to(x.dtype)


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        monkeypatch.setattr(T, "dropout_forward", stated)
    elif not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    return request.param


def layer(device):
    g = torch.Generator().manual_seed(4)
    lin = torch.nn.Linear(40, 24, bias=False)
    lin.weight.data.copy_(torch.randn(24, 40, generator=g))
    return lin.to(device), torch.randn(30, 40, generator=g).to(device)


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_forward_passes_draw_again(device, reentrant):
    """Gradients under activation checkpointing are those of the pass that made the loss: bit for bit those without it."""
    from torch.utils.checkpoint import checkpoint
    lin, x = layer(device)
    drop = T.Dropout(0.5)

    def grads(through):
        torch.manual_seed(12)
        lin.weight.grad = None
        a = x.clone().requires_grad_()
        h = through(lambda v: lin(drop(v)), a)
        y = through(lambda v: drop(v) * v, h)   # a second call of the same module
        (y * y).sum().backward()
        return y.detach().clone(), a.grad.clone(), lin.weight.grad.clone()

    want = grads(lambda f, v: f(v))
    got = grads(lambda f, v: checkpoint(f, v, use_reentrant=reentrant))
    for a, b, name in zip(got, want, ("y", "dx", "dw")):
        assert torch.equal(a, b), name
    assert not torch.equal(drop(x), drop(x))


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_given_seed_counts_and_so_refuses_to_be_recomputed(device, reentrant):
    from torch.utils.checkpoint import checkpoint
    lin, x = layer(device)
    drop = T.Dropout(0.5, seed=3)
    a = x.clone().requires_grad_()
    y = checkpoint(lambda v: lin(drop(v)), a, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="seed"):
        y.sum().backward()
    # a state is drawn from as it stands, however often
    state = torch.tensor([7, 8], dtype=torch.int64, device=device)
    grads = []
    for through in (lambda f, v: f(v), lambda f, v: checkpoint(f, v, use_reentrant=reentrant)):
        a = x.clone().requires_grad_()
        lin.weight.grad = None
        through(lambda v: lin(drop(v, state=state)), a).sum().backward()
        grads.append((a.grad, lin.weight.grad))
    for p, q in zip(*grads):
        assert torch.equal(p, q)


def test_copies_drop_elements_of_their_own(device):
    _, x = layer(device)
    torch.manual_seed(5)
    drop = T.Dropout(0.5)
    twin = copy.deepcopy(drop)
    assert not torch.equal(drop(x), twin(x))
    # the same generator's state, the same elements
    torch.manual_seed(5)
    a = drop(x)
    torch.manual_seed(5)
    assert torch.equal(a, T.Dropout(0.5)(x))


def test_training_taken_up_again(device):
    """A module with a seed goes on at the call it had come to; one without follows torch's generator."""
    _, x = layer(device)
    drop = T.Dropout(0.5, seed=11)
    drop(x), drop(x)
    kept = torch.nn.ModuleDict({"drop": drop}).state_dict()
    third = drop(x)
    again = torch.nn.ModuleDict({"drop": T.Dropout(0.5, seed=11)})
    again.load_state_dict(kept)
    assert again["drop"].calls == 2 and torch.equal(again["drop"](x), third)
    assert torch.equal(third, T.dropout_forward(x, 0.5, 11, 2))
    # weights saved without the count, and one saved where no count is kept
    again.load_state_dict({})
    assert again["drop"].calls == 3
    free = torch.nn.ModuleDict({"drop": T.Dropout(0.5)})
    assert not free.state_dict()
    free.load_state_dict(kept)
    torch.manual_seed(21)
    free["drop"](x)
    held = torch.get_rng_state()
    want = free["drop"](x)
    torch.set_rng_state(held)
    assert torch.equal(torch.nn.ModuleDict({"drop": T.Dropout(0.5)})["drop"](x), want)


def test_a_default_device_of_its_own(device):
    """Numbers come from the generator on the CPU whatever torch's default device is."""
    _, x = layer(device)
    drop = T.Dropout(0.5)
    torch.manual_seed(31)
    want = drop(x)
    torch.manual_seed(31)
    with torch.device("meta"):
        got = drop(x)
    assert torch.equal(got, want)


def test_states_of_calls(device):
    """Calls that share a state drop the same elements; the rows of one tensor are states of their own."""
    _, x = layer(device)
    drops = [T.Dropout(0.5), T.Dropout(0.5, seed=3)]
    state = torch.tensor([[7, 8], [7, 9]], dtype=torch.int64, device=device)
    one, two = (d(x, state=state[0]) for d in drops)
    assert torch.equal(one, two) and torch.equal(one, T.dropout_forward(x, 0.5, 7, 8))
    one, two = (d(x, state=s) for d, s in zip(drops, state))
    assert not torch.equal(one, two) and torch.equal(two, T.dropout_forward(x, 0.5, 7, 9))
