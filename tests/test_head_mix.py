"""The head loss without teacher entries is the cross entropy, whatever mix says."""
import pytest

torch = pytest.importorskip("torch")
from oracle import head as H  # noqa: E402


def inputs(rows, d, vocab, device, dtype=torch.float32):
    g = torch.Generator().manual_seed(6)
    x, w = torch.randn(rows, d, generator=g).to(dtype), torch.randn(vocab, d, generator=g).to(dtype)
    labels = torch.randint(-1, vocab, (rows,), generator=g)
    r = torch.rand(rows, generator=g) + 0.5
    return tuple(t.to(device) for t in (x, w, labels, r))


def no_entries(rows, device):
    return torch.empty((rows, 0), device=device), torch.empty((rows, 0), dtype=torch.int64, device=device)


@pytest.mark.parametrize("mix", [0.3, 1.0])
def test_oracle(mix):
    x, w, labels, r = inputs(9, 5, 21, "cpu")
    want = H.head(x, w, labels, weight=r)
    assert want.loss.max() > 0
    for t, ids in ((None, None), no_entries(9, "cpu")):
        got = H.head(x, w, labels, t, ids, r, T=2.0, mix=mix)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [9, 150])
@pytest.mark.parametrize("mix", [0.3, 1.0])
def test_calls(mix, rows, dtype):
    from monarch_block_diagonal_amd import torch_api as T
    x, w, labels, r = inputs(rows, 40, 333, "cuda", dtype)
    want = T.head_loss_step(x, w, labels, row_weight=r)
    assert want[0].max() > 0 and want[1].any() and want[2].any()
    for t, ids in ((None, None), no_entries(rows, "cuda")):
        how = dict(temperature=2.0, mix=mix)
        got = T.head_loss_step(x, w, labels, t, ids, r, **how)
        loss, stats = T.head_loss_forward(x, w, labels, t, ids, **how)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(loss, want[0])
        for a, b in zip(T.head_loss_backward(r, x, w, labels, t, ids, stats, **how), want[1:]):
            assert torch.equal(a, b)


def test_a_teacher_needs_its_share():
    """Not given, it is 0 where there is no teacher, and nothing leaves a teacher out silently."""
    from monarch_block_diagonal_amd import torch_api as T
    x, w, labels, r = inputs(9, 40, 33, "cpu")
    t, ids = torch.zeros((9, 2)), torch.zeros((9, 2), dtype=torch.int64)
    for call in (lambda: T.head_loss_forward(x, w, labels, t, ids), lambda: T.head_loss_step(x, w, labels, t, ids, r),
                 lambda: T.head_loss_backward(r, x, w, labels, t, ids, None), lambda: T.HeadLossFunction.apply(x, w, labels, t, ids, 2.0)):
        with pytest.raises(ValueError, match="mix"):
            call()
    assert T._teachers_share(None, None) == T._teachers_share(None, no_entries(9, "cpu")[0]) == 0.0
    assert T._teachers_share(0.5, None) == 0.5 and T._teachers_share(0.0, t) == 0.0
