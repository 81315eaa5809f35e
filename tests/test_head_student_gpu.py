"""Dropout, the residual join and the head loss as a training step uses them: one after the other
with their gradients, captured whole, and in the distilled student."""
import numpy as np
import pytest

from oracle import dropout as OD

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from oracle import head as OH  # noqa: E402


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def inputs(rows, d, vocab, top, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, h = rnd(rows, d).to(dtype), rnd(rows, d).to(dtype)
    w = (rnd(vocab, d) * d ** -0.5).to(dtype)
    ids = torch.rand((rows, vocab), generator=g, device="cuda").topk(top, dim=1)[1]
    labels = torch.randint(-1, vocab, (rows,), generator=g, device="cuda")
    return x, h, w, rnd(rows, top), ids, labels


def test_a_block_s_end_and_the_loss(api):
    """loss(h + dropout(x)) in fp32: the chain's values and gradients are the statement's, within 1e-5 of
    the largest one (the loss's own bound for these sizes is 4e-6 of it, dropout adds 2^-23)."""
    x, h, w, t, ids, labels = inputs(60, 48, 333, 5, torch.float32)
    a, b, c = (v.clone().requires_grad_() for v in (x, h, w))
    y = api.DropoutFunction.apply(a, 0.3, 17, 5, b, None)
    loss = api.HeadLossFunction.apply(y, c, labels, t, ids, 2.0, 0.5)
    loss.mean().backward()
    num = lambda v: v.double().cpu().numpy()  # noqa: E731
    ry, keep = OD.dropout(num(x), 0.3, 17, 5, num(h))
    r = torch.full((60,), 1 / 60, device="cuda")
    o = OH.head(torch.from_numpy(ry).cuda(), w, labels, t, ids, r, 2.0, 0.5)
    cut = round(0.3 * 65536)
    want = {"loss": (loss, o.loss), "dw": (c.grad, o.dw), "dh": (b.grad, o.dx),
            "dx": (a.grad, o.dx * torch.from_numpy(keep * (65536 / (65536 - cut))).cuda())}
    for name, (got, ref) in want.items():
        assert float((got.double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max()), name


def test_step_captured_whole(api):
    """A step of both operators in a graph whose generator's state moves on inside it: every replay is the
    eager step with that state, bit for bit, with other work between the replays."""
    rows, d, vocab = 300, 96, 1501
    x, h, w, t, ids, labels = inputs(rows, d, vocab, 6, torch.bfloat16)
    r = torch.full((rows,), 1 / rows, device="cuda")
    state = torch.tensor([99, 0], dtype=torch.int64, device="cuda")

    def step(how):
        y = api.dropout_forward(x, 0.1, residual=h, **how)
        loss, dy, dw = api.head_loss_step(y, w, labels, t, ids, r, temperature=2.0, mix=0.5)
        return loss, api.dropout_backward(dy, 0.1, **how), dy, dw

    step(dict(state=state))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(dict(state=state))
        state[1] += 1
    state.copy_(torch.tensor([99, 40]))
    other = torch.randn(1 << 18, device="cuda")
    seen = []
    for k in range(4):
        other.mul_(1.5).add_(float(k))
        for v in got:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(dict(seed=99, offset=40 + k))):
            assert torch.equal(a, b), k
        seen.append(got[2].clone())
    assert not torch.equal(seen[0], seen[1])


def test_two_calls_at_once(api):
    """Calls on two streams keep out of each other's memory."""
    sets = [inputs(200, 64, 4000, 4, torch.bfloat16, seed=s) for s in (3, 4)]
    how = dict(temperature=1.0, mix=0.5)
    call = lambda v, **kw: api.head_loss_step(v[0], v[2], v[5], v[3], v[4], **how, **kw)  # noqa: E731
    want = [call(v) for v in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [call(v, stream=s) for v, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_student_without_logits(api):
    """The student trains without its logits and with dropout; the first step's loss and head gradient are those of the
    kept logits within the roundings that those have (bf16 logits: 2^-8 of up to 8, twice, in the loss)."""
    from monarch_block_diagonal_amd import distill_student as D
    kept, a = D.train(steps=1, rows=256, vocab=1003)
    free, b = D.train(steps=1, rows=256, vocab=1003, keep_logits=False)
    assert abs(float(a[0]) - float(b[0])) <= 2 * 8 * 2.0 ** -8
    ga, gb = kept.head.weight.grad.float(), free.head.weight.grad.float()
    assert gb.shape == ga.shape and torch.isfinite(gb).all()
    # directions agree: both are the same gradient up to roundings of 2^-8 of their terms
    assert float((ga * gb).sum() / (ga.norm() * gb.norm())) > 0.99
    student, losses = D.train(steps=3, rows=200, vocab=701, keep_logits=False, dropout=0.2)
    assert torch.isfinite(losses).all()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in student.parameters())
    assert [m.calls for m in student.drop] == [3, 3]
