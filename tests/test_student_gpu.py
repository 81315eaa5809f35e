"""The sandwich norm and the distillation loss as a training program uses them:
autograd functions, modules, HIP graphs, and a student that learns."""
import numpy as np
import pytest

from oracle import distill as OD
from oracle import sandwich as OS

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol=2e-5):
    # fp32 throughout, sums of at most 64 terms: within 2e-5 of the largest value
    assert np.abs(host(got) - want).max() <= tol * max(1.0, np.abs(want).max())


def test_sandwich_module_and_its_gradients(api):
    torch.manual_seed(3)
    rows, d = 24, 64
    m = api.SandwichNorm(d, post_norm=2, pre_norm=1, bias=True, gated=True, branch_scale=0.5, device="cuda")
    with torch.no_grad():
        for p in m.parameters():
            p.add_(torch.randn_like(p) * 0.2)
    h = torch.randn(4, 6, d, device="cuda", requires_grad=True)
    y = torch.randn(4, 6, d, device="cuda", requires_grad=True)
    h_out, n = m(h, y)
    a, b = torch.randn_like(h_out), torch.randn_like(n)
    ((h_out * a).sum() + (n * b).sum()).backward()
    arg = (host(h).reshape(rows, d), host(y).reshape(rows, d), host(m.post_weight), host(m.post_bias), host(m.gate),
           host(m.pre_weight), host(m.pre_bias))
    how = dict(post="layer", pre="rms", branch=0.5)
    rh, rn = OS.forward(*arg, **how)
    g = OS.backward(host(a).reshape(rows, d), host(b).reshape(rows, d), *arg, **how)
    close(h_out.reshape(rows, d), rh)
    close(n.reshape(rows, d), rn)
    close(h.grad.reshape(rows, d), g["dh"])
    close(y.grad.reshape(rows, d), g["dy"])
    for p, k in ((m.post_weight, "dpost_w"), (m.post_bias, "dpost_b"), (m.gate, "dgate"), (m.pre_weight, "dpre_w"),
                 (m.pre_bias, "dpre_b")):
        close(p.grad, g[k])


def test_unused_results_have_no_gradient(api):
    h = torch.randn(8, 32, device="cuda", requires_grad=True)
    y = torch.randn(8, 32, device="cuda", requires_grad=True)
    m = api.SandwichNorm(32, device="cuda")
    h_out, n = m(h, y)
    h_out.sum().backward()
    close(h.grad, np.ones((8, 32)))
    assert not m.pre_weight.grad.any()
    h.grad = y.grad = None
    last = api.SandwichNorm(32, pre_norm=0, device="cuda")
    h_out, n = last(h, y)
    assert n is None
    h_out.sum().backward()
    close(h.grad, np.ones((8, 32)))


def test_distill_function(api):
    torch.manual_seed(4)
    z = torch.randn(16, 700, device="cuda", requires_grad=True)
    t, ids = torch.randn(16, 9, device="cuda"), torch.rand(16, 700, device="cuda").topk(9, dim=1)[1]
    labels = torch.randint(0, 700, (16,), device="cuda")
    loss = api.DistillLossFunction.apply(z, t, ids, labels, 2.0, 0.5)
    w = torch.rand(16, device="cuda")
    (loss * w).sum().backward()
    rl, rd, _, _ = OD.rows(host(z), host(t), ids.cpu().numpy(), labels.cpu().numpy(), host(w), 2.0, 0.5)
    close(loss, rl)
    close(z.grad, rd)


def test_graph_replays_equal_eager(api):
    """Forward, backward and loss captured once and replayed after other work, bit for bit."""
    rows, d, V, K = 300, 520, 3001, 20
    bf = torch.bfloat16
    torch.manual_seed(5)
    h, y, dh, dn = (torch.randn(rows, d, device="cuda").to(bf) for _ in range(4))
    w, g = torch.rand(d, device="cuda").to(bf), torch.rand(3, d, device="cuda").to(bf)
    z = torch.randn(rows, V, device="cuda").to(bf)
    t, ids = torch.randn(rows, K, device="cuda"), torch.randint(0, V, (rows, K), device="cuda")
    labels = torch.randint(0, V, (rows,), device="cuda")

    def step():
        h_out, n, stats = api.sandwich_forward(h, y, w, w, g, w, None)
        grads = api.sandwich_backward(dh, dn, h_out, y, stats, w, w, g, w, None)
        return [h_out, n, *[x for x in grads if x is not None],
                *api.distill_step(z, t, ids, labels, temperature=2.0, mix=0.5)]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    other = torch.randn(1 << 20, device="cuda")
    for k in range(3):
        other.mul_(1.5).add_(float(k))
        for x in got:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (k, i)


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_a_given_stream(api, raw):
    """Work goes to the stream that is named, and its memory comes from there."""
    rows, d, V = 4096, 768, 2000
    torch.manual_seed(6)
    h, y, w = torch.randn(rows, d, device="cuda"), torch.randn(rows, d, device="cuda"), torch.rand(d, device="cuda")
    z, t = torch.randn(rows, V, device="cuda"), torch.randn(rows, 8, device="cuda")
    ids = torch.randint(0, V, (rows, 8), device="cuda")

    def step(**on):
        h_out, n, stats = api.sandwich_forward(h, y, w, None, None, w, None, **on)
        grads = api.sandwich_backward(h, y, h_out, y, stats, w, None, None, w, None, **on)
        loss, dz = api.distill_step(z, t, ids, **on)
        loss2, saved = api.distill_forward(z, t, ids, **on)
        return [h_out, n, *[g for g in grads if g is not None], loss, dz, api.distill_backward(loss2, z, t, ids, None, saved, **on)]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        slow = [torch.randn(2048, 2048, device="cuda") @ torch.randn(2048, 2048, device="cuda") for _ in range(8)]
    got = step(stream=side.cuda_stream if raw else side)
    # allocations of the current stream must not take what the side stream still writes
    other = [torch.full((rows, d), float("nan"), device="cuda") for _ in range(16)]
    side.synchronize()
    torch.cuda.synchronize()
    assert len(slow) + len(other) == 24
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


def test_student_learns():
    from monarch_block_diagonal_amd.distill_student import train
    _, losses = train(steps=40, rows=1024)
    losses = losses.cpu()
    assert torch.isfinite(losses).all()
    # the teacher repeats over 512 tokens: a student that learns at all halves its loss
    assert losses[-5:].mean() < 0.5 * losses[:2].mean(), losses
