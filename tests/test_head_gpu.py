"""GPU parity of the head loss and its gradients against the fp64 statement of
oracle/head.py, whose bounds() derives how far they may be off, and the calls that are
refused."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from oracle import head as H  # noqa: E402

U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    return torch_api


def draw(rows, d, vocab, dtype, top=0, holes=False, seed=0, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = (rnd(vocab, d) * scale * d ** -0.5).to(dtype)
    labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    x = (rnd(rows, d) + 1.5 * w[labels].float()).to(dtype)
    t = ids = None
    if top:
        t = rnd(rows, top) * 2
        ids = (torch.randint(0, vocab, (rows, 1), generator=g, device="cuda") +
               torch.arange(top, device="cuda") * max(1, vocab // top)) % vocab
        ids = ids.contiguous()
        labels = torch.where(torch.rand((rows,), generator=g, device="cuda") < 0.5, ids[:, 0], labels)
    if holes:
        u = torch.rand((rows,), generator=g, device="cuda")
        labels = torch.where(u < 0.4, -100, labels)
        if top:
            ids = torch.where((u < 0.3)[:, None], -1, ids)
            ids[:, -1] = vocab
            t[u > 0.8, 0] = float("-inf")
    r = torch.rand((rows,), generator=g, device="cuda") + 0.5
    return x, w, labels, t, ids, r


def near(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    off = ((got.double() - want).abs() - bound).max() if got.numel() else torch.zeros(())
    assert float(off) <= 0, f"{what}: {float(off):.3g} past its bound, largest value {float(want.abs().max()):.3g}"


def check(api, x, w, labels, t, ids, r, T, mix):
    o = H.head(x, w, labels, t, ids, r, T, mix)
    b_loss, b_dx, b_dw = H.bounds(o, x, w, U[x.dtype], T)
    how = dict(temperature=T, mix=mix)
    loss, stats = api.head_loss_forward(x, w, labels, t, ids, **how)
    near(loss, o.loss, b_loss, "loss")
    dx, dw = api.head_loss_backward(r, x, w, labels, t, ids, stats, **how)
    near(dx, o.dx, b_dx, "dx")
    near(dw, o.dw, b_dw, "dw")
    again = api.head_loss_step(x, w, labels, t, ids, r, **how)
    for a, b, name in zip(again, (loss, dx, dw), ("loss", "dx", "dw")):
        assert torch.equal(a, b), f"step and forward + backward differ: {name}"
    assert not dx[~o.used].any() and not loss[~o.used].any()


SIZES = [(1, 1, 1), (1, 8, 512), (1, 64, 1000), (3, 33, 700), (8, 768, 5003), (32, 40, 131), (33, 96, 640), (64, 100, 129),
         (100, 256, 4096), (129, 57, 727), (257, 160, 2000), (300, 130, 999)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,d,vocab", SIZES)
def test_cross_entropy(api, rows, d, vocab, dtype):
    x, w, labels, _, _, r = draw(rows, d, vocab, dtype, holes=rows > 2)
    check(api, x, w, labels, None, None, r, 1.0, 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,mix", [(1.0, 1.0), (1.0, 0.5), (2.0, 0.5), (0.5, 0.9), (3.0, 1.0)])
@pytest.mark.parametrize("rows,d,vocab,top", [(1, 16, 40, 1), (20, 64, 300, 7), (70, 33, 1001, 64), (260, 128, 600, 512)])
def test_distillation(api, rows, d, vocab, top, T, mix, dtype):
    x, w, labels, t, ids, r = draw(rows, d, vocab, dtype, top=top, holes=rows > 2, seed=5)
    check(api, x, w, labels, t, ids, r, T, mix)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,d,vocab,top", [(1, 320, 70001, 0), (16, 72, 40000, 5), (17, 264, 33000, 0), (32, 600, 20050, 3), (29, 37, 50257, 2), (5, 1028, 66000, 0)])
def test_few_rows(api, rows, d, vocab, top, dtype):
    """Runs of words over several tiles, that end inside a tile; K tiles that end inside a row."""
    x, w, labels, t, ids, r = draw(rows, d, vocab, dtype, top=top, holes=rows > 2, seed=23)
    for T, mix in (((1.0, 0.0),) if not top else ((2.0, 0.5), (1.3, 0.7), (1.0, 1.0))):
        check(api, x, w, labels, t, ids, r, T, mix)


@pytest.mark.parametrize("rows,d,vocab,top", [(1, 64, 700, 0), (16, 40, 5000, 3), (17, 129, 2000, 0), (32, 264, 3001, 2), (33, 72, 4000, 0), (64, 256, 2500, 5)])
def test_few_rows_round_g_twice(api, rows, d, vocab, top):
    """Up to 64 rows g has two bf16 parts: off by 2^-8 of 2^-8, before dx and dw are rounded by 2^-8. Row weights
    lie 10^6 apart, and rows are left out."""
    x, w, labels, t, ids, r = draw(rows, d, vocab, BF16, top, holes=rows > 1, seed=rows)
    r = r * 10.0 ** torch.linspace(-3, 3, rows, device="cuda")
    how = dict(temperature=2.0, mix=0.5 if top else 0.0)
    o = H.head(x, w, labels, t, ids, r, 2.0, how["mix"])
    _, dx, dw = H.bounds(o, x, w, 2.0 ** -16, 2.0)
    got = api.head_loss_step(x, w, labels, t, ids, r, **how)
    near(got[1], o.dx, dx + 2.0 ** -8 * (o.dx.abs() + dx), "dx")
    near(got[2], o.dw, dw + 2.0 ** -8 * (o.dw.abs() + dw), "dw")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,d,vocab", [(8, 64, 300), (30, 37, 1001), (32, 264, 515), (50, 96, 700), (64, 33, 257), (90, 72, 400)])
def test_none_or_one_of_few_rows_counts(api, rows, d, vocab, dtype):
    x, w, labels, _, _, r = draw(rows, d, vocab, dtype, seed=9)
    for only in (None, rows - 1):
        few = torch.full_like(labels, -1)
        if only is not None:
            few[only] = labels[only]
        # memory that a workspace may get holds NaN
        for n in (1 << 20, 1 << 22, 1 << 24):
            torch.full((n,), float("nan"), device="cuda")
        check(api, x, w, few, None, None, r, 1.0, 0.0)


@pytest.mark.parametrize("rows,d,vocab,dtype", [(5, 8, 3000001, F32), (3, 6, 1500007, F32), (20, 8, 4300003, BF16)])
def test_pieces_of_few_rows(api, rows, d, vocab, dtype):
    """More words than a piece of g has. In fp32 a wave adds one 2048th of a piece's words in turn, 128 of
    these sums a thread, 16 threads and two pieces: fewer than 2^11 additions in sequence for dx, where bounds() counts one a
    word."""
    x, w, labels, _, _, r = draw(rows, d, vocab, dtype, seed=5)
    labels[0], labels[-1] = 1, vocab - 1
    o = H.head(x, w, labels, None, None, r)
    b_loss, b_dx, b_dw = H.bounds(o, x, w, U[dtype])
    loss, dx, dw = api.head_loss_step(x, w, labels, row_weight=r)
    near(loss, o.loss, b_loss, "loss")
    if dtype == F32:
        assert vocab / 2048 + 4 + 128 + 16 + 2 < 2 ** 11
        b_dx = b_dx - (vocab - 2 ** 11) * 2.0 ** -24 * (o.g.abs() @ w.double().abs())
    near(dx, o.dx, b_dx, "dx")
    near(dw, o.dw, b_dw, "dw")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_wide_tiles(api, dtype):
    """Enough tiles for the 256 x 256 products; words and rows that end inside a tile, a third of the rows left out."""
    x, w, labels, t, ids, r = draw(1100, 136, 20011, dtype, top=9, holes=True, seed=7)
    check(api, x, w, labels, t, ids, r, 2.0, 0.5)


@pytest.mark.parametrize("rows,d,vocab,dtype", [(9000, 64, 65000, BF16), (4100, 40, 50257, F32), (2000, 32, 300, BF16), (5000, 320, 512, F32)])
def test_pieces_and_splits(api, rows, d, vocab, dtype):
    """More than one piece of the vocabulary; few output tiles, whose sums are split."""
    x, w, labels, _, _, r = draw(rows, d, vocab, dtype, holes=True, seed=11)
    check(api, x, w, labels, None, None, r, 1.0, 0.0)


def test_entries_that_name_one_word(api):
    x, w, labels, t, ids, r = draw(40, 64, 200, F32, top=12, seed=3)
    ids[:, 5] = ids[:, 1]
    ids[:, 9] = ids[:, 1]
    ids[10:, 2] = labels[10:]
    check(api, x, w, labels, t, ids, r, 2.0, 0.5)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rows_left_out_hold_anything(api, dtype):
    """NaN and infinities in rows without label and entry, in their weights, and in the teacher's padding."""
    x, w, labels, t, ids, r = draw(300, 64, 700, dtype, top=4, holes=True, seed=13)
    out = ((labels < 0) & (ids[:, :-1] < 0).all(dim=1))
    assert out.sum() > 20
    x[out, 3], r[out] = float("nan"), float("nan")
    x[out, 5] = float("inf")
    t[:, -1] = float("nan")
    check(api, x, w, labels, t, ids, r, 2.0, 0.5)


def test_no_row_counts(api):
    x, w, labels, _, _, r = draw(50, 64, 300, BF16)
    loss, dx, dw = api.head_loss_step(x, w, torch.full_like(labels, -100), row_weight=r)
    assert not loss.any() and not dx.any() and not dw.any()
    loss, dx, dw = api.head_loss_step(x[:0], w, labels[:0], row_weight=r[:0])
    assert loss.shape == (0,) and dx.shape == (0, 64) and not dw.any()
    assert api.head_loss_forward(x[:0], w, labels[:0])[0].shape == (0,)


def test_a_logit_that_is_nan_comes_out(api):
    x, w, labels, _, _, r = draw(40, 64, 300, F32)
    x[7, 3] = float("nan")
    loss, dx, dw = api.head_loss_step(x, w, labels, row_weight=r)
    assert torch.isnan(loss[7]) and torch.isnan(dx[7]).all() and torch.isnan(dw).all()
    rest = torch.arange(40, device="cuda") != 7
    assert torch.isfinite(loss[rest]).all() and torch.isfinite(dx[rest]).all()


def test_far_logits(api):
    """Logits hundreds apart: sums of exponentials stay finite, a loss is a difference of logits."""
    for dtype in (F32, BF16):
        x, w, labels, t, ids, r = draw(64, 64, 500, dtype, top=3, seed=17, scale=80.0)
        check(api, x, w, labels, t, ids, r, 1.0, 0.5)


@pytest.mark.parametrize("rows", [5, 200])
def test_largest_fp32_values(api, rows):
    """Features at the end of fp32's range (they round to infinity in bf16) against words that are 0 or tiny there."""
    x, w, labels, _, _, r = draw(rows, 64, 500, F32)
    big = torch.finfo(F32).max
    x[:, 3] = big * torch.where(torch.arange(rows, device="cuda") % 2 == 0, 1.0, -1.0)
    w[:, 3] = torch.where(torch.arange(500, device="cuda") % 3 == 0, 0.0, 1e-38)
    o = H.head(x, w, labels, None, None, r)
    loss, dx, dw = api.head_loss_step(x, w, labels, row_weight=r)
    near(loss, o.loss, H.bounds(o, x, w, 0.0)[0], "loss")
    near(dx, o.dx, H.bounds(o, x, w, 0.0)[1], "dx")


def test_rows_apart_and_unaligned(api):
    """Rows of x that lie apart or off 16-byte boundaries (a position of every sequence)."""
    for dtype in (F32, BF16):
        x, w, labels, _, _, r = draw(90, 64, 500, dtype)
        wide = torch.full((90, 77), float("nan"), dtype=dtype, device="cuda")
        wide[:, 5:69] = x
        a = api.head_loss_step(wide[:, 5:69], w, labels, row_weight=r)
        for p, q in zip(a, api.head_loss_step(x, w, labels, row_weight=r)):
            assert torch.equal(p, q)


def test_function(api):
    """Batches of sequences, a sliced head off 16-byte boundaries, gradients that add to others'."""
    x, w, labels, t, ids, r = draw(24, 48, 301, F32, top=5)
    big = torch.zeros((302, 48), device="cuda")
    big[1:] = w
    x3 = x.view(4, 6, 48).clone().requires_grad_()
    head = big.clone().requires_grad_()
    loss = api.HeadLossFunction.apply(x3, head[1:], labels.view(4, 6), t.view(4, 6, 5), ids.view(4, 6, 5), 2.0, 0.5)
    assert loss.shape == (4, 6)
    (loss * r.view(4, 6)).sum().backward()
    want = api.head_loss_step(x, w, labels, t, ids, r, temperature=2.0, mix=0.5)
    assert torch.equal(loss.detach().view(-1), want[0]) and torch.equal(x3.grad.view(24, 48), want[1])
    assert torch.equal(head.grad[1:], want[2]) and not head.grad[0].any()
    with pytest.raises(RuntimeError, match="second derivatives"):
        y = x.clone().requires_grad_()
        g, = torch.autograd.grad(api.HeadLossFunction.apply(y, w, labels, None, None).sum(), y, create_graph=True)
        g.sum().backward()


def test_refusals(api):
    x, w, labels, t, ids, r = draw(6, 16, 40, F32, top=3)
    ok = lambda **kw: api.head_loss_forward(**{**dict(x=x, w=w, labels=labels, teacher=t, ids=ids, mix=0.5), **kw})  # noqa: E731
    ok()
    for kw in (dict(x=x[0]), dict(w=w[:, :8]), dict(w=w.t()), dict(labels=labels[:5]), dict(teacher=None), dict(ids=None), dict(ids=ids[:, :2]),
               dict(teacher=t[:5]), dict(x=x.t()), dict(x=x.cpu()), dict(labels=labels.cpu()), dict(w=torch.zeros((40, 16)))):
        with pytest.raises(ValueError):
            ok(**kw)
    for kw in (dict(w=w.bfloat16()), dict(labels=labels.int()), dict(ids=ids.int()), dict(teacher=t.double()), dict(x=x.half(), w=w.half())):
        with pytest.raises(TypeError):
            ok(**kw)
    for kw in (dict(mix=1.5), dict(temperature=0.0)):
        with pytest.raises(RuntimeError):
            ok(**kw)
    loss, stats = api.head_loss_forward(x, w, labels)
    for bad in (stats[:-1], stats.double()):
        with pytest.raises(ValueError):
            api.head_loss_backward(r, x, w, labels, None, None, bad)
    with pytest.raises(ValueError):
        api.head_loss_backward(r[:5], x, w, labels, None, None, stats)


def test_stream_and_capture(api):
    """On a stream of the caller's, and captured: replays with other inputs, eager work between them."""
    x, w, labels, t, ids, r = draw(200, 64, 900, BF16, top=6, holes=True)
    how = dict(temperature=2.0, mix=0.5)
    want = api.head_loss_step(x, w, labels, t, ids, r, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.head_loss_step(x, w, labels, t, ids, r, stream=s, **how)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    sx, sl = x.clone(), labels.clone()
    with torch.cuda.stream(s):
        api.head_loss_step(sx, w, sl, t, ids, r, **how)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.head_loss_step(sx, w, sl, t, ids, r, **how)
    for k in range(4):
        x2, w2, l2, t2, i2, r2 = draw(200, 64, 900, BF16, top=6, holes=True, seed=30 + k)
        sx.copy_(x2)
        sl.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        eager = api.head_loss_step(x2, w, l2, t, ids, r, **how)
        for a, b in zip(out, eager):
            assert torch.equal(a, b), k
