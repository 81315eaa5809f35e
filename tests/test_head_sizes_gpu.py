"""The head loss of more rows or words than one launch takes workgroups for (2^22; 2^32 threads are a
launch's limit), against oracle/head.py under its derived bounds."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from oracle import head as H  # noqa: E402

U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required for the gpu-marked tests")
    from monarch_block_diagonal_amd import torch_api
    yield torch_api
    torch.cuda.empty_cache()


def near(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    off = ((got.double() - want).abs() - bound).max()
    assert float(off) <= 0, f"{what}: {float(off):.3g} past its bound, largest value {float(want.abs().max()):.3g}"


def test_many_rows(api):
    """More than four launches of a workgroup a row (rows copied, entries, their columns of g), two of four rows."""
    rows, d, vocab, T, mix = (1 << 24) + 261, 8, 24, 2.0, 0.5
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = rnd(rows, d).bfloat16(), rnd(vocab, d).bfloat16()
    labels = torch.randint(-2, vocab, (rows,), generator=g, device="cuda")
    t = rnd(rows, 2)
    first = torch.randint(-3, vocab, (rows, 1), generator=g, device="cuda")
    ids = torch.cat((first, (first + 5) % vocab), dim=1).contiguous()
    labels[:5], ids[:5] = -1, -1
    labels[-1] = 7
    r = torch.rand((rows,), generator=g, device="cuda") + 0.5
    o = H.head(x, w, labels, t, ids, r, T, mix)
    b_loss, b_dx, b_dw = H.bounds(o, x, w, U[x.dtype], T)
    # bounds() counts an addition a row for dw: of 256 splits of rows one adds 2^16 and a few in turn, and these
    # are added up
    b_dw -= (rows - 2 ** 17) * 2.0 ** -24 * (o.g.abs().T @ torch.where(o.used[:, None], x.double(), 0.0).abs())
    loss, dx, dw = api.head_loss_step(x, w, labels, t, ids, r, temperature=T, mix=mix)
    near(loss, o.loss, b_loss, "loss")
    near(dx, o.dx, b_dx, "dx")
    near(dw, o.dw, b_dw, "dw")
    assert not dx[~o.used].any() and not loss[~o.used].any() and o.used[-1]


def test_many_words(api):
    """An fp32 head of more words than one launch copies, in pieces of g."""
    rows, d, vocab = 40, 4, (1 << 24) + 300
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = torch.randn((rows, d), generator=g, device="cuda"), torch.randn((vocab, d), generator=g, device="cuda")
    labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    labels[0], labels[1], labels[2] = -1, 1, vocab - 1
    r = torch.rand((rows,), generator=g, device="cuda") + 0.5
    o = H.head(x, w, labels, None, None, r)
    b_loss, b_dx, b_dw = H.bounds(o, x, w, U[x.dtype])
    # Sums of exponentials: 128 words of a tile in turn, then 256 slices of the 131075 tiles, each joined by two
    # products and an addition: 128 + 3 * 513 + 8 roundings, 1e-4 of a sum.
    b_loss += 1e-4
    b_dx += 1e-4 * (o.s_g @ w.double().abs())
    b_dw += 1e-4 * (o.s_g.T @ x.double().abs())
    loss, dx, dw = api.head_loss_step(x, w, labels, row_weight=r)
    near(loss, o.loss, b_loss, "loss")
    near(dx, o.dx, b_dx, "dx")
    near(dw, o.dw, b_dw, "dw")
