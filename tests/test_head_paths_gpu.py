"""The head loss on every path that its plan may take, large tiles first. Each test names the kernels that it is for, and
asks the library (monarch_head_describe) whether the call takes them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from monarch_block_diagonal_amd import binding as B  # noqa: E402
from oracle import head as H  # noqa: E402
from test_head_gpu import U, api, check, draw, near  # noqa: E402,F401

F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def takes(x, w, top, *kernels):
    rows, d = x.shape
    code = B.BF16 if x.dtype == BF16 else B.F32
    step = B.monarch_head_describe(B.HEAD_STEP, rows, d, w.shape[0], top, code)
    assert set(kernels) <= set(step), (kernels, step)
    # a forward and a backward pass take the same tiles
    for call in (B.HEAD_FWD, B.HEAD_BWD):
        names = B.monarch_head_describe(call, rows, d, w.shape[0], top, code)
        for kind in ("head_sums", "head_grad", "head_products"):
            mine = [k for k in names if k.startswith(kind)]
            assert not mine or mine == [k for k in step if k.startswith(kind)]


@TYPES
@pytest.mark.parametrize("T,mix", [(1.0, 0.0), (2.0, 0.5), (1.3, 0.7), (1.0, 1.0)])
@pytest.mark.parametrize("d", [776, 777])
def test_large_tiles(api, d, T, mix, dtype):  # noqa: F811
    """256 x 256 tiles in all three products and every epilogue: 12 K tiles and a part of one over the features (the loop's
    middle runs from 5 on), 17 and a part over the rows, hundreds over the words; rows, words and features that end inside a tile."""
    top = 7 if mix else 0
    x, w, labels, t, ids, r = draw(1100, d, 30011, dtype, top=top, holes=True, seed=31)
    takes(x, w, top, "head_sums_256", "head_grad_256", "head_products_256")
    check(api, x, w, labels, t, ids, r, T, mix)


@TYPES
@pytest.mark.parametrize("T,mix", [(1.0, 0.0), (2.0, 0.5), (1.3, 0.7)])
@pytest.mark.parametrize("rows,d,vocab", [(700, 520, 3001), (333, 415, 6000)])
def test_small_tiles_with_many_steps(api, rows, d, vocab, T, mix, dtype):  # noqa: F811
    """128 x 128 tiles with more K tiles than are in flight."""
    top = 3 if mix else 0
    x, w, labels, t, ids, r = draw(rows, d, vocab, dtype, top=top, holes=True, seed=33)
    takes(x, w, top, "head_sums_128", "head_grad_128", "head_products_128")
    check(api, x, w, labels, t, ids, r, T, mix)


@pytest.mark.parametrize("rows,vocab,dtype", [(5200, 70001, F32), (16400, 70001, BF16)], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,mix", [(2.0, 0.5), (1.3, 0.7)])
def test_pieces_with_entries(api, rows, vocab, dtype, T, mix):  # noqa: F811
    """Three pieces of the vocabulary in large tiles: later ones' sums for dx are added to the first one's, and
    entries and labels lie in each, also at the borders between them."""
    x, w, labels, t, ids, r = draw(rows, 136, vocab, dtype, top=5, holes=True, seed=35)
    takes(x, w, 5, "head_grad_256*3", "head_taught*3", "head_products_256*3")
    third = (vocab // 3 + 256) // 256 * 256
    for k, at in enumerate((third - 1, third, 2 * third - 1, 2 * third, vocab - 1)):
        labels[k], ids[100 + k, 0], ids[100 + k, 2] = at, at, at
    check(api, x, w, labels, t, ids, r, T, mix)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,d,vocab,dtype,kernels", [
    (20, 8, 4300003, BF16, ("head_thin_grad*2", "head_products_32*2")), (20, 8, 1500007, F32, ("head_thin_grad*2", "head_few_products*2")),
    (20, 6, 1500007, F32, ("head_grad_32*2", "head_few_products*2")), (50, 16, 4300003, BF16, ("head_grad_128*2", "head_products_128*2"))])
def test_pieces_of_few_rows_with_entries(api, rows, d, vocab, dtype, kernels):  # noqa: F811
    x, w, labels, t, ids, r = draw(rows, d, vocab, dtype, top=3, holes=True, seed=37)
    takes(x, w, 3, "head_taught*2", *kernels)
    half = (vocab // 2 + 255) // 256 * 256
    for k, at in enumerate((half - 1, half, vocab - 1)):
        labels[k], ids[4 + k, 0], ids[4 + k, 1] = at, at, at
    o = H.head(x, w, labels, t, ids, r, 1.3, 0.7)
    b_loss, b_dx, b_dw = H.bounds(o, x, w, U[dtype], 1.3)
    # bounds() has sums of exponentials of up to 2^17 terms. Up to 32 rows a workgroup takes a 256th of the words, 64 at a
    # time, of which a lane adds four and then scales its sum: 263 * 5 roundings, a few to join lanes and workgroups. Above, 128
    # words a tile, and a 256th of 33600 tiles in turn, each by two products and an addition: 128 + 400. So under 2^11, 1.3e-4.
    b_loss += 1.3e-4 * 1.3 ** 2
    e_g = 1.3e-4 * o.s_g
    b_dx += e_g @ w.double().abs()
    b_dw += e_g.T @ torch.where(o.used[:, None], x.double(), 0.0).abs()
    loss, dx, dw = api.head_loss_step(x, w, labels, t, ids, r, temperature=1.3, mix=0.7)
    near(loss, o.loss, b_loss, "loss")
    near(dx, o.dx, b_dx, "dx")
    near(dw, o.dw, b_dw, "dw")


@pytest.mark.parametrize("d", [4104, 4099])
@pytest.mark.parametrize("rows", [5, 32, 50])
def test_few_wide_rows(api, rows, d):  # noqa: F811
    """Few rows of more features than one workgroup copies, g in two parts."""
    x, w, labels, t, ids, r = draw(rows, d, 700, BF16, top=2, holes=True, seed=39)
    takes(x, w, 2, "head_copy_x")
    check(api, x, w, labels, t, ids, r, 2.0, 0.5)


@TYPES
@pytest.mark.parametrize("rows,d", [(1, 64), (9, 72), (17, 37), (32, 264), (5, 4104), (50, 96), (300, 65)])
def test_rows_apart_and_unaligned(api, rows, d, dtype):  # noqa: F811
    """Rows of x that lie apart, off 16-byte boundaries, NaN between them: bit for bit what close rows give."""
    x, w, labels, t, ids, r = draw(rows, d, 500, dtype, top=3, seed=41)
    how = dict(temperature=2.0, mix=0.5)
    want = api.head_loss_step(x, w, labels, t, ids, r, **how)
    for shift, more in ((5, 13), (8, 8), (1, 0)):
        wide = torch.full((rows, d + shift + more), float("nan"), dtype=dtype, device="cuda")
        wide[:, shift:shift + d] = x
        for p, q in zip(api.head_loss_step(wide[:, shift:shift + d], w, labels, t, ids, r, **how), want):
            assert torch.equal(p, q)


def test_large_tiles_captured(api):  # noqa: F811
    """Captured and replayed with other inputs, eager work between the replays."""
    x, w, labels, t, ids, r = draw(1100, 776, 30011, BF16, top=7, holes=True, seed=43)
    takes(x, w, 7, "head_sums_256", "head_grad_256", "head_products_256")
    how = dict(temperature=2.0, mix=0.5)
    sx, sl = x.clone(), labels.clone()
    api.head_loss_step(sx, w, sl, t, ids, r, **how)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.head_loss_step(sx, w, sl, t, ids, r, **how)
    for k in range(3):
        x2, _, l2, _, _, _ = draw(1100, 776, 30011, BF16, top=7, holes=True, seed=50 + k)
        sx.copy_(x2)
        sl.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, api.head_loss_step(x2, w, l2, t, ids, r, **how)):
            assert torch.equal(a, b), k
