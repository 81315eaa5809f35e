"""Pins of the head loss's and dropout's oracles (CPU)."""
import numpy as np
import pytest

from oracle import distill, dropout
torch = pytest.importorskip("torch")
from oracle import head as H  # noqa: E402


def inputs(rows=7, d=5, vocab=23, top=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(rows, d, generator=g).double(), torch.randn(vocab, d, generator=g).double()
    t = torch.randn(rows, top, generator=g) * 2
    ids = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(rows)])
    labels = torch.randint(0, vocab, (rows,), generator=g)
    r = torch.rand(rows, generator=g) + 0.5
    ids[1] = -1
    labels[1] = -100
    labels[2] = -1
    ids[3, 1] = ids[3, 0]
    ids[4, 2] = vocab
    t[5, 1] = float("-inf")
    return x, w, labels, t, ids, r


@pytest.mark.parametrize("T,mix", [(1.0, 0.0), (2.0, 0.5), (0.7, 1.0), (1.0, 0.3)])
def test_is_the_distillation_loss_of_the_products(T, mix):
    x, w, labels, t, ids, r = inputs()
    o = H.head(x, w, labels, t, ids, r, T, mix)
    loss, dz, sl, sd = distill.rows((x @ w.T).numpy(), t.double().numpy(), ids.numpy(), labels.numpy(), r.numpy(), T, mix)
    assert np.allclose(o.loss, loss, rtol=1e-12, atol=1e-12)
    assert np.allclose(o.g, dz, rtol=1e-12, atol=1e-13)
    assert np.allclose(o.s_loss, sl, rtol=1e-12) and np.allclose(o.s_g, sd, rtol=1e-12, atol=1e-15)
    assert float(o.loss[1]) == 0 and not o.dx[1].any()


@pytest.mark.parametrize("T,mix", [(1.0, 0.0), (2.0, 0.5), (0.7, 1.0)])
def test_gradients_are_differences(T, mix):
    x, w, labels, t, ids, r = inputs(seed=3)
    o = H.head(x, w, labels, t, ids, r, T, mix)
    total = lambda a, b: float((H.head(a, b, labels, t, ids, None, T, mix).loss * r).sum())  # noqa: E731
    g = torch.Generator().manual_seed(9)
    for _ in range(4):
        dx, dw = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
        e = 1e-5
        by = (total(x + e * dx, w + e * dw) - total(x - e * dx, w - e * dw)) / (2 * e)
        # the central difference is off by e^2 times a third derivative of order 100
        assert abs(by - float((o.dx * dx).sum() + (o.dw * dw).sum())) < 1e-6


def test_rows_left_out_hold_anything():
    x, w, labels, t, ids, r = inputs()
    a = H.head(x, w, labels, t, ids, r, 2.0, 0.5)
    x[1], r[1] = float("nan"), float("nan")
    b = H.head(x, w, labels, t, ids, r, 2.0, 0.5)
    assert torch.equal(a.dw, b.dw) and torch.equal(a.dx, b.dx) and torch.equal(a.loss, b.loss)


def test_philox_known_answers():
    """The generator's published known answers (counter, key, output)."""
    kat = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
           ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
           ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
            (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for ctr, key, out in kat:
        assert tuple(int(v) for v in dropout.philox(np.array([ctr], dtype=np.uint64), key)[0]) == out


def test_draws_by_place():
    d = dropout.draws(100, 12345678901234, 7)
    assert np.array_equal(dropout.draws(31, 12345678901234, 7, first=13), d[13:44])
    assert not np.array_equal(dropout.draws(100, 12345678901234, 8), d)
    x = np.ones(1 << 16)
    y, keep = dropout.dropout(x, 0.25, 3, 4)
    # 65536 draws at 3/4: the mean is off by less than 5 standard deviations of sqrt(3/16 / 65536)
    assert abs(keep.mean() - 0.75) < 5 * (3 / 16 / 65536) ** 0.5
    assert np.array_equal(y, np.where(keep, 4 / 3, 0.0))
    assert not dropout.dropout(x, 1.0, 3, 4)[1].any() and dropout.dropout(x, 0.0, 3, 4)[1].all()
