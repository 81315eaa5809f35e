"""Pins of the distillation oracle (CPU): closed forms, finite differences, rows
with nothing to learn from."""
import numpy as np
import pytest

from oracle import distill as D


def draw(V=11, K=4, seed=3):
    r = np.random.default_rng(seed)
    return r.standard_normal(V) * 2, r.standard_normal(K), r.permutation(V)[:K]


def test_equal_distributions_cost_nothing():
    z = np.log(np.array([0.5, 0.25, 0.125, 0.125]))
    loss, dz, _, _ = D.row(z, z + 3.0, np.arange(4), None, 1.0, 1.0)
    assert abs(loss) < 1e-15
    np.testing.assert_allclose(dz, 0, atol=1e-15)


def test_one_entry_is_a_label():
    z, _, _ = draw()
    a = D.row(z, np.array([-7.0]), np.array([5]), None, 1.0, 1.0)
    b = D.row(z, np.zeros(0), np.zeros(0, np.int64), 5, 1.0, 0.0)
    assert abs(a[0] - b[0]) < 1e-14
    np.testing.assert_allclose(a[1], b[1], atol=1e-14)
    assert abs(b[0] - (np.log(np.exp(z).sum()) - z[5])) < 1e-14


@pytest.mark.parametrize("T,mix,label", [(1.0, 1.0, None), (2.0, 0.5, 3), (0.5, 0.25, 0), (3.0, 0.0, 10), (2.0, 0.5, -100)])
def test_gradient_against_differences(T, mix, label):
    z, t, ids = draw()
    loss, dz, _, _ = D.row(z, t, ids, label, T, mix)
    step = 1e-6
    for j in range(z.size):
        e = np.zeros_like(z)
        e[j] = step
        diff = (D.row(z + e, t, ids, label, T, mix)[0] - D.row(z - e, t, ids, label, T, mix)[0]) / (2 * step)
        assert abs(diff - dz[j]) < 1e-8, j
    # a softmax does not see a constant: the gradient sums to 0
    assert abs(dz.sum()) < 1e-13


def test_entries_that_are_not_there():
    z, t, ids = draw()
    base = D.row(z, t[:2], ids[:2], 1, 2.0, 0.5)
    more = D.row(z, np.concatenate([t[:2], [9.0, 9.0, -np.inf]]), np.concatenate([ids[:2], [-1, 11, ids[2]]]), 1, 2.0, 0.5)
    assert base[0] == more[0] and np.array_equal(base[1], more[1])


def test_entries_of_one_id_add_up():
    z, t, ids = draw()
    twice = D.row(z, np.array([0.3, 0.3]), np.array([4, 4]), None, 1.0, 1.0)
    once = D.row(z, np.array([0.3]), np.array([4]), None, 1.0, 1.0)
    np.testing.assert_allclose(twice[1], once[1], atol=1e-15)
    # every entry counts by itself in the loss: log(1/2) of each half
    assert abs(twice[0] - (once[0] - np.log(2.0))) < 1e-14


def test_rows_with_nothing():
    z, t, ids = draw()
    for row in (D.row(z, t, np.full(4, -1), None, 1.0, 1.0), D.row(z, t, ids, -100, 1.0, 0.0),
                D.row(np.full(11, np.nan), t, np.full(4, -1), -100, 1.0, 0.5),
                D.row(np.full(11, -np.inf), t, ids, 2, 1.0, 0.5)):
        assert row[0] == 0 and not row[1].any()


def test_masked_logits():
    z, t, ids = draw()
    z[[j for j in range(11) if j not in ids][:3]] = -np.inf
    loss, dz, _, _ = D.row(z, t, ids, None, 2.0, 1.0)
    assert np.isfinite(loss) and np.isfinite(dz).all() and (dz == 0).sum() == 3
    z[ids[0]] = -np.inf   # the teacher wants what the student may not say
    assert np.isinf(D.row(z, t, ids, None, 2.0, 1.0)[0])


def test_a_planted_mistake_is_seen():
    """The temperature's power: T^2 in the loss makes T in the gradient."""
    z, t, ids = draw()
    step, j = 1e-6, int(draw()[2][0])
    e = np.zeros_like(z)
    e[j] = step
    diff = (D.row(z + e, t, ids, None, 3.0, 1.0)[0] - D.row(z - e, t, ids, None, 3.0, 1.0)[0]) / (2 * step)
    dz = D.row(z, t, ids, None, 3.0, 1.0)[1][j]
    assert abs(diff - dz) < 1e-8 < abs(diff - 3.0 * dz)
