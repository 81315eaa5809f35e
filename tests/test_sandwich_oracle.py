"""Pins of the sandwich-norm oracle (CPU): closed forms, finite differences,
special cases that reduce to simpler formulas."""
import itertools

import numpy as np
import pytest

from oracle import sandwich as S

KINDS = ("none", "rms", "layer")


def inputs(rows, d, gates, bias, seed=5):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    return dict(h=n(rows, d), y=n(rows, d) + 0.3, post_w=1 + 0.3 * n(d), post_b=n(d) if bias else None,
                gate=n(gates, d) if gates else None, pre_w=1 + 0.3 * n(d),
                pre_b=n(d) if bias else None)


def test_norms_of_a_known_row():
    v = np.array([[3.0, -4.0, 0.0, 0.0]])
    rms = np.sqrt(25.0 / 4.0)
    np.testing.assert_allclose(S.norm(v, "rms", 0.0)[0], v / rms, rtol=1e-15)
    c = v + 0.25
    np.testing.assert_allclose(S.norm(v, "layer", 0.0)[0], c / np.sqrt((c * c).mean()), rtol=1e-15)
    np.testing.assert_array_equal(S.norm(v, "none", 0.0)[0], v)


def test_rows_of_one_feature_and_equal_features():
    # a layer norm of equal features is 0, its gradient 0 (eps keeps rho finite)
    v = np.full((2, 5), 7.0)
    assert np.all(S.norm(v, "layer", 1e-5)[0] == 0)
    np.testing.assert_allclose(S.norm_grad(np.ones((2, 5)), v, "layer", 1e-5), 0, atol=1e-12)
    one = np.array([[-2.0]])
    np.testing.assert_allclose(S.norm(one, "rms", 0.0)[0], [[-1.0]])


def test_no_norms_is_a_gated_residual():
    a = inputs(4, 6, 2, False)
    h_out, n = S.forward(a["h"], a["y"], gate=a["gate"], post="none", pre="none", skip=0.5, branch=3.0)
    assert n is None
    want = 0.5 * a["h"] + 3.0 * np.concatenate([a["gate"][:1]] * 2 + [a["gate"][1:]] * 2) * a["y"]
    np.testing.assert_allclose(h_out, want, rtol=1e-14)


@pytest.mark.parametrize("post,pre", itertools.product(KINDS, KINDS))
@pytest.mark.parametrize("gates,bias", [(0, False), (1, True), (2, True), (6, False)])
def test_gradients_against_differences(post, pre, gates, bias):
    rows, d, step = 6, 5, 1e-6
    a = inputs(rows, d, gates, bias)
    kw = dict(post=post, pre=pre, skip=0.7, branch=-1.3, eps=1e-3)
    if pre == "none":
        a["pre_w"] = a["pre_b"] = None
    r = np.random.default_rng(9)
    dh, dn = r.standard_normal((rows, d)), r.standard_normal((rows, d))

    def total(b):
        h_out, n = S.forward(**b, **kw)
        return (dh * h_out).sum() + (0.0 if n is None else (dn * n).sum())

    g = S.backward(dh, dn, a["h"], a["y"], a["post_w"], a["post_b"], a["gate"], a["pre_w"], a["pre_b"], **kw)
    names = {"h": "dh", "y": "dy", "post_w": "dpost_w", "post_b": "dpost_b", "gate": "dgate",
             "pre_w": "dpre_w", "pre_b": "dpre_b"}
    for key, name in names.items():
        if a[key] is None:
            continue
        flat = a[key].reshape(-1)
        for i in range(0, flat.size, 3):
            b = dict(a)
            up, down = flat.copy(), flat.copy()
            up[i] += step
            down[i] -= step
            b[key] = up.reshape(a[key].shape)
            hi = total(b)
            b[key] = down.reshape(a[key].shape)
            # central difference: error ~ step^2 times third derivatives, and rounding ~ 1e-16 / step
            assert abs((hi - total(b)) / (2 * step) - g[name].reshape(-1)[i]) < 1e-6, (name, i)


@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_norm_before_the_first_block(pre):
    a = inputs(3, 8, 0, True)
    h_out, n = S.forward(a["h"], None, pre_w=a["pre_w"], pre_b=a["pre_b"], pre=pre)
    assert h_out is not None and np.array_equal(h_out, a["h"])
    np.testing.assert_allclose(n, S.norm(a["h"], pre, 1e-5)[0] * a["pre_w"] + a["pre_b"])
    g = S.backward(None, n, a["h"], None, pre_w=a["pre_w"], pre_b=a["pre_b"], pre=pre)
    # a norm ignores the scale of its row: its gradient stands (up to eps) at a right angle to the centred row
    assert np.all(np.abs((g["dh"] * a["h"]).sum(axis=1)) < 1e-3)
    assert set(g) == {"dh", "dpre_w", "dpre_b"}


def test_a_planted_mistake_is_seen():
    """Leaving out the projection on the row (here, in the oracle's place) breaks the difference test."""
    v = np.random.default_rng(1).standard_normal((1, 6))
    dq = np.random.default_rng(2).standard_normal((1, 6))
    rho = S.norm(v, "rms", 1e-3)[2]
    step = 1e-6
    e = np.zeros((1, 6))
    e[0, 2] = step
    diff = ((dq * S.norm(v + e, "rms", 1e-3)[0]).sum() - (dq * S.norm(v - e, "rms", 1e-3)[0]).sum()) / (2 * step)
    assert abs(diff - S.norm_grad(dq, v, "rms", 1e-3)[0, 2]) < 1e-6
    assert abs(diff - (rho * dq)[0, 2]) > 1e-3
