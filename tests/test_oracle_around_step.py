"""The oracle of the step's norm, vocabulary cross entropy and orthogonalised update,
against differences and against what the singular values do.  CPU only."""

import numpy as np
import pytest

from oracle import step

MUON = (3.4445, -4.7750, 2.0315)


def central(f, v, at, h=1e-6):
    w = v.copy()
    w[at] += h
    up = f(w)
    w[at] -= 2 * h
    return (up - f(w)) / (2 * h)


def test_norm_gradients_by_differences():
    rng = np.random.default_rng(0)
    s, w, dy, ds = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    y, rstd = step.rms_norm(s, w, 1e-2)
    np.testing.assert_allclose(y, s / np.sqrt((s * s).mean(1, keepdims=True) + 1e-2) * w, rtol=1e-13)
    # the residual goes on beside the norm: ds is the gradient of that branch
    dx, dw = step.rms_norm_backward(s, w, rstd, dy, ds)
    total = lambda s, w: (step.rms_norm(s, w, 1e-2)[0] * dy).sum() + (s * ds).sum()  # noqa: E731
    for at in np.ndindex(3, 5):
        assert abs(central(lambda v: total(v, w), s, at) - dx[at]) < 1e-8
    for at in range(5):
        assert abs(central(lambda v: total(s, v), w, at) - dw[at]) < 1e-8


def test_cross_entropy_gradients_by_differences():
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(4, 3)), rng.normal(size=(6, 3))
    target, weight = [2, -1, 5, 0], [0.5, 1.0, 2.0, 0.25]
    loss, lse, dx, dw, dz = step.cross_entropy(x, w, target, weight)
    np.testing.assert_allclose(lse[[0, 2, 3]], np.log(np.exp(x @ w.T).sum(1))[[0, 2, 3]], rtol=1e-13)
    assert loss[1] == lse[1] == 0 and not dx[1].any() and not dz[1].any()
    total = lambda x, w: step.cross_entropy(x, w, target, weight)[0].sum()  # noqa: E731
    for at in np.ndindex(4, 3):
        assert abs(central(lambda v: total(v, w), x, at) - dx[at]) < 1e-8
    for at in np.ndindex(6, 3):
        assert abs(central(lambda v: total(x, v), w, at) - dw[at]) < 1e-8


def test_cross_entropy_of_rows_that_are_left_out_or_are_not_numbers():
    x = np.array([[1.0, 2.0], [np.nan, 0.0], [0.0, np.inf]])
    w = np.array([[1.0, 0.5], [0.0, 1.0]])
    loss, lse, dx, dw, _ = step.cross_entropy(x, w, [0, -1, 7])
    assert np.isfinite(loss).all() and np.isfinite(dw).all() and not dx[1:].any()
    loss, _, dx, dw, _ = step.cross_entropy(x, w, [0, 1, -1])
    assert np.isnan(loss[1]) and np.isnan(dx[1]).all() and np.isnan(dw).all() and np.isfinite(dx[0]).all()


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 7), (1, 1)])
def test_orthogonalise_acts_on_the_singular_values(shape):
    g = np.random.default_rng(2).normal(size=shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for a, b, c in [MUON] * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    np.testing.assert_allclose(step.orthogonalise(g, [MUON] * 5), (u * s) @ v, atol=1e-12)
    assert not step.orthogonalise(np.zeros(shape), [MUON]).any()
