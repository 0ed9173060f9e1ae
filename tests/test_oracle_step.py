"""The float64 oracle of the training-step operators: its gradients against
central differences of its own values, and closed forms.  CPU only."""

import math

import numpy as np
import pytest

from oracle import step


def central(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


# A central difference with h = 1e-5 is off by h^2 f''' / 6 (1e-10 times a
# third derivative of order one) and by rounding (1e-16 / h = 1e-11).
TOL = dict(rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_ff_gradients_against_differences(act):
    rng = np.random.default_rng(0)
    x, wg, wu = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 5))
    dh = rng.normal(size=(3, 4))
    dx, dwg, dwu, _, _ = step.gated_ff_backward(x, wg, wu, dh, act)
    np.testing.assert_allclose(dx, central(lambda v: (step.gated_ff(v, wg, wu, act) * dh).sum(), x), **TOL)
    np.testing.assert_allclose(dwg, central(lambda v: (step.gated_ff(x, v, wu, act) * dh).sum(), wg), **TOL)
    np.testing.assert_allclose(dwu, central(lambda v: (step.gated_ff(x, wg, v, act) * dh).sum(), wu), **TOL)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(rest):
    rng = np.random.default_rng(1)
    z, teacher, tau = rng.normal(size=(3, 9)), rng.normal(size=(3, 9)), 1.7
    idx = np.array([[2, 5, 8], [0, -1, 3], [7, 1, -1]])
    top = np.take_along_axis(teacher, np.maximum(idx, 0), 1)
    lse = np.log(np.exp(teacher / tau).sum(1)) if rest else None
    w = np.array([1.0, 0.5, 0.0])
    loss, dz = step.distill(z, idx, top, lse, tau, w)
    assert loss[2] == 0 and not dz[2].any()
    assert (loss[:2] > 0).all()  # a divergence between different distributions
    np.testing.assert_allclose(dz, central(lambda v: step.distill(v, idx, top, lse, tau, w)[0].sum(), z), **TOL)


def test_distill_of_a_full_list_is_the_divergence():
    rng = np.random.default_rng(2)
    z, teacher = rng.normal(size=(1, 6)), rng.normal(size=(1, 6))
    p = np.exp(teacher) / np.exp(teacher).sum()
    q = np.exp(z) / np.exp(z).sum()
    idx = np.arange(6)[None]
    for lse in (None, np.log(np.exp(teacher).sum(1))):
        loss, dz = step.distill(z, idx, teacher, lse)
        assert loss[0] == pytest.approx((p * np.log(p / q)).sum(), rel=1e-12)
        np.testing.assert_allclose(dz, q - p, atol=1e-15)


def test_policy_gradient_against_differences():
    rng = np.random.default_rng(3)
    n = 24
    z = rng.normal(size=(n, 7))
    action = rng.integers(0, 7, n)
    action[3] = -1
    adv = rng.normal(size=n)
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1, tau=0.8)
    logp = step.policy(z, action, adv, tau=0.8)[1]
    old, ref = logp + 0.4 * rng.normal(size=n), logp + rng.normal(size=n)
    loss, _, kl, dz = step.policy(z, action, adv, old, ref, **kw)
    r = np.exp(logp - old)
    assert ((r < 0.8) | (r > 1.3)).any() and ((r > 0.8) & (r < 1.3)).any()
    assert loss[3] == 0 and not dz[3].any() and (kl >= 0).all()
    np.testing.assert_allclose(dz, central(lambda v: step.policy(v, action, adv, old, ref, **kw)[0].sum(), z), **TOL)


@pytest.mark.parametrize("eps", [0.0, 0.2])
def test_preference_gradient_against_differences(eps):
    rng = np.random.default_rng(4)
    offsets = [1, 4, 4, 7, 9]  # row 0 in no sequence, one empty sequence
    z = rng.normal(size=(9, 6))
    target = rng.integers(0, 6, 9)
    target[5] = -1
    ref = -rng.random(9) * 3
    w = [1.0, 0.5]
    loss, reward, dz = step.preference(z, target, offsets, ref, 0.7, eps, w)
    assert reward[1] == 0 and not dz[0].any() and not dz[5].any()
    np.testing.assert_allclose(dz, central(lambda v: step.preference(v, target, offsets, ref, 0.7, eps, w)[0].sum(), z), **TOL)
    assert step.preference(z, target, [0, 0, 0], ref, 0.7, eps)[0][0] == pytest.approx(math.log(2))
