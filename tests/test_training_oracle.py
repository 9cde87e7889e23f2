"""The fp64 definitions of the training-step operators: their gradients against central
differences, and closed forms."""
import math

import numpy as np
import pytest

from oracle import training as TR


def central(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("reduction", ["sum", "token_mean", "seq_mean"])
def test_policy_gradient_is_the_losses(kl, reduction):
    rng = np.random.default_rng(1)
    T, offsets = 23, [2, 9, 9, 20]
    old = -np.abs(rng.standard_normal(T))
    lp = old + 0.3 * rng.standard_normal(T)
    ref = old + 0.2 * rng.standard_normal(T)
    active = (rng.random(T) < 0.8).astype(np.uint8)
    kw = dict(ref=ref, active=active, offsets=offsets, per_seq=True, dual_clip=1.5, kl=kl,
              kl_coef=0.3, reduction=reduction, scale=0.7)
    adv = np.array([1.3, 0.2, -0.9])
    _, _, grad, _ = TR.policy_loss(lp, old, adv, **kw)
    num = central(lambda v: TR.policy_loss(v, old, adv, **kw)[0], lp)
    # the loss is smooth away from the clip's borders, which these draws keep clear of
    assert np.abs(grad - num).max() <= 1e-8


def test_policy_closed_forms():
    lp = np.array([-1.0, -1.0, -1.0])
    old = lp - np.log([1.5, 1.1, 0.5])
    loss, stats, grad, _ = TR.policy_loss(lp, old, [1.0, 1.0, -1.0], reduction="sum")
    # 1.5 is clipped to 1.2, 1.1 stays, and 0.5 with a negative advantage is clipped to 0.8
    assert abs(loss - (-1.2 - 1.1 + 0.8)) < 1e-12 and stats[2] == 2.0
    assert np.allclose(grad, [0.0, -1.1, 0.0], atol=1e-12)
    # no tokens, no loss
    assert TR.policy_loss(lp, old, [1.0] * 3, active=[0, 0, 0])[0] == 0.0


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("layout", ["adjacent", "halves"])
def test_preference_gradient_is_the_losses(kind, layout):
    rng = np.random.default_rng(2)
    offsets = [1, 5, 5, 9, 14]
    lp = rng.standard_normal(16)
    kw = dict(ref=rng.standard_normal(16), active=(rng.random(16) < 0.8).astype(np.uint8),
              beta=0.4, kind=kind, layout=layout, length_normalize=True, scale=1.7,
              label_smoothing=0.1 if kind == "sigmoid" else 0.0,
              margin=0.25 if kind != "ipo" else 0.0)
    grad = TR.preference_loss(lp, offsets, **kw)[3]
    num = central(lambda v: TR.preference_loss(v, offsets, **kw)[0], lp)
    assert np.abs(grad - num).max() <= 1e-8


def test_preference_of_equal_sequences_is_log_2():
    lp = np.array([-0.5, -1.0, -0.5, -1.0])
    loss, _, rewards, _, _ = TR.preference_loss(lp, [0, 2, 4])
    assert abs(loss - math.log(2)) < 1e-15 and rewards[0] == rewards[1]


def test_rmsnorm_gradient_is_the_norms():
    rng = np.random.default_rng(3)
    x, gamma = rng.standard_normal((3, 6)), 1 + 0.1 * rng.standard_normal(6)
    dy, eps = rng.standard_normal((3, 6)), 1e-3

    def f(xv, gv):
        return float((dy * xv / np.sqrt((xv * xv).mean(1, keepdims=True) + eps) * gv).sum())
    dx, dg = TR.rmsnorm_backward(dy, x, gamma, eps)
    assert np.abs(dx - central(lambda v: f(v, gamma), x)).max() <= 1e-8
    assert np.abs(dg - central(lambda v: f(x, v), gamma)).max() <= 1e-8


def test_clip_scale():
    assert TR.clip_scale([np.array([3.0]), np.array([4.0])], 1.0) == (5.0, 0.2)
    assert TR.clip_scale([np.array([3.0])], 3.0) == (3.0, 1.0)
    assert TR.clip_scale([np.array([np.inf])], 1.0)[1] == 1.0
