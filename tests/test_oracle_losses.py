"""Pins of the losses' and the optimizer's oracle: gradients against central differences, closed
forms, planted mistakes that the differences must catch, what stochastic rounding keeps."""
import math

import numpy as np
import pytest

from oracle import losses as ls
from test_oracle_training import TOL, _diff


def _rows(rng, m=5, v=7):
    z = rng.normal(size=(m, v)) * 2
    y = rng.integers(0, v, m)
    return z, y


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_token_gradient_is_the_difference(scale):
    rng = np.random.default_rng(1)
    z, y = _rows(rng)
    y[2] = -1
    on = y >= 0
    a, h = rng.normal(size=5), rng.normal(size=5)

    def f():
        lp, _, ent, _, _ = ls.token_stats(z, y, scale)
        return float((on * (a * lp + h * ent)).sum())
    d = ls.token_gradient(z, y, a, h, scale)
    assert np.abs(d - _diff(f, z)).max() < TOL
    assert (d[2] == 0).all()
    # a gradient without the entropy's share is seen
    assert np.abs(ls.token_gradient(z, y, a, None, scale) - d).max() > 1e3 * TOL


def test_token_stats_closed_forms():
    z = np.zeros((1, 8))
    lp, lse, h, p, _ = ls.token_stats(z, np.array([3]))
    assert np.allclose([lp[0], lse[0], h[0]], [-math.log(8), math.log(8), math.log(8)])
    z[0, 1:] = -np.inf   # one column alone
    lp, lse, h, p, _ = ls.token_stats(z, np.array([0]))
    assert (lp[0], lse[0], h[0]) == (0, 0, 0)


@pytest.mark.parametrize("old,ref,mean,weighted", [(True, True, True, False), (False, True, False, True),
                                                   (True, False, True, True), (True, True, False, False)])
def test_policy_gradient_is_the_difference(old, ref, mean, weighted):
    rng = np.random.default_rng(2)
    z, y = _rows(rng, 9)
    y[4] = -1
    lp = ls.token_stats(z, y)[0]
    # ratios of 1.6 and 0.6 in turn: both sides of the clipping, with advantages of either sign
    o = lp + np.where(np.arange(9) % 2, 0.5, -0.5) + 0.1 * rng.normal(size=9) if old else None
    k = dict(adv=rng.normal(size=9), ref=lp + rng.normal(size=9) * 0.5 if ref else None,
             weights=np.where(np.arange(9) == 6, 0.0, rng.uniform(0.5, 2, 9)) if weighted else None, low=0.2, high=0.3,
             kl_coef=0.1 if ref else 0.0, ent_coef=0.05, mean=mean)
    # without old log-probabilities the ratio is taken to the present policy, held fixed
    fixed = lp.copy()
    f = lambda: float(ls.policy_loss(z, y, old=fixed if o is None else o, **k)[0][0])  # noqa: E731
    stats, logp, d, _, _ = ls.policy_loss(z, y, old=o, **k)
    assert np.abs(d - _diff(f, z)).max() < TOL
    assert (d[4] == 0).all() and logp[4] == 0 and (not weighted or (d[6] == 0).all())
    if old:
        assert stats[2] > 0


def test_policy_loss_of_nothing_is_zero():
    stats, logp, d, _, _ = ls.policy_loss(np.full((3, 4), np.nan), np.full(3, -1), np.ones(3))
    assert (stats == 0).all() and (logp == 0).all() and (d == 0).all()


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("smoothing,average,margin", [(0.0, False, 0.0), (0.2, True, 0.3)])
def test_preference_gradient_is_the_difference(kind, smoothing, average, margin):
    rng = np.random.default_rng(3)
    z, y = _rows(rng, 14)
    y[[3, 8]] = -1
    off = np.array([0, 4, 4, 7, 9, 12, 14])  # three pairs, an empty sequence among them
    ref = rng.normal(size=14) - 2
    k = dict(ref=ref, kind=kind, beta=0.4, smoothing=smoothing, average=average, margin=margin)
    loss, margins, logp, d, _ = ls.preference_loss(z, y, off, **k)
    assert np.abs(d - _diff(lambda: float(ls.preference_loss(z, y, off, **k)[0]), z)).max() < TOL
    assert margins.shape == (3,) and (d[[3, 8]] == 0).all()


def test_preference_of_equal_sequences():
    z = np.tile(np.arange(5.0), (4, 1))
    loss, margins, _, _, _ = ls.preference_loss(z, np.array([1, 2, 1, 2]), np.array([0, 2, 4]))
    assert margins[0] == 0 and np.isclose(loss, math.log(2))


def test_adamw_first_step_is_the_sign():
    w, g = np.array([1.0, -2.0, 3.0]), np.array([0.5, -1e-3, 0.0])
    got, m, v = ls.adamw(w, g, np.zeros(3), np.zeros(3), 1, 0.1, eps=0.0 + 1e-30, weight_decay=0.0)
    assert np.allclose(got, w - 0.1 * np.sign(g))
    got, _, _ = ls.adamw(w, g, np.zeros(3), np.zeros(3), 1, 0.1, weight_decay=0.5)
    assert np.allclose(got - w, -0.1 * np.sign(g) - 0.05 * w, atol=1e-5)  # eps 1e-8 beside 1e-3


def test_random_words_are_even():
    w = ls.words(12345678901234567, 7, 3, 1 << 16)
    bits = (w[:, None] >> np.arange(32, dtype=np.uint64)) & np.uint64(1)
    # 65536 draws of a half: the mean's standard deviation is 0.00195; 5.5 of them
    assert np.abs(bits.mean(0) - 0.5).max() < 0.0107
    for other in (ls.words(12345678901234567, 8, 3, 1 << 16), ls.words(12345678901234567, 7, 4, 1 << 16),
                  ls.words(12345678901234567 + (1 << 40), 7, 3, 1 << 16)):
        assert (w == other).mean() < 1e-3


def test_packed_states_are_neighbours_and_right_in_the_mean():
    rng = np.random.default_rng(5)
    n = 700
    m, v = rng.normal(size=n) * 1e-3, (rng.normal(size=n) * 1e-3) ** 2
    v[10] = 0
    means = np.zeros(n), np.zeros(n)
    turns = 400
    for s in range(turns):
        mq, scale, code, low, gap, _, _ = ls.pack(m, v, ls.words(s, 1, 0, n))
        a, b = ls.unpack(mq, scale, code, low, gap)
        big = np.repeat(scale, 256)[:n]
        step = ls.e4m3_step(m / big) * big
        ratio = np.exp2(np.repeat(gap, 256)[:n])
        assert (np.abs(a - m) <= step * (1 + 1e-9)).all()
        kept = np.where(v > 0, np.maximum(v, np.exp2(np.repeat(low, 256)[:n])), 1.0)  # (2^-24 of the largest at least)
        assert ((b / kept <= ratio * (1 + 1e-9)) & (kept / np.where(v > 0, b, 1) <= ratio * (1 + 1e-9)))[v > 0].all()
        assert b[10] == 0
        means[0][:] += a / turns
        means[1][:] += b / turns
    # the mean of 400 roundings: half a step each at most, five standard deviations
    assert (np.abs(means[0] - m) <= 5 * 0.5 * step / math.sqrt(turns) + 1e-12).all()
    kept, span = np.where(v > 0, kept, 0.0), np.where(v > 0, kept, 0.0) * (ratio - 1)
    # (the correction of the mean leaves a tenth of a percent of a step at the widest spacing)
    assert (np.abs(means[1] - kept) <= 5 * 0.5 * span / math.sqrt(turns) + 0.01 * span + 1e-30).all()


def test_eight_bit_averages_follow_a_constant_gradient():
    """m and v of a gradient that changed stay where they are when rounded to the nearest; rounded at random
    they arrive."""
    n, g = 256, 1e-3
    rng = np.random.default_rng(6)
    m, v = np.full(n, 0.75 * g) * rng.uniform(0.9, 1.1, n), np.full(n, 0.5 * g * g) * rng.uniform(0.5, 2, n)
    got = []
    for step in range(1, 1500):
        _, m, v = ls.adamw(np.zeros(n), np.full(n, g), m, v, step, 0.0)
        mq, scale, code, low, gap, _, _ = ls.pack(m, v, ls.words(9, step, 0, n))
        m, v = ls.unpack(mq, scale, code, low, gap)
        if step > 1400:
            got.append((m.mean(), v.mean()))
    a, b = np.mean(got, 0)
    # 256 elements x 10 independent times: m's spread of 8% and v's of 25% over 50; v has had 1500 steps of
    # its 1000: exp(-1.5) of the way (at most half of v) is left
    assert abs(a / g - 1) < 0.01
    assert abs(b / g ** 2 - 1) < 0.5 * math.exp(-1.4) + 0.03
