"""Pins of the training operators' oracle: gradients against central differences of the forward
definitions, closed forms, and planted mistakes that the differences must catch."""
import math

import numpy as np
import pytest

from oracle import training as tr


def _diff(f, x, h=1e-5):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        down = f()
        flat[i] = keep
        out[i] = (up - down) / (2 * h)
    return g


# central differences: truncation h^2 f''' ~ 1e-10, rounding 1e-16 / h ~ 1e-11 of values of order 10
TOL = 1e-7


@pytest.mark.parametrize("lq,lk,h,hkv,causal", [(5, 5, 2, 2, True), (4, 7, 4, 2, True), (6, 3, 2, 1, True),
                                                (3, 5, 3, 1, False), (1, 1, 1, 1, True)])
def test_attention_gradients_are_the_differences(lq, lk, h, hkv, causal):
    rng = np.random.default_rng(7 * lq + lk)
    q, k, v = rng.normal(size=(lq, h, 4)), rng.normal(size=(lk, hkv, 4)), rng.normal(size=(lk, hkv, 4))
    do = rng.normal(size=(lq, h, 4))
    o, lse, p = tr.attn_forward(q, k, v, causal)
    f = lambda: float((tr.attn_forward(q, k, v, causal)[0] * do).sum())  # noqa: E731
    dq, dk, dv = tr.attn_backward(q, k, v, o, lse, do, causal)[:3]
    for got, x in ((dq, q), (dk, k), (dv, v)):
        assert np.abs(got - _diff(f, x)).max() < TOL
    # rows without keys: nothing attends
    empty = ~tr.attn_mask(lq, lk, causal).any(1)
    assert np.isneginf(lse[:, empty]).all() and (o[empty] == 0).all() and (dq[empty] == 0).all()
    # a dropped delta is seen by the differences (one key per row would hide it)
    if lk > 1 and lq > 1:
        wrong = tr.attn_backward(q, k, v, 0 * o, lse, do, causal)[0]
        assert np.abs(wrong - dq).max() > 1e3 * TOL


def test_attention_rows_are_weighted_means():
    rng = np.random.default_rng(3)
    q, k = rng.normal(size=(6, 2, 8)), rng.normal(size=(6, 1, 8))
    o, lse, p = tr.attn_forward(q, k, np.ones((6, 1, 8)))
    assert np.allclose(o, 1.0) and np.allclose(p.sum(-1), 1.0)
    assert np.allclose(lse[:, 0], (q[0] @ k[0, 0]) / math.sqrt(8))  # the first query sees one key


@pytest.mark.parametrize("post,gate,pre,rest", [(True, "row", True, True), (False, None, True, True),
                                                (True, "token", False, True), (True, "row", True, False)])
def test_norm_gradients_are_the_differences(post, gate, pre, rest):
    rng = np.random.default_rng(11)
    m, c = 3, 5
    r, y = rng.normal(size=(m, c)), rng.normal(size=(m, c))
    w_post = rng.normal(size=c) if post else None
    w_pre = rng.normal(size=c) if pre else None
    g = {"row": rng.normal(size=c), "token": rng.normal(size=(m, c)), None: None}[gate]
    dx = rng.normal(size=(m, c)) if pre else None
    dr = rng.normal(size=(m, c)) if rest else None

    def f():
        r_out, x, _ = tr.norm_residual(r, y, w_post, g, w_pre, 0.75, 1e-3)
        return float((x * dx).sum() if pre else 0.0) + float((r_out * dr).sum() if rest else 0.0)

    r_out = tr.norm_residual(r, y, w_post, g, w_pre, 0.75, 1e-3)[0]
    got, _ = tr.norm_residual_backward(r_out, y, dx, dr, w_post, g, w_pre, 0.75, 1e-3)
    for name, x in (("r", r), ("y", y), ("w_post", w_post), ("gate", g), ("w_pre", w_pre)):
        if x is not None:
            assert np.abs(got[name] - _diff(f, x)).max() < TOL, name


def test_norm_rows_have_unit_mean_square():
    x = tr.norm_residual(np.random.default_rng(1).normal(size=(4, 64)) * 3, None, w_pre=np.ones(64), eps=0.0)[1]
    assert np.allclose((x * x).mean(-1), 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_pairs_and_keeps_lengths(interleaved):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 2, 10))
    freq, amp = tr.rope_frequencies(6, 10000.0)
    y = tr.rope(x, [0, 1, 5, 1000], freq, interleaved=interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(tr.rope(y, [0, 1, 5, 1000], freq, interleaved=interleaved, sign=-1.0), x)
    # scores depend on distances alone
    q, k = np.tile(x[:1], (4, 1, 1)), np.tile(x[1:2], (4, 1, 1))
    s = [(tr.rope(q, np.full(4, p + 7), freq, interleaved=interleaved) * tr.rope(k, np.full(4, p), freq, interleaved=interleaved)).sum(-1)
         for p in (0, 31)]
    assert np.allclose(s[0], s[1])


def test_rope_gradient_is_the_opposite_turn():
    rng = np.random.default_rng(9)
    x, d = rng.normal(size=(3, 1, 6)), rng.normal(size=(3, 1, 6))
    freq, amp = tr.rope_frequencies(4, 100.0, "ramped", 4.0, 1.0, 32.0, 4096)
    assert amp == 0.1 * math.log(4.0) + 1.0
    f = lambda: float((tr.rope(x, [2, 9, 4], freq, amp) * d).sum())  # noqa: E731
    assert np.abs(tr.rope(d, [2, 9, 4], freq, amp, sign=-1.0) - _diff(f, x)).max() < TOL


def test_rope_scalings():
    plain, _ = tr.rope_frequencies(128, 500000.0)
    assert np.allclose(tr.rope_frequencies(128, 500000.0, "linear", 4.0)[0], plain / 4)
    turns = 8192 * plain / (2 * math.pi)
    f = tr.rope_frequencies(128, 500000.0, "banded", 8.0, 1.0, 4.0, 8192)[0]
    assert np.allclose(f[turns > 4], plain[turns > 4]) and np.allclose(f[turns < 1], plain[turns < 1] / 8)
    assert (np.diff(f) < 0).all()
    f = tr.rope_frequencies(128, 10000.0, "ramped", 16.0, 1.0, 32.0, 4096)[0]
    plain = tr.rope_frequencies(128, 10000.0)[0]
    assert f[0] == plain[0] and np.isclose(f[-1], plain[-1] / 16) and (np.diff(f) < 0).all()
