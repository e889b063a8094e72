"""Slow fp64 definitions of the losses from logits and of the AdamW step, with the states' 8-bit
form.  Logits are [tokens, vocabulary] (all ranks' columns side by side)."""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------------------
# rows of logits
# ---------------------------------------------------------------------------
def token_stats(z, targets, scale=1.0):
    """(logp, lse, H, p, log p) of every row; rows without a target (negative) count as id 0."""
    z = scale * np.asarray(z, np.float64)
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.exp(z - top)
        log_s = np.log(e.sum(1, keepdims=True))
        lp = z - top - log_s
        p = np.exp(lp)
        h = -np.where(p > 0, p * lp, 0.0 * p).sum(1)
    y = np.maximum(targets, 0)
    return lp[np.arange(len(y)), y], (top + log_s)[:, 0], h, p, lp


def token_gradient(z, targets, a, h=None, scale=1.0):
    """dlogits of sum a logp + h H; rows without a target: 0."""
    _, _, ent, p, lp = token_stats(z, targets, scale)
    d = -a[:, None] * p
    if h is not None:
        d -= h[:, None] * p * (np.where(p > 0, lp, 0.0) + ent[:, None])
    y = np.maximum(targets, 0)
    d[np.arange(len(y)), y] += a
    d[targets < 0] = 0.0
    return scale * d


def policy_rows(logp, entropy, old, adv, ref, low, high, kl_coef, ent_coef):
    """Per token: (loss, KL term, clipped, dL/dlogp)"""
    ratio = np.exp(logp - (logp if old is None else old))
    free, held = ratio * adv, np.clip(ratio, 1 - low, 1 + high) * adv
    clipped = held < free
    x = np.zeros_like(logp) if ref is None else ref - logp
    kl = np.zeros_like(logp) if ref is None else np.expm1(x) - x
    loss = -np.minimum(free, held) + kl_coef * kl - ent_coef * entropy
    return loss, kl, clipped, np.where(clipped, 0.0, -free) - kl_coef * np.expm1(x)


def policy_loss(z, targets, adv, old=None, ref=None, weights=None, low=0.2, high=0.2, kl_coef=0.0, ent_coef=0.0,
                mean=True, scale=1.0):
    """(stats, logp, dlogits, a, h): a = dL/dlogp and h = dL/dH of every row"""
    w = np.ones(len(targets)) if weights is None else np.asarray(weights, np.float64)
    on = (targets >= 0) & (w != 0)
    stats, logp, grad = np.zeros(4), np.zeros(len(targets)), np.zeros(np.shape(z))
    a, h = np.zeros(len(targets)), np.zeros(len(targets))
    if not on.any():
        return stats, logp, grad, a, h
    pick = lambda v: None if v is None else np.asarray(v, np.float64)[on]  # noqa: E731
    w = w[on] / (w[on].sum() if mean else 1.0)
    lp, _, ent, _, _ = token_stats(z[on], targets[on], scale)
    loss, kl, clipped, da = policy_rows(lp, ent, pick(old), pick(adv), pick(ref), low, high, kl_coef, ent_coef)
    stats[:] = [(w * x).sum() for x in (loss, kl, clipped, ent)]
    logp[on], a[on], h[on] = lp, w * da, -ent_coef * w
    grad[on] = token_gradient(z[on], targets[on], a[on], h[on], scale)
    return stats, logp, grad, a, h


def pair_loss(kind, beta, d):
    """(l(d), l'(d))"""
    if kind == "sigmoid":
        return np.logaddexp(0.0, -beta * d), -beta / (1 + np.exp(beta * d))
    if kind == "squared":
        return (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta)
    return np.maximum(0.0, 1 - beta * d), np.where(beta * d < 1, -beta, 0.0)


def preference_loss(z, targets, offsets, ref=None, kind="sigmoid", beta=0.1, smoothing=0.0, margin=0.0, average=False,
                    scale=1.0):
    """(loss, margins, logp, dlogits, a)"""
    pairs = len(offsets) // 2
    logp = token_stats(z, targets, scale)[0]
    on = targets >= 0
    ratio = np.where(on, logp - (0.0 if ref is None else ref), 0.0)
    score, share = np.zeros(2 * pairs), np.ones(2 * pairs)
    for s in range(2 * pairs):
        rows = slice(offsets[s], offsets[s + 1])
        if average:
            share[s] = 1.0 / max(1, int(on[rows].sum()))
        score[s] = ratio[rows].sum() * share[s]
    gap = score[:pairs] - score[pairs:] - margin
    loss, slope = pair_loss(kind, beta, gap)
    other, back = pair_loss(kind, beta, -gap)
    loss, slope = (1 - smoothing) * loss + smoothing * other, (1 - smoothing) * slope - smoothing * back
    a = np.zeros(len(targets))
    for s in range(2 * pairs):
        sign = 1.0 if s < pairs else -1.0
        a[offsets[s]:offsets[s + 1]] = sign * slope[s % pairs] / pairs * share[s]
    a = np.where(on, a, 0.0)
    return loss.mean(), beta * gap, np.where(on, logp, 0.0), token_gradient(z, targets, a, None, scale), a


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
BLOCK = 256


def adamw(w, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, factor=1.0):
    """(w, m, v) after the step; factor: grad_scale times the clipping"""
    g = factor * g
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return w - lr * (weight_decay * w + mh / (np.sqrt(vh) + eps)), m, v


def scatter(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def words(seed, step, tensor, n):
    """The 32 random bits of each of a tensor's n elements."""
    key = scatter(scatter((seed & 0xFFFFFFFF) ^ int(scatter(step))) ^ np.uint64(seed >> 32 & 0xFFFFFFFF))
    at = np.arange(n, dtype=np.uint64)
    base = scatter(scatter(key + np.uint64(tensor)) + at // np.uint64(BLOCK))
    return scatter(base + (at % np.uint64(BLOCK)) * np.uint64(0x9E3779B9))


def _blocks(x, fill):
    n = len(x)
    out = np.full(-(-n // BLOCK) * BLOCK, fill, np.float64)
    out[:n] = x
    return out.reshape(-1, BLOCK)


def e4m3_step(x):
    """Distance of e4m3 values around |x| (at most 448)."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)


def pack(m, v, word):
    """8-bit form as values: (m / scale, scale, code of v, low, gap, and how far the random part of a step is
    from deciding otherwise, for m and v, in steps)"""
    n = len(m)
    mb, vb = _blocks(m, 0.0), _blocks(v, 0.0)
    scale = np.abs(mb).max(1) / 448
    x = (mb / np.where(scale > 0, scale, 1.0)[:, None]).reshape(-1)[:n]
    part = np.abs(x) / e4m3_step(x)
    r = (word & np.uint64(0xFFFF)).astype(np.float64) / 65536
    mq = np.sign(x) * np.floor(part + r) * e4m3_step(x)
    near_m = np.abs(part + r - np.round(part + r))
    with np.errstate(divide="ignore"):
        lg = np.where(vb > 0, np.log2(np.where(vb > 0, vb, 1.0)), np.nan)
    some = (vb > 0).any(1)
    top = np.where(some, np.nanmax(np.where(np.isnan(lg), -1e9, lg), axis=1), 0.0)
    low = np.where(some, np.maximum(np.nanmin(np.where(np.isnan(lg), 1e9, lg), axis=1), top - 24), 0.0)
    gap = (top - low) / 254
    y = np.where(gap[:, None] > 0, (lg - low[:, None]) / np.where(gap > 0, gap, 1.0)[:, None], 0.0)
    y = np.clip(np.nan_to_num(y), 0, 254).reshape(-1)[:n]
    f = y - np.floor(y)
    f = f - 0.5 * math.log(2) * np.repeat(gap, BLOCK)[:n] * f * (1 - f)
    r = (word >> np.uint64(16)).astype(np.float64) / 65536
    code = np.where(np.asarray(v) > 0, 1 + np.floor(y) + (r < f), 0)
    return mq, scale, code, low, gap, near_m, np.minimum(np.abs(r - f), np.abs(y - np.round(y)) + 1.0 * (y == 0))


def unpack(mq, scale, code, low, gap):
    n = len(mq)
    rep = lambda x: np.repeat(x, BLOCK)[:n]  # noqa: E731
    return mq * rep(scale), np.where(code > 0, np.exp2(rep(low) + (code - 1) * rep(gap)), 0.0)
