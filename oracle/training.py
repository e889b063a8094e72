"""Slow fp64 definitions of the training operators around the projections: attention with row
statistics and its backward pass, norms before and after a block with gate and residual, rotary
positions.  Every function also returns, where a test needs it, the sum of magnitudes that an
error bound of the operation is relative to."""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------------------
# attention: Q [Lq, H, D], K, V [Lk, Hkv, D]
# ---------------------------------------------------------------------------
def attn_mask(lq: int, lk: int, causal: bool) -> np.ndarray:
    i, j = np.arange(lq)[:, None], np.arange(lk)[None, :]
    return j <= i + (lk - lq) if causal else np.ones((lq, lk), bool)


def attn_forward(q, k, v, causal=True, scale=None):
    """(O [Lq, H, D], LSE [H, Lq], P [H, Lq, Lk])"""
    lq, h, d = q.shape
    lk, hkv, _ = k.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    keep = attn_mask(lq, lk, causal)
    o, lse, p = np.zeros((lq, h, d)), np.full((h, lq), -np.inf), np.zeros((h, lq, lk))
    for a in range(h):
        b = a // (h // hkv)
        s = scale * (q[:, a] @ k[:, b].T)
        for i in range(lq):
            js = np.nonzero(keep[i])[0]
            if js.size == 0:
                continue
            top = s[i, js].max()
            e = np.exp(s[i, js] - top)
            lse[a, i] = top + math.log(e.sum())
            p[a, i, js] = e / e.sum()
        o[:, a] = p[a] @ v[:, b]
    return o, lse, p


def attn_backward(q, k, v, o, lse, do, causal=True, scale=None):
    """Gradients from the given O and LSE; and the magnitudes of dQ, dK, dV's sums:
    (dQ, dK, dV, mQ, mK, mV, mS) with mS the largest magnitude sum inside a score."""
    lq, h, d = q.shape
    lk, hkv, _ = k.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    keep = attn_mask(lq, lk, causal)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    mq, mk, mv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    ms = 0.0
    for a in range(h):
        b = a // (h // hkv)
        s = scale * (q[:, a] @ k[:, b].T)
        if s.size:
            ms = max(ms, scale * (np.abs(q[:, a]) @ np.abs(k[:, b]).T).max())
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(keep, np.exp(s - lse[a][:, None]), 0.0)
        delta = (do[:, a] * o[:, a]).sum(-1, keepdims=True)
        ds = p * (do[:, a] @ v[:, b].T - delta)
        mds = p * (np.abs(do[:, a]) @ np.abs(v[:, b]).T + np.abs(do[:, a] * o[:, a]).sum(-1, keepdims=True))
        dq[:, a] = scale * ds @ k[:, b]
        dk[:, b] += scale * ds.T @ q[:, a]
        dv[:, b] += p.T @ do[:, a]
        mq[:, a] = scale * mds @ np.abs(k[:, b])
        mk[:, b] += scale * mds.T @ np.abs(q[:, a])
        mv[:, b] += p.T @ np.abs(do[:, a])
    return dq, dk, dv, mq, mk, mv, ms


# ---------------------------------------------------------------------------
# norms with gate and residual: [tokens, H]
# ---------------------------------------------------------------------------
def _rms(v, eps):
    return np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def norm_residual(r, y, w_post=None, gate=None, w_pre=None, alpha=1.0, eps=1e-6):
    """(R_out, X, magnitude of R_out's sum)"""
    if y is None:
        r_out, mag = r, np.abs(r)
    else:
        z = y if w_post is None else y / _rms(y, eps) * w_post
        gz = z if gate is None else gate * z
        r_out, mag = alpha * r + gz, np.abs(alpha * r) + np.abs(gz)
    x = None if w_pre is None else r_out / _rms(r_out, eps) * w_pre
    return r_out, x, mag


def norm_residual_backward(r_out, y, dx, dr_out, w_post=None, gate=None, w_pre=None, alpha=1.0, eps=1e-6):
    """Gradients {r, y, w_post, gate, w_pre} and, under the same names, the magnitudes of their
    sums (per-token gates: [tokens, H])."""
    t = np.zeros_like(r_out) if dr_out is None else dr_out
    mt = np.abs(t)
    g, mag = {}, {}
    if w_pre is not None:
        rr = _rms(r_out, eps)
        n, dn = r_out / rr, dx * w_pre
        g["w_pre"], mag["w_pre"] = (dx * n).sum(0), np.abs(dx * n).sum(0)
        t = t + (dn - n * (dn * n).mean(-1, keepdims=True)) / rr
        mt = mt + (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(-1, keepdims=True)) / rr
    g["r"], mag["r"] = alpha * t, np.abs(alpha) * mt
    if y is None:
        return g, mag
    ry = _rms(y, eps) if w_post is not None else 1.0
    u = y / ry
    z = u if w_post is None else u * w_post
    if gate is not None:
        per_token = np.ndim(gate) == 2
        g["gate"] = t * z if per_token else (t * z).sum(0)
        mag["gate"] = mt * np.abs(z) if per_token else (mt * np.abs(z)).sum(0)
    dz = t if gate is None else t * gate
    mz = mt if gate is None else mt * np.abs(gate)
    if w_post is not None:
        g["w_post"], mag["w_post"] = (dz * u).sum(0), (mz * np.abs(u)).sum(0)
        du, mu = dz * w_post, mz * np.abs(w_post)
        dz = (du - u * (du * u).mean(-1, keepdims=True)) / ry
        mz = (mu + np.abs(u) * (mu * np.abs(u)).mean(-1, keepdims=True)) / ry
    g["y"], mag["y"] = dz, mz
    return g, mag


# ---------------------------------------------------------------------------
# rotary positions: X [tokens, heads, head_dim]
# ---------------------------------------------------------------------------
def rope_frequencies(rot_dim, base, scaling=None, factor=1.0, low=1.0, high=4.0, length=0):
    """(radians per position of each pair, amplitude); low and high in turns over `length`."""
    out, amplitude = [], 1.0
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling is None:
            keep = 1.0
        elif scaling == "linear":
            keep = 0.0
        elif scaling == "banded":
            keep = (length * f / (2 * math.pi) - low) / (high - low)
        else:
            amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
            first, last = (rot_dim * math.log(length / (2 * math.pi * b)) / (2 * math.log(base)) for b in (high, low))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rot_dim - 1)
            keep = 1.0 - (i - first) / max(last - first, 0.001)
        keep = min(max(keep, 0.0), 1.0)
        out.append(f / factor * (1 - keep) + f * keep)
    return np.array(out), amplitude


def rope(x, positions, freq, amplitude=1.0, interleaved=False, sign=1.0):
    rot = 2 * len(freq)
    angle = sign * np.asarray(positions, np.float64)[:, None] * freq[None, :]
    c, s = (amplitude * np.cos(angle))[:, None, :], (amplitude * np.sin(angle))[:, None, :]
    y = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y
