"""Attention over thousands of keys, forward and backward, against the definitions in fp64 (on the GPU, one head at a
time), for spread attention and for peaked (scores of standard deviation 8: running maxima that move late, blocks whose
delta is corrected by a second walk).

Tolerances, element by element, as for short sequences (a bf16 rounding is at most 2^-8; E is a weight's error: its
score is an fp32 sum of d products, its exponential 2^-21), and for each product over n rows n 2^-24 of its magnitude
sum, which is what n fp32 additions can lose."""
import math

import pytest
import torch

from helpers import guarded

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


def _within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), bad.nonzero()[:3].tolist())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk,causal", [(8192, 8192, True), (300, 9001, True), (5000, 4097, False)])
@pytest.mark.parametrize("std", [1.0, 8 ** 0.5])
def test_against_fp64(d, lq, lk, causal, std):
    import overlapped_tensor_gemm_gb300 as fo
    h, kv = 2, 1
    g = torch.Generator(device="cuda").manual_seed(lq + d)
    rnd = lambda rows, heads, s: (torch.randn((rows, heads * d), generator=g, device="cuda") * s).to(torch.bfloat16)  # noqa: E731
    q, k, v, do = rnd(lq, h, std), rnd(lk, kv, std), rnd(lk, kv, 1.0), rnd(lq, h, 1.0)
    O, LSE = guarded((lq, h * d), torch.bfloat16), guarded((h, lq), torch.float32)
    dQ, dK, dV = (guarded((n, c * d), torch.bfloat16) for n, c in ((lq, h), (lk, kv), (lk, kv)))
    kw = dict(heads=h, kv_heads=kv, head_dim=d, causal=causal)
    scale = d ** -0.5
    with fo.Context(0) as c:
        c.attn_forward([q], [k], [v], [O], [LSE], **kw)
        torch.cuda.synchronize()
        c.poll()
        got_o, got_lse = O.clone(), LSE.clone()
        K, V = k.double(), v.double()
        hidden = ~(torch.arange(lk, device="cuda")[None] <= torch.arange(lq, device="cuda")[:, None] + lk - lq) if causal else None
        want, more = {}, [torch.zeros(lk, d, dtype=torch.float64, device="cuda") for _ in range(4)]  # dK, dV, their magnitudes
        for a in range(h):
            cols = slice(a * d, (a + 1) * d)
            Q, D = q[:, cols].double(), do[:, cols].double()
            S = scale * (Q @ K.T)
            ms = float((scale * (Q.abs() @ K.abs().T)).max())
            if causal:
                S.masked_fill_(hidden, -math.inf)
            lse = torch.logsumexp(S, 1)
            w = torch.exp(S - lse[:, None])
            o = w @ V
            e = 2 * (d + 16) * 2.0 ** -24 * ms + 2.0 ** -21
            _within(got_o[:, cols], o, (HALF + e + lk * 2.0 ** -24) * (w @ V.abs()) + HALF * o.abs(), f"O {a}")
            _within(got_lse[a], lse, e + lk * 2.0 ** -24 + 2.0 ** -22 * (lse.abs() + 1), f"LSE {a}")
            # the backward pass from the reference's own O and LSE
            O[:, cols], LSE[a] = o.to(torch.bfloat16), lse.float()
            w = torch.exp(S - LSE[a].double()[:, None])
            delta = (D * o).sum(1, keepdim=True)
            ds = w * (D @ V.T - delta)
            mag = w * (D.abs() @ V.abs().T + (D * o).abs().sum(1, keepdim=True))
            e += 2 * (d + 16) * 2.0 ** -24
            want[a] = scale * ds @ K, (2 * HALF + e + lk * 2.0 ** -24) * scale * (mag @ K.abs())
            for t, x in zip(more, (scale * ds.T @ Q, w.T @ D, scale * mag.T @ Q.abs(), w.T @ D.abs())):
                t += x
            del S, w, ds, mag
        c.attn_backward([q], [k], [v], [O], [LSE], [do], [dQ], [dK], [dV], **kw)
        torch.cuda.synchronize()
        c.poll()
    for a in range(h):
        _within(dQ[:, a * d:(a + 1) * d], want[a][0], want[a][1] + HALF * want[a][0].abs(), f"dQ {a}")
    rows = h * lq * 2.0 ** -24
    _within(dK, more[0], (2 * HALF + e + rows) * more[2] + HALF * more[0].abs(), "dK")
    _within(dV, more[1], (HALF + e + rows) * more[3] + HALF * more[1].abs(), "dV")
