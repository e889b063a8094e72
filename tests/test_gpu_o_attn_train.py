"""Attention with row statistics and its backward pass (fo_attn_forward, fo_attn_backward) against
the fp64 oracle.

Tolerances, element by element.  E is the relative error of a softmax weight: its exponent is a
score in fp32 (products of head_dim bf16 pairs and a few more operations: (head_dim + 16) 2^-24 of
the largest magnitude sum inside a score), the exponential itself 2^-21.
  O:  a weight rounded to bf16 (2^-8) and E, relative to sum p |v|; the output's own 2^-8.
  LSE: fp32: the exponents' error, and 2^-22 of the value and of 1.
  dV: as O with sum p |dO|.  dQ, dK: dS rounded to bf16, its dP and delta in fp32
      (head_dim + 16 roundings of their magnitude sums), relative to scale sum mag(dS) |K|.
A gradient's rounding of dS is relative to |dS| <= mag(dS); delta is the exact one (the oracle's O before its
rounding), which the kernel corrects its delta to or, where it is near enough, does not: off by at most the rounding of
O, 2^-8 sum |dO O|, whose product with P is at most 2^-8 mag(dS) again."""
import numpy as np
import pytest
import torch

import fo_workloads as wl
from helpers import f64, guarded, to_bits
from oracle import bf16, training as tr

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a bf16 step, relative


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _round(x):
    return bf16.to_f64(bf16.from_f64(x))


def _within(got, want, tol, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(),
                           float(np.abs(got - want)[bad].max()), float(np.broadcast_to(tol, bad.shape)[bad].max()))


def _weight_error(d, ms):
    return 2 * (d + 16) * 2.0 ** -24 * ms + 2.0 ** -21


class Problem:
    """P ranks of packed or single sequences; Q, K, V as columns of one matrix where they have as many rows.
    Rows outside the sequences hold NaN."""

    def __init__(self, P, heads, kv_heads, d, seqs, causal, seed, front=0, behind=0, std=1.0, packed=None, scale=None):
        self.P, self.h, self.kv, self.d, self.causal, self.seqs, self.scale = P, heads, kv_heads, d, causal, seqs, scale
        self.packed = len(seqs) > 1 or front > 0 or behind > 0 if packed is None else packed
        self.q_off = front + np.cumsum([0] + [a for a, _ in seqs])
        self.k_off = front + np.cumsum([0] + [b for _, b in seqs])
        self.mq, self.mk = int(self.q_off[-1]) + behind, int(self.k_off[-1]) + behind
        g = torch.Generator().manual_seed(seed)
        rnd = lambda rows, cols: (torch.randn((rows, cols), generator=g) * std).to(torch.bfloat16)  # noqa: E731
        self.same = self.mq == self.mk and all(a == b for a, b in seqs)
        self.q, self.k, self.v, self.do = [], [], [], []
        for _ in range(P):
            if self.same:
                m = rnd(self.mq, (heads + 2 * kv_heads) * d)
                self._nan(m, self.q_off)
                m = m.cuda()
                q, k, v = m.split([heads * d, kv_heads * d, kv_heads * d], 1)
            else:
                q, k, v = rnd(self.mq, heads * d), rnd(self.mk, kv_heads * d), rnd(self.mk, kv_heads * d)
                for x, off in ((q, self.q_off), (k, self.k_off), (v, self.k_off)):
                    self._nan(x, off)
                q, k, v = q.cuda(), k.cuda(), v.cuda()
            do = rnd(self.mq, heads * d)
            self._nan(do, self.q_off)
            for lst, x in ((self.q, q), (self.k, k), (self.v, v), (self.do, do.cuda())):
                lst.append(x)
        self.kw = dict(heads=heads, kv_heads=kv_heads, head_dim=d, causal=causal, scale=scale)
        if self.packed:
            dev = lambda o: torch.tensor(o, dtype=torch.int32, device="cuda")  # noqa: E731
            self.kw["q_offsets"] = dev(self.q_off)
            if not self.same:
                self.kw["k_offsets"] = dev(self.k_off)

    @staticmethod
    def _nan(x, off):
        x[:int(off[0])] = float("nan")
        x[int(off[-1]):] = float("nan")

    def parts(self, p):
        """(rank's q, k, v, dO of each sequence in fp64, row ranges)"""
        for (a, b), (c, e) in zip(zip(self.q_off, self.q_off[1:]), zip(self.k_off, self.k_off[1:])):
            cut = lambda t, lo, hi, n: f64(to_bits(t[int(lo):int(hi)].contiguous())).reshape(int(hi - lo), n, self.d)  # noqa: E731
            yield (cut(self.q[p], a, b, self.h), cut(self.k[p], c, e, self.kv), cut(self.v[p], c, e, self.kv),
                   cut(self.do[p], a, b, self.h), slice(int(a), int(b)), slice(int(c), int(e)))

    def outputs(self):
        rows = lambda m, n: [guarded((m, n * self.d), torch.bfloat16) for _ in range(self.P)]  # noqa: E731
        return (rows(self.mq, self.h), [guarded((self.h, self.mq), torch.float32) for _ in range(self.P)],
                rows(self.mq, self.h), rows(self.mk, self.kv), rows(self.mk, self.kv))


def _np(t, n, d):
    return t.double().cpu().numpy().reshape(t.shape[0], n, d)


def _check(ctx, pb, **kw):
    O, LSE, dQ, dK, dV = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw, **kw)
    torch.cuda.synchronize()
    ctx.poll()
    d = pb.d
    ref = []
    for p in range(pb.P):
        got_o, got_l = _np(O[p], pb.h, d), LSE[p].double().cpu().numpy()
        inside = np.zeros(pb.mq, bool)
        for q, k, v, do, qs, ks in pb.parts(p):
            inside[qs] = True
            o, lse, w = tr.attn_forward(q, k, v, pb.causal, pb.scale)
            scale = pb.scale or d ** -0.5
            ms = 0.0
            if q.size and k.size:
                ms = max(scale * (np.abs(q[:, a]) @ np.abs(k[:, a // (pb.h // pb.kv)]).T).max() for a in range(pb.h))
            e = _weight_error(d, ms)
            mag = np.stack([w[a] @ np.abs(v[:, a // (pb.h // pb.kv)]) for a in range(pb.h)], 1)
            _within(got_o[qs], o, (HALF + e) * mag + HALF * np.abs(o), f"O rank {p} rows {qs}")
            empty = np.isneginf(lse)
            assert np.array_equal(np.isneginf(got_l[:, qs]), empty)
            assert (got_o[qs].transpose(1, 0, 2)[empty] == 0).all()
            with np.errstate(invalid="ignore"):
                _within(np.where(empty, 0, got_l[:, qs]), np.where(empty, 0, lse),
                        e + 2.0 ** -22 * (np.where(empty, 0, np.abs(lse)) + 1), f"LSE rank {p} rows {qs}")
            ref.append((p, q, k, v, do, qs, ks, o, lse.astype(np.float32).astype(np.float64)))
        # rows outside the sequences are left alone
        assert torch.isnan(O[p][torch.from_numpy(~inside).cuda()]).all()
        assert torch.isnan(LSE[p][:, torch.from_numpy(~inside).cuda()]).all()
    # the backward pass from the oracle's O and LSE
    for p, q, k, v, do, qs, ks, o, lse in ref:
        O[p][qs] = torch.from_numpy(_round(o).reshape(o.shape[0], pb.h * d)).to(torch.bfloat16).cuda()
        LSE[p][:, qs] = torch.from_numpy(lse).float().cuda()
    ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw, **kw)
    torch.cuda.synchronize()
    ctx.poll()
    done_q, done_k = [np.zeros(pb.mq, bool) for _ in range(pb.P)], [np.zeros(pb.mk, bool) for _ in range(pb.P)]
    for p, q, k, v, do, qs, ks, o, lse in ref:
        done_q[p][qs] = True
        done_k[p][ks] = True
        rq, rk, rv, mq, mk, mv, ms = tr.attn_backward(q, k, v, o, lse, do, pb.causal, pb.scale)
        e = _weight_error(d, ms) + 2 * (d + 16) * 2.0 ** -24
        for name, got, want, mag, n in (("dQ", _np(dQ[p], pb.h, d)[qs], rq, mq, 2), ("dK", _np(dK[p], pb.kv, d)[ks], rk, mk, 2),
                                     ("dV", _np(dV[p], pb.kv, d)[ks], rv, mv, 1)):
            _within(got, want, (n * HALF + e) * mag + HALF * np.abs(want), f"{name} rank {p} rows {qs} {ks}")
    for p in range(pb.P):
        assert torch.isnan(dQ[p][torch.from_numpy(~done_q[p]).cuda()]).all()
        assert torch.isnan(dK[p][torch.from_numpy(~done_k[p]).cuda()]).all()
        assert torch.isnan(dV[p][torch.from_numpy(~done_k[p]).cuda()]).all()
    return O, LSE, dQ, dK, dV


# P, heads, kv_heads, head_dim, (queries, keys), causal
SINGLE = [
    (1, 1, 1, 128, (1, 1), True), (1, 1, 1, 64, (1, 1), False), (1, 2, 2, 128, (128, 128), True),
    (2, 2, 1, 128, (129, 129), True), (1, 3, 3, 64, (127, 127), True), (1, 4, 2, 128, (256, 256), True),
    (1, 2, 2, 64, (257, 257), True), (1, 5, 1, 128, (333, 333), True), (1, 2, 1, 128, (300, 300), False),
    (1, 2, 2, 128, (1, 300), True), (1, 2, 2, 128, (130, 513), True), (1, 2, 1, 64, (300, 129), True),
    (1, 1, 1, 128, (513, 1), True), (1, 1, 1, 64, (400, 2), False), (2, 2, 2, 128, (200, 77), False),
    (1, 1, 1, 128, (1000, 1000), True), (1, 8, 8, 64, (384, 640), True),
]


@pytest.mark.parametrize("case", SINGLE, ids=str)
def test_single_sequences(ctx, case):
    P, h, kv, d, (lq, lk), causal = case
    _check(ctx, Problem(P, h, kv, d, [(lq, lk)], causal, 17 * lq + lk))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_sequences(ctx, d, causal):
    lens = [1, 0, 128, 63, 130, 300, 0, 5, 256]
    _check(ctx, Problem(2, 4, 2, d, [(n, n) for n in lens], causal, 5 + d, front=3, behind=70))


@pytest.mark.parametrize("d", [64, 128])
def test_packed_sequences_with_their_own_key_lengths(ctx, d):
    # more keys than queries, fewer (queries without keys), none on either side
    seqs = [(5, 200), (140, 20), (0, 33), (70, 0), (256, 257), (1, 129)]
    _check(ctx, Problem(1, 2, 1, d, seqs, True, 77 + d, front=1, behind=9))
    _check(ctx, Problem(1, 2, 1, d, seqs, False, 78 + d))


@pytest.mark.parametrize("d", [64, 128])
def test_walks_cut_into_parts(ctx, d):
    """Few key blocks under many query heads (dK, dV summed from parts), few queries under many keys (dQ likewise),
    packed and with rows outside the sequences."""
    _check(ctx, Problem(1, 16, 1, d, [(390, 390)], True, 51 + d))
    _check(ctx, Problem(1, 1, 1, d, [(70, 2200)], True, 52 + d))
    _check(ctx, Problem(1, 8, 1, d, [(260, 260), (0, 0), (300, 300)], True, 53 + d, front=2, behind=30))
    _check(ctx, Problem(1, 2, 2, d, [(1500, 130)], False, 54 + d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1, 2, 3, 4, 5, 6, 7, 8] * 12, [3] * 100, [20] * 20, [130]])
def test_gradients_of_rows_with_few_keys(ctx, d, lens):
    """Where a row has few keys dP and delta cancel, and a delta from the rounded O would be most of the error.
    2-norms: dS and the output are each rounded to bf16, independently and by at most 2^-8 (root mean square at most
    2^-8 / sqrt(3)), and delta may be off by 2^-11 of the row sums."""
    pb = Problem(1, 2, 1, d, [(n, n) for n in lens], True, 61 + len(lens))
    O, LSE, dQ, dK, dV = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
    ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)
    want = [np.zeros((pb.mq, n, d)) for n in (2, 1, 1)]
    for q, k, v, do, qs, ks in pb.parts(0):
        o, lse, _ = tr.attn_forward(q, k, v)
        for w, g, rows in zip(want, tr.attn_backward(q, k, v, o, lse, do)[:3], (qs, ks, ks)):
            w[rows] = g
    for name, got, w in zip(("dQ", "dK", "dV"), (dQ, dK, dV), want):
        err = np.linalg.norm(_np(got[0], w.shape[1], d) - w) / np.linalg.norm(w)
        assert err <= HALF * (2 / 3) ** 0.5 + 2.0 ** -11, (name, err)


def test_more_sequences_than_one_pass_of_the_table_kernel(ctx):
    rng = np.random.default_rng(4)
    _check(ctx, Problem(1, 1, 1, 64, [(int(n), int(n)) for n in rng.integers(0, 4, 1500)], True, 9))


def test_scale_and_large_scores(ctx):
    # scores of magnitude ~40: the running maximum moves between blocks
    _check(ctx, Problem(1, 2, 2, 128, [(500, 500)], True, 31, std=2.0))
    _check(ctx, Problem(1, 2, 2, 64, [(260, 260)], False, 32, scale=0.5))


def test_growing_maximum(ctx):
    # keys ordered so that every block raises the row maximum, and a last key that dominates
    pb = Problem(1, 1, 1, 128, [(384, 384)], False, 33)
    ramp = torch.linspace(0.0, 6.0, 384, device="cuda")[:, None]
    pb.k[0].copy_((pb.q[0][:1].float() * ramp / 11.3).to(torch.bfloat16))
    pb.q[0].copy_(pb.q[0][:1].expand(384, 128).clone())
    _check(ctx, pb)


def test_constant_values_come_through(ctx):
    pb = Problem(1, 2, 1, 128, [(200, 200)], True, 34)
    pb.v[0].fill_(1.5)
    O, LSE, *_ = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
    # sum of bf16-rounded weights over the sum of the unrounded ones: half a step, and the output's own
    assert (O[0].float() - 1.5).abs().max() <= 1.5 * 2 * HALF


@pytest.mark.parametrize("n,d", [(700, 128), (90, 128), (700, 64), (90, 64)])
def test_a_nan_stays_in_its_row(ctx, n, d):
    """A NaN query turns its row's output and statistic into NaN, in its head alone, and nothing else."""
    pb = Problem(1, 2, 1, d, [(n, n)], True, 37)
    (O, LSE, *_), (O2, LSE2, *_) = pb.outputs(), pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
    pb.q[0][50, d + 3] = float("nan")
    ctx.attn_forward(pb.q, pb.k, pb.v, O2, LSE2, **pb.kw)
    assert torch.isnan(O2[0][50, d:]).all() and torch.isnan(LSE2[0][1, 50])
    O2[0][50, d:], LSE2[0][1, 50] = O[0][50, d:], LSE[0][1, 50]
    assert torch.equal(O2[0], O[0]) and torch.equal(LSE2[0], LSE[0])


def test_bad_offsets_are_reported(ctx):
    import overlapped_tensor_gemm_gb300 as fo
    pb = Problem(1, 2, 2, 64, [(40, 40), (30, 30)], True, 35, behind=1)
    for bad in ([0, 40, 30], [-1, 40, 70], [0, 40, 72], [0, 80, 70]):
        O, LSE, dQ, dK, dV = pb.outputs()
        kw = dict(pb.kw, q_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **kw)
        torch.cuda.synchronize()
        with pytest.raises(fo.FoError) as e:
            ctx.poll()
        assert e.value.status == fo.FO_ERR_RANGE and "offsets" in str(e.value)
        ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **kw)
        torch.cuda.synchronize()
        with pytest.raises(fo.FoError):
            ctx.poll()
        for t in O + LSE + dQ + dK + dV:
            assert torch.isnan(t).all()
    _check(ctx, pb)


def test_same_bits_again_and_on_another_stream(ctx):
    pb = Problem(2, 4, 1, 128, [(700, 700)], True, 36)
    first = [[t.clone() for t in x] for x in _check(ctx, pb)]
    O, LSE, dQ, dK, dV = pb.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ctx.attn_backward(pb.q, pb.k, pb.v, first[0], first[1], pb.do, dQ, dK, dV, **pb.kw)
    side.synchronize()
    for a, b in zip(first[2:], (dQ, dK, dV)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_captured_and_replayed(ctx):
    pb = Problem(1, 4, 2, 128, [(300, 300), (90, 90)], True, 37)
    O, LSE, dQ, dK, dV = pb.outputs()

    def step():
        ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
        ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # other values and other boundaries at the same addresses; a larger call in between grows the workspace
    pb.q[0].copy_(torch.randn(pb.q[0].shape, device="cuda").to(torch.bfloat16))
    pb.kw["q_offsets"].copy_(torch.tensor([0, 111, 390], dtype=torch.int32))
    big = Problem(4, 8, 8, 64, [(600, 600), (700, 700)], True, 38)
    bo = big.outputs()
    ctx.attn_forward(big.q, big.k, big.v, bo[0], bo[1], **big.kw)
    ctx.attn_backward(big.q, big.k, big.v, bo[0], bo[1], big.do, *bo[2:], **big.kw)
    graph.replay()
    torch.cuda.synchronize()
    ctx.poll()
    got = [t[0].clone() for t in (O, LSE, dQ, dK, dV)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (O, LSE, dQ, dK, dV)):
        assert torch.equal(a, b[0])


@pytest.mark.parametrize("lq,lk", [(0, 40), (40, 0), (0, 0)])
@pytest.mark.parametrize("packed", [False, True])
def test_no_queries_or_no_keys(ctx, lq, lk, packed):
    pb = Problem(1, 2, 1, 64, [(lq, lk)], True, 39, packed=packed)
    O, LSE, dQ, dK, dV = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
    ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)
    torch.cuda.synchronize()
    ctx.poll()
    assert (O[0] == 0).all() and torch.isneginf(LSE[0]).all()
    assert (dQ[0] == 0).all() and (dK[0] == 0).all() and (dV[0] == 0).all()


def test_a_capture_before_the_first_call_is_refused():
    """Growing a workspace is not something a stream capture can hold: the call says so and enqueues nothing."""
    import overlapped_tensor_gemm_gb300 as fo
    pb = Problem(1, 2, 2, 64, [(50, 50)], True, 40)
    O, LSE, dQ, dK, dV = pb.outputs()
    with fo.Context(0) as c:
        c.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)  # one sequence: needs no workspace
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(fo.FoError) as e:
                c.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)
            c.attn_forward(pb.q, pb.k, pb.v, O, LSE, **pb.kw)
        assert e.value.status == fo.FO_ERR_UNSUPPORTED and "capture" in str(e.value)
        graph.replay()
        c.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, **pb.kw)
        torch.cuda.synchronize()
        c.poll()
    assert torch.isfinite(dQ[0].float()).all()


def test_a_short_timeout_ends_the_call_with_an_error(ctx):
    """Waits are bounded: with a limit of one microsecond the kernels give up (or, on a lucky run, finish), the poll
    says so, and the context computes correctly afterwards."""
    import overlapped_tensor_gemm_gb300 as fo
    pb = Problem(1, 2, 1, 128, [(1500, 1500)], True, 42)
    O, LSE, dQ, dK, dV = pb.outputs()
    ctx.attn_forward(pb.q, pb.k, pb.v, O, LSE, timeout_us=1, **pb.kw)
    ctx.attn_backward(pb.q, pb.k, pb.v, O, LSE, pb.do, dQ, dK, dV, timeout_us=1, **pb.kw)
    torch.cuda.synchronize()
    try:
        ctx.poll()
    except fo.FoError as e:
        assert e.status == fo.FO_ERR_TIMEOUT
    _check(ctx, Problem(1, 2, 1, 128, [(300, 300)], True, 43))


def test_a_block_of_a_training_step(ctx):
    """The operators together: norm, QKV projection, rotary positions, attention, output projection, gated residual;
    and back.  Against fp32 torch autograd of the same chain on the rounded weights: rel-L2 of each gradient within
    the number of bf16 roundings on its way (at most 12 on the longest) times 2^-8."""
    import math

    import overlapped_tensor_gemm_gb300 as fo
    from oracle import training as tr_
    P, m, Hd, h, kv, d = 1, 256, 512, 4, 2, 64
    g = torch.Generator().manual_seed(40)
    rnd = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g) * std + mean).to(torch.bfloat16).cuda()  # noqa: E731
    R, w1, w2, w3, gate = rnd(m, Hd), rnd(Hd, std=.1, mean=1.), rnd(Hd, std=.1, mean=1.), rnd(Hd, std=.1, mean=1.), rnd(Hd, std=.2, mean=.5)
    nq = (h + 2 * kv) * d
    Wqkv, Wo = rnd(nq, Hd, std=Hd ** -0.5), rnd(Hd, h * d, std=(h * d) ** -0.5)
    dX2, dR2 = rnd(m, Hd), rnd(m, Hd)
    table = fo.RopeTable(d)
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    X, QKV, O, Y, RO, X2, LSE = new(m, Hd), new(m, nq), new(m, h * d), new(m, Hd), new(m, Hd), new(m, Hd), torch.empty((h, m), device="cuda")
    ctx.norm_residual([R], None, None, [X], w_pre=w1)
    ctx.ag_gemm([X], [Wqkv], [QKV])
    qk = QKV[:, :(h + kv) * d]
    ctx.rope([qk], [qk], table)
    cols = lambda t: ([t[:, :h * d]], [t[:, h * d:(h + kv) * d]], [t[:, (h + kv) * d:]])  # noqa: E731
    Q, K, V = cols(QKV)
    how = dict(heads=h, kv_heads=kv, head_dim=d)
    ctx.attn_forward(Q, K, V, [O], [LSE], **how)
    ctx.gemm_rs([O], [Wo], [Y])
    ctx.norm_residual([R], [Y], [RO], [X2], w_post=w2, gate=gate, w_pre=w3)
    # back
    dR, dY, dO, dWo, dQKV, dX, dWqkv = new(m, Hd), new(m, Hd), new(m, h * d), new(Hd, h * d), new(m, nq), new(m, Hd), new(nq, Hd)
    vec = lambda: torch.empty(Hd, device="cuda")  # noqa: E731
    dw1, dw2, dw3, dgate, dR0 = vec(), vec(), vec(), vec(), new(m, Hd)
    ctx.norm_residual_backward([RO], [Y], [dX2], [dR2], [dR], [dY], w_post=w2, gate=gate, w_pre=w3, dw_post=dw2,
                               dgate=dgate, dw_pre=dw3)
    ctx.row_linear_backward([O], [Wo], [dY], [dO], [dWo])
    dQ, dK, dV = cols(dQKV)
    ctx.attn_backward(Q, K, V, [O], [LSE], [dO], dQ, dK, dV, **how)
    dqk = dQKV[:, :(h + kv) * d]
    ctx.rope_backward([dqk], [dqk], table)
    ctx.col_linear_backward([X], [Wqkv], [dQKV], [dX], [dWqkv])
    ctx.norm_residual_backward([R], None, [dX], [dR], [dR0], None, w_pre=w1, dw_pre=dw1)
    torch.cuda.synchronize()
    ctx.poll()

    leaf = {k: t.double().requires_grad_() for k, t in dict(R=R, w1=w1, w2=w2, w3=w3, gate=gate, Wqkv=Wqkv, Wo=Wo).items()}
    norm = lambda t, w: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    freq, _ = tr_.rope_frequencies(d, 10000.0)
    ang = torch.arange(m, device="cuda").double()[:, None] * torch.tensor(freq, device="cuda")[None]

    def turn(t):
        a, b = t[..., :d // 2], t[..., d // 2:]
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    qkv = norm(leaf["R"], leaf["w1"]) @ leaf["Wqkv"].T
    q, k, v = (t.reshape(m, -1, d) for t in qkv.split([h * d, kv * d, kv * d], 1))
    q, k = turn(q), turn(k)
    k, v = (t.repeat_interleave(h // kv, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
    s = s.masked_fill(torch.ones((m, m), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(m, h * d)
    ro = leaf["R"] + leaf["gate"] * norm(o @ leaf["Wo"].T, leaf["w2"])
    x2 = norm(ro, leaf["w3"])
    want = torch.autograd.grad((x2 * dX2.double()).sum() + (ro * dR2.double()).sum(), list(leaf.values()))
    got = dict(R=dR0, w1=dw1, w2=dw2, w3=dw3, gate=dgate, Wqkv=dWqkv, Wo=dWo)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(X2, x2.detach()) <= 8 * HALF
    for (name, ref) in zip(leaf, want):
        assert rel(got[name], ref) <= 12 * HALF, name
