"""Losses from sharded logits (fo_token_logprobs and its backward, fo_policy_loss, fo_preference_loss)
against the fp64 oracle.

Tolerances, u = 2^-24.  A row's d = z - max z carries one rounding, its product with log2 e two, the
exponential 2^-22: a weight exp d is off by (3|d| + 4) u relative.  Sums of n columns add one rounding per
column that a thread sums and the joins of at most 2^15 threads' parts (15, each with a factor exp of a
difference of maxima): S = (n / 128 + 64 + 60 D) u with D the row's spread.  Hence logp and lse: S + a few
roundings of their own size; p: S + (3|d| + 4) u; the entropy: the same, times its terms.  A gradient is
rounded once to its type, and the loss's factors carry logp's error."""
import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import losses as ls

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
u = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


class Rows:
    """Logits of m rows on P ranks of `cols` columns each, padded with NaN; rows without a target hold NaN,
    rows with one a -infinity, the type's lowest value and a peak here and there."""

    def __init__(self, m, cols, dtype=BF, seed=0, masked=0.3, spread=2.0, special=True, temperature=1.0):
        rng = np.random.default_rng(seed)
        self.m, self.cols, self.P, self.dtype, self.scale = m, cols, len(cols), dtype, 1.0 / temperature
        vocab = self.vocab = sum(cols)
        self.y = rng.integers(0, vocab, m)
        z = rng.normal(size=(m, vocab)) * spread
        z[np.arange(m), self.y] += rng.uniform(0, 6, m)
        lowest = float(torch.finfo(dtype).min)
        if special and vocab > 2:
            for i in range(0, m, 3):
                z[i, rng.integers(0, vocab, 3)] = [-np.inf, lowest, -np.inf]
                z[i, self.y[i]] = rng.normal()
            if m > 4:
                z[1] += 300.0       # far from zero
                z[4, self.y[4]] += 60.0  # certain
        off = rng.random(m) < masked
        if m > 1:
            off[-1], off[0] = masked > 0, False
        self.y[off] = -1 - rng.integers(0, 3, off.sum())
        t = torch.from_numpy(z).to(dtype)
        t[torch.from_numpy(off)] = float("nan")
        self.z64 = t.double().numpy()
        self.logits = []
        at = 0
        for c in cols:
            per = 16 // t.element_size()
            base = torch.full((m, -(-c // per) * per + per), float("nan"), dtype=dtype, device="cuda")
            base[:, :c] = t[:, at:at + c].cuda()
            self.logits.append(base[:, :c])
            at += c
        self.targets = torch.from_numpy(self.y).int().cuda()
        self.on = self.y >= 0

    def outputs(self, dtype):
        return [guarded((self.m, c), dtype) for c in self.cols]

    def copies(self):
        """The logits again, with a pitch that the calls take."""
        out = [guarded((self.m, c), self.dtype) for c in self.cols]
        for a, b in zip(out, self.logits):
            a.copy_(b)
        return out

    def bounds(self, rows):
        """(S, d relative to the maximum) of the chosen rows"""
        z = self.z64[rows] * self.scale
        d = z - z.max(1, keepdims=True)
        near = np.where(d > -110, d, 0.0)  # columns below have weight 0 in fp32 and less than 2^-150 in truth
        return (self.vocab / 128 + 64 - 60 * near.min(1)) * u, near

    def joined(self, mats):
        return np.concatenate([t.double().cpu().numpy() for t in mats], 1)


def _vec(x):
    return torch.from_numpy(np.asarray(x, np.float64)).float().cuda()


def _within(got, ref, tol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got.size, np.abs(got - ref)[bad][:4], tol[bad][:4], ref[bad][:4])


def _check_gradient(r, got, dtype, a, h, err_a, err_h=0.0):
    """dlogits from a = dL/dlogp, h = dL/dH of every row; err_a, err_h: what they may be off"""
    got = r.joined(got)
    assert (got[~r.on] == 0).all()
    on = r.on
    if not on.any():
        return
    ref = ls.token_gradient(r.z64[on], r.y[on], a[on], h[on], r.scale)
    S, d = r.bounds(on)
    _, _, ent, p, lp = ls.token_stats(r.z64[on], r.y[on], r.scale)
    lp = np.where(p > 0, lp, 0.0)
    hot = np.zeros_like(p)
    hot[np.arange(len(ref)), r.y[on]] = 1
    size_h = (np.abs(lp) + np.abs(ent[:, None])) * p
    rel = 2 * S[:, None] + (6 * np.abs(d) + 24) * u
    an, hn = np.abs(a[on])[:, None], np.abs(h[on])[:, None]
    tol = r.scale * ((an * (hot + p) + hn * size_h) * rel + hn * p * 4 * S[:, None] * (1 + np.abs(ent[:, None]))
                     + (err_a[on] if np.ndim(err_a) else err_a) [:, None] * (hot + p)
                     + (err_h[on][:, None] if np.ndim(err_h) else err_h) * size_h)
    tol += HALF[dtype] * (np.abs(ref) + tol) + 2.0 ** -126  # (gradients of a subnormal size may read 0)
    _within(got[on], ref, tol, "dlogits")


def _logp_error(r, rows):
    S, d = r.bounds(rows)
    lp, lse, _, _, _ = ls.token_stats(r.z64[rows], r.y[rows], r.scale)
    return S + 4 * u * (np.abs(lp) + np.abs(lse) + 1)


SHAPES = [  # rows, columns of the ranks
    (1, [1]), (1, [5]), (3, [1, 1]), (7, [8, 3, 0, 9]), (33, [257]), (5, [1000, 1001, 7]), (130, [96]), (64, [4096, 4096]),
    (9, [32000]), (300, [515, 2, 1024, 8, 9, 1, 64, 100]), (3, [50001]), (2, [131072]), (2, [40000] * 8), (1, [300007])]
IDS = ["x".join(map(str, [m] + c)) for m, c in SHAPES]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_token_logprobs(ctx, shape, dtype):
    r = Rows(*shape, dtype=dtype, seed=sum(shape[1]), temperature=0.8)
    logp, lse, ent = (guarded((1, r.m), F32)[0] for _ in range(3))
    ctx.token_logprobs(r.logits, r.targets, logp, lse=lse, entropy=ent, scale=r.scale)
    only = guarded((1, r.m), F32)[0]
    ctx.token_logprobs(r.logits, r.targets, only, scale=r.scale)
    torch.cuda.synchronize()
    ctx.poll()
    # (the entropy's sum changes nothing about the others')
    assert torch.equal(only, logp)
    for t in (logp, lse, ent):
        assert (t.cpu().numpy()[~r.on] == 0).all()
    if not r.on.any():
        return
    on = r.on
    ref = ls.token_stats(r.z64[on], r.y[on], r.scale)
    err = _logp_error(r, on)
    pick = torch.from_numpy(on).cuda()
    _within(logp[pick], ref[0], err, "logp")
    _within(lse[pick], ref[1], err, "lse")
    S, d = r.bounds(on)
    weight = (ref[3] * np.abs(d)).sum(1)
    _within(ent[pick], ref[2], (weight + np.abs(ref[2]) + 1) * 4 * S, "entropy")


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_token_logprobs_backward(ctx, shape, types):
    r = Rows(*shape, dtype=types[0], seed=sum(shape[1]) + 1, temperature=1.3)
    rng = np.random.default_rng(1)
    a, h = _vec(np.where(r.on, rng.normal(size=r.m), np.nan)), _vec(np.where(r.on, rng.normal(size=r.m), np.nan))
    logp, lse, ent = (torch.empty(r.m, device="cuda") for _ in range(3))
    ctx.token_logprobs(r.logits, r.targets, logp, lse=lse, entropy=ent, scale=r.scale)
    a64, h64 = (np.nan_to_num(x.double().cpu().numpy()) for x in (a, h))
    lse_off = np.zeros(r.m)
    if r.on.any():  # the given lse's rounding is the probabilities' error
        lse_off[r.on] = _logp_error(r, r.on)
    for dent in (None, h):
        d = r.outputs(types[1])
        ctx.token_logprobs_backward(r.logits, r.targets, lse, a, d, entropy=None if dent is None else ent,
                                    dentropy=dent, scale=r.scale)
        torch.cuda.synchronize()
        hh = h64 if dent is not None else 0 * h64
        _check_gradient(r, d, types[1], a64, hh, np.abs(a64) * lse_off, np.abs(hh) * 2 * lse_off)
        if types[0] == types[1]:  # over the logits
            same = r.copies()
            ctx.token_logprobs_backward(same, r.targets, lse, a, same, entropy=None if dent is None else ent,
                                        dentropy=dent, scale=r.scale)
            for x, y in zip(same, d):
                assert torch.equal(x, y)
    ctx.poll()


POLICY = [  # old, ref, weights, mean, entropy coefficient
    (True, True, False, True, 0.0), (True, False, True, True, 0.02), (False, True, True, False, 0.0),
    (False, False, False, False, 0.05)]


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("how", POLICY, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_policy_loss(ctx, shape, how, types):
    old, ref, weighted, mean, coef = how
    r = Rows(*shape, dtype=types[0], seed=sum(shape[1]) + 2, temperature=0.9)
    rng = np.random.default_rng(2)
    lp = np.zeros(r.m)
    if r.on.any():
        lp[r.on] = ls.token_stats(r.z64[r.on], r.y[r.on], r.scale)[0]
    nan = np.where(r.on, 0.0, np.nan)  # rows that do not count may hold anything
    o = _vec(lp + rng.normal(size=r.m) * 0.3 + nan) if old else None
    f = _vec(lp + rng.normal(size=r.m) * 0.3 + nan) if ref else None
    adv = _vec(rng.normal(size=r.m) + nan)
    w = _vec(np.where(rng.random(r.m) < 0.2, 0.0, rng.uniform(0.5, 2, r.m))) if weighted else None
    k = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1 if ref else 0.0, entropy_coef=coef, mean=mean, scale=r.scale)
    vec64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    c64 = lambda x: float(np.float32(x))  # noqa: E731
    lo, hi = 1 - float(np.float32(1) - np.float32(0.2)), float(np.float32(1) + np.float32(0.3)) - 1
    want, wlogp, _, a, h = ls.policy_loss(r.z64, r.y, vec64(adv), vec64(o), vec64(f), vec64(w), lo, hi,
                                          c64(k["kl_coef"]), c64(coef), mean, r.scale)
    stats, logp = guarded((1, 4), F32)[0], guarded((1, r.m), F32)[0]
    d = r.outputs(types[1])
    ctx.policy_loss(r.logits, r.targets, adv, stats, old_logp=o, ref_logp=f, weights=w, logp=logp, dlogits=d, **k)
    torch.cuda.synchronize()
    ctx.poll()
    if weighted:
        r.on = r.on & (vec64(w) != 0)
    on = r.on
    assert (logp.cpu().numpy()[~on] == 0).all()
    err = np.zeros(r.m)
    if on.any():
        err[on] = _logp_error(r, on)
        _within(logp.cpu().numpy()[on], wlogp[on], err[on], "logp")
    # a loss's terms: ratio and exp(x) carry logp's error and 4 roundings; each is followed by a few more
    w64 = np.ones(r.m) if w is None else vec64(w)
    w64 = np.where(on, w64, 0.0) / (max(w64[on].sum(), 1e-30) if mean else 1.0)
    ratio = np.exp(wlogp - vec64(o)) if old else np.ones(r.m)
    x = vec64(f) - wlogp if ref else np.zeros(r.m)
    kl = c64(k["kl_coef"])
    err_a = np.nan_to_num(w64 * (np.abs(ratio * vec64(adv)) * (err + 16 * u) + kl * np.exp(x) * (err + 16 * u)
                                 + 8 * u * (np.abs(ratio * vec64(adv)) + kl * np.abs(np.expm1(x)))))
    _check_gradient(r, d, types[1], a, h, err_a, np.abs(h) * 8 * u)
    if on.any():
        S, dd = r.bounds(on)
        s4, _, ent, p, _ = ls.token_stats(r.z64[on], r.y[on], r.scale)
        e_ent = ((p * np.abs(dd)).sum(1) + np.abs(ent) + 1) * 4 * S
        e_kl = (np.exp(x[on]) + 1) * (err[on] + 16 * u) * (np.abs(x[on]) + 1)
        e_loss = err_a[on] / w64[on] + kl * e_kl + c64(coef) * e_ent + 8 * u * (np.abs(ratio * vec64(adv))[on] + kl * np.abs(x[on]))
        size = np.abs(w64[on])
        tol = np.array([(size * e).sum() for e in (e_loss, e_kl, 0 * e_kl, e_ent)]) + 8 * u * (np.abs(want) + size.sum())
        _within(stats, want, tol, "stats")
    else:
        assert (stats == 0).all()
    # the same without a gradient, and over the logits: the same bits
    again, lp2 = torch.empty(4, device="cuda"), torch.empty(r.m, device="cuda")
    ctx.policy_loss(r.logits, r.targets, adv, again, old_logp=o, ref_logp=f, weights=w, logp=lp2, **k)
    assert torch.equal(again, stats) and torch.equal(lp2, logp)
    if types[0] == types[1]:
        same = r.copies()
        ctx.policy_loss(same, r.targets, adv, again, old_logp=o, ref_logp=f, weights=w, dlogits=same, **k)
        for s, t in zip(same, d):
            assert torch.equal(s, t)
        assert torch.equal(again, stats)


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("how", [(0.0, False, 0.0, True), (0.1, True, 0.25, True), (0.3, False, -0.5, False)], ids=str)
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] > 4], ids=[i for i, s in zip(IDS, SHAPES) if s[0] > 4])
def test_preference_loss(ctx, shape, how, kind):
    smoothing, average, margin, ref = how
    types = (BF, F32) if average else (F32, BF)
    r = Rows(*shape, dtype=types[0], seed=sum(shape[1]) + 3, masked=0.2)
    rng = np.random.default_rng(3)
    lp = np.zeros(r.m)
    lp[r.on] = ls.token_stats(r.z64[r.on], r.y[r.on], r.scale)[0]
    f = _vec(np.where(r.on, lp + rng.normal(size=r.m) * 0.3, np.nan)) if ref else None
    pairs = 3
    # rows in front of the first and behind the last sequence stay as they are; one sequence is empty
    off = np.sort(rng.integers(1, r.m - 1, 2 * pairs + 1))
    off[2] = off[1]
    offsets = torch.from_numpy(off).int().cuda()
    k = dict(kind=kind, beta=0.2, label_smoothing=smoothing, margin=margin, average=average)
    c64 = lambda x: float(np.float32(x))  # noqa: E731
    ref64 = None if f is None else np.nan_to_num(f.double().cpu().numpy())
    inside = np.zeros(r.m, bool)
    inside[off[0]:off[-1]] = True
    z = np.where(r.on[:, None], r.z64, 0.0)
    want, wmargins, wlogp, _, a = ls.preference_loss(z, r.y, off, ref64, kind, c64(0.2), c64(smoothing), c64(margin),
                                                     average)
    loss, margins, logp = guarded((1, 1), F32)[0], guarded((1, pairs), F32)[0], guarded((1, r.m), F32)[0]
    d = r.outputs(types[1])
    ctx.preference_loss(r.logits, r.targets, offsets, loss, ref_logp=f, logp=logp, margins=margins, dlogits=d, **k)
    torch.cuda.synchronize()
    ctx.poll()
    assert torch.isnan(logp[torch.from_numpy(~inside).cuda()]).all()
    for t in d:
        assert torch.isnan(t[torch.from_numpy(~inside).cuda()]).all()
        t[torch.from_numpy(~inside).cuda()] = 0
    r.on = r.on & inside
    on = r.on
    err = np.zeros(r.m)
    err[on] = _logp_error(r, on)
    _within(torch.nan_to_num(logp).cpu().numpy()[inside], np.where(on, wlogp, 0)[inside], err[inside], "logp")
    e_score = np.array([err[off[s]:off[s + 1]].sum() / (max(1, on[off[s]:off[s + 1]].sum()) if average else 1)
                        for s in range(2 * pairs)])
    gap = wmargins / c64(0.2)
    e_gap = e_score[:pairs] + e_score[pairs:] + 2 * u * np.abs(gap) + u * abs(margin)
    _within(margins, wmargins, c64(0.2) * e_gap + 2 * u * np.abs(wmargins), "margins")
    # |l'| <= beta, or for squared its own size; l'' <= beta^2 / 4, 2, or 0 away from the corner
    slope = np.abs(ls.pair_loss(kind, c64(0.2), gap)[1]) + np.abs(ls.pair_loss(kind, c64(0.2), -gap)[1])
    curve = {"sigmoid": c64(0.2) ** 2, "squared": 4.0, "hinge": 0.0}[kind]
    size = np.abs(ls.pair_loss(kind, c64(0.2), gap)[0]) + np.abs(ls.pair_loss(kind, c64(0.2), -gap)[0])
    _within(loss, np.array([want]), np.array([(slope * e_gap + curve * e_gap ** 2 + 32 * u * (size + 1)).mean()]), "loss")
    err_a = np.zeros(r.m)
    for s in range(2 * pairs):
        i = s % pairs
        rows = slice(off[s], off[s + 1])
        share = 1.0 / max(1, on[rows].sum()) if average else 1.0
        err_a[rows] = share / pairs * (curve * e_gap[i] + 32 * u * (slope[i] + abs(c64(0.2))))
    _check_gradient(r, d, types[1], np.where(on, a, 0.0), np.zeros(r.m), err_a)
    # without the optional outputs, over the logits: the same bits
    again = torch.empty(1, device="cuda")
    same = r.copies()
    ctx.preference_loss(same, r.targets, offsets, again, ref_logp=f, dlogits=same if types[0] == types[1] else None, **k)
    assert torch.equal(again, loss)


def test_many_pairs_and_single_rows(ctx):
    """700 pairs of sequences of 0 to 2 rows."""
    rng = np.random.default_rng(9)
    n = rng.integers(0, 3, 1400)
    off = np.concatenate([[0], np.cumsum(n)])
    r = Rows(int(off[-1]), [40, 33], dtype=F32, seed=4, masked=0.1, special=False)
    z = np.where(r.on[:, None], r.z64, 0.0)
    want, wmargins, _, _, a = ls.preference_loss(z, r.y, off, None, "sigmoid", float(np.float32(0.5)))
    loss, margins, d = torch.empty(1, device="cuda"), torch.empty(700, device="cuda"), r.outputs(F32)
    ctx.preference_loss(r.logits, r.targets, torch.from_numpy(off).int().cuda(), loss, margins=margins, dlogits=d, beta=0.5)
    torch.cuda.synchronize()
    err = np.zeros(r.m)
    err[r.on] = _logp_error(r, r.on)
    worst = 4 * err.max()
    _within(margins, wmargins, np.full(700, worst) + 4 * u * np.abs(wmargins), "margins")
    _within(loss, np.array([want]), np.array([worst + 32 * u * abs(want)]), "loss")
    _check_gradient(r, d, F32, a, np.zeros(r.m), np.full(r.m, (worst + 32 * u) / 700))


@pytest.mark.parametrize("bad", [[-1, 2, 4], [0, 5, 4], [0, 2, 11]], ids=str)
def test_bad_offsets_compute_nothing(ctx, bad):
    import overlapped_tensor_gemm_gb300 as fo
    r = Rows(10, [30], seed=5)
    loss, logp, d = guarded((1, 1), F32)[0], guarded((1, 10), F32)[0], r.outputs(BF)
    ctx.preference_loss(r.logits, r.targets, torch.tensor(bad, dtype=torch.int32, device="cuda"), loss, logp=logp,
                        dlogits=d)
    torch.cuda.synchronize()
    with pytest.raises(fo.FoError) as e:
        ctx.poll()
    assert e.value.status == fo.FO_ERR_RANGE and "offsets" in str(e.value)
    for t in [loss, logp] + d:
        assert torch.isnan(t).all()
    test_many_pairs_and_single_rows(ctx)


def test_targets_behind_the_vocabulary(ctx):
    import overlapped_tensor_gemm_gb300 as fo
    r = Rows(6, [20, 12], seed=6, masked=0.0, dtype=F32)
    r.targets[3] = 32
    logp, stats, d = torch.empty(6, device="cuda"), torch.empty(4, device="cuda"), r.outputs(BF)
    ctx.policy_loss(r.logits, r.targets, torch.ones(6, device="cuda"), stats, logp=logp, dlogits=d)
    torch.cuda.synchronize()
    with pytest.raises(fo.FoError) as e:
        ctx.poll()
    assert e.value.status == fo.FO_ERR_RANGE and "row 3" in str(e.value)
    r.y[3], r.on[3] = -1, False
    assert logp[3] == 0
    want, _, _, a, h = ls.policy_loss(r.z64, r.y, np.ones(6))
    _within(stats, want, np.abs(want) * 1e-4 + 1e-5, "stats")
    _check_gradient(r, d, BF, a, h, np.abs(a) * 8 * u + 2.0 ** -20)


def test_rows_of_infinities_and_nan(ctx):
    """What the formula gives: a row of nothing but -infinity, one with a NaN or +infinity where it counts."""
    z = torch.zeros((5, 40), device="cuda")
    z[1] = -float("inf")
    z[2, 7] = float("nan")
    z[3, 9] = float("inf")
    y = torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    logp, lse, ent = (torch.empty(5, device="cuda") for _ in range(3))
    ctx.token_logprobs([z], y, logp, lse=lse, entropy=ent)
    want = torch.log_softmax(z.double(), 1).gather(1, y.long()[:, None])[:, 0]
    assert torch.equal(torch.isnan(logp), torch.isnan(want)) and logp[0] == logp[4]
    assert torch.isnan(ent[1:4]).all() and torch.isfinite(ent[[0, 4]]).all()
    # a target of -infinity: probability 0
    z[4, 5] = -float("inf")
    ctx.token_logprobs([z], y, logp)
    assert logp[4] == -float("inf")


def test_no_rows(ctx):
    z = torch.empty((0, 64), dtype=BF, device="cuda")
    none, y = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    stats, loss, margins = torch.full((4,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda"), torch.ones(2, device="cuda")
    ctx.token_logprobs([z], y, none)
    ctx.token_logprobs_backward([z], y, none, none, [z.clone()])
    ctx.policy_loss([z], y, none, stats, dlogits=[z.clone()])
    ctx.preference_loss([z], y, torch.zeros(5, dtype=torch.int32, device="cuda"), loss, margins=margins, dlogits=[z.clone()])
    torch.cuda.synchronize()
    ctx.poll()
    assert (stats == 0).all() and (margins == 0).all()
    assert abs(loss.item() - np.log(2)) < 4 * u


def test_a_captured_update_is_the_eager_one(ctx):
    """Policy and preference losses in one graph, replayed on new inputs, on a stream of its own."""
    r, r2 = Rows(40, [700, 33], seed=7), Rows(40, [700, 33], seed=8)
    off = torch.tensor([0, 9, 20, 31, 40], dtype=torch.int32, device="cuda")
    adv = torch.randn(40, device="cuda")
    stats, loss = torch.empty(4, device="cuda"), torch.empty(1, device="cuda")
    d, d2 = r.outputs(BF), r.outputs(BF)

    def step():
        ctx.policy_loss(r.logits, r.targets, adv, stats, dlogits=d, entropy_coef=0.1)
        ctx.preference_loss(r.logits, r.targets, off, loss, dlogits=d2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in zip(r.logits, r2.logits):
        a.copy_(b)
    r.targets.copy_(r2.targets)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (stats, loss, *d, *d2)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    ctx.poll()
    for a, b in zip(got, (stats, loss, *d, *d2)):
        assert torch.equal(a, b)


def test_rows_behind_2_31_elements(ctx):
    """40000 rows of 65536 logits in place (5.2 GB): the same bits as the same rows alone."""
    m, v = 40000, 65536
    z = torch.empty((m, v), dtype=BF, device="cuda")
    for at in range(0, m, 4000):
        z[at:at + 4000].normal_(generator=torch.Generator(device="cuda").manual_seed(at))
    y = torch.arange(m, dtype=torch.int32, device="cuda") * 7 % v
    y[::2] = -1
    # (log-probabilities are near -11.6: ratios near a half, which a negative advantage would clip)
    adv, old = 0.5 + torch.rand(m, device="cuda"), torch.full((m,), -11.0, device="cuda")
    rows = torch.tensor([1, 3, 32767, 32769, 39997, 39999], device="cuda")
    some = z[rows].clone()
    logp, stats = torch.empty(m, device="cuda"), torch.empty(4, device="cuda")
    ctx.policy_loss([z], y, adv, stats, old_logp=old, logp=logp, dlogits=[z], mean=False)
    few, s2 = torch.empty(6, device="cuda"), torch.empty(4, device="cuda")
    ctx.policy_loss([some], y[rows], adv[rows], s2, old_logp=old[rows], logp=few, dlogits=[some], mean=False)
    torch.cuda.synchronize()
    ctx.poll()
    # (fewer rows may be cut otherwise: the sums' order differs)
    assert torch.allclose(logp[rows], few, rtol=0, atol=1e-4)
    assert torch.allclose(z[rows].float(), some.float(), rtol=2.0 ** -7, atol=1e-9)
    assert z[rows].abs().sum() > 0 and (z[32768] == 0).all()


def test_a_pair_whose_target_has_no_probability(ctx):
    """The preferred sequence holds a token of probability 0: the loss is infinite, the other pair's gradient is not."""
    z = torch.zeros((4, 16), device="cuda")
    z[0, 3] = -float("inf")
    y = torch.tensor([3, 1, 2, 1], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    (loss, margins, logp), d = (torch.empty(n, device="cuda") for n in (1, 2, 4)), torch.empty_like(z)
    ctx.preference_loss([z], y, off, loss, logp=logp, margins=margins, dlogits=[d], beta=0.5)
    torch.cuda.synchronize()
    ctx.poll()
    assert loss.item() == float("inf") and margins[0] == -float("inf") and margins[1] == 0
    assert logp[0] == -float("inf") and torch.isfinite(logp[1:]).all()
    # pair 1: slope -beta / 2, over two pairs
    p = 1 / 16
    want = torch.full((16,), 0.125 * p, device="cuda")
    want[1] -= 0.125
    assert torch.allclose(d[1], want, atol=1e-6) and torch.allclose(d[3], -want, atol=1e-6)


def test_summed_log_probabilities_keep_twice_fp32(ctx):
    """A pair of 4000 tokens a side: its gap, a difference of sums near -40000, to 4000 errors of a token's own sum
    (its exponentials' 2^-22 and roundings, at random signs: 3e-7 each) -- fp32 sums would be off by 2e-3."""
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn((8000, 600), generator=g, device="cuda") * 2
    y = torch.randint(0, 600, (8000,), generator=g, device="cuda", dtype=torch.int32)
    off = torch.tensor([0, 4000, 8000], dtype=torch.int32, device="cuda")
    loss, margins = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ctx.preference_loss([z], y, off, loss, margins=margins, beta=1.0)
    lp = torch.log_softmax(z.double(), 1).gather(1, y.long()[:, None])[:, 0]
    gap = (lp[:4000].sum() - lp[4000:].sum()).item()
    assert abs(margins.item() - gap) <= 2.0 ** -24 * abs(gap) + 5 * 3e-7 * 8000 ** 0.5


@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)], ids=str)
@pytest.mark.parametrize("m", [1, 5])
def test_rows_that_do_not_fit_shared_memory(ctx, types, m):
    """Vocabularies of a million: a policy loss's rows are read twice."""
    r = Rows(m, [500001, 400008, 7, 100000], dtype=types[0], seed=m, masked=0.2)
    rng = np.random.default_rng(6)
    lp = np.zeros(m)
    lp[r.on] = ls.token_stats(r.z64[r.on], r.y[r.on])[0]
    adv, old = rng.uniform(0.5, 1.5, m), lp + 0.1
    want, wlogp, _, a, h = ls.policy_loss(r.z64, r.y, adv.astype(np.float32).astype(np.float64),
                                          old.astype(np.float32).astype(np.float64), ent_coef=float(np.float32(0.02)))
    stats, logp, d = torch.empty(4, device="cuda"), torch.empty(m, device="cuda"), r.outputs(types[1])
    ctx.policy_loss(r.logits, r.targets, _vec(adv), stats, old_logp=_vec(old), logp=logp, dlogits=d, entropy_coef=0.02)
    torch.cuda.synchronize()
    ctx.poll()
    err = np.zeros(m)
    err[r.on] = _logp_error(r, r.on)
    _within(logp, wlogp, err, "logp")
    # (the ratio is exp of a difference that is off by err)
    _check_gradient(r, d, types[1], a, h, np.abs(a) * (err + 32 * u), np.abs(h) * 8 * u)
    if types[0] == types[1]:
        same = r.copies()
        ctx.policy_loss(same, r.targets, _vec(adv), stats, old_logp=_vec(old), dlogits=same, entropy_coef=0.02)
        for x, y in zip(same, d):
            assert torch.equal(x, y)


def test_calls_behind_a_failed_one(ctx):
    """The losses wait for nothing that an earlier call's failure ends: with its abort word raised they are right."""
    import overlapped_tensor_gemm_gb300 as fo
    from test_gpu_p_training_failures import _fail
    r = Rows(50, [3000, 1001], seed=9)
    adv, stats, loss = torch.ones(50, device="cuda"), torch.empty(4, device="cuda"), torch.empty(1, device="cuda")
    off = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    got = []
    with fo.Context(0) as c:
        for fail in (False, True):
            if fail:
                _fail(c)
            d, d2 = r.outputs(BF), r.outputs(BF)
            c.policy_loss(r.logits, r.targets, adv, stats, dlogits=d)
            c.preference_loss(r.logits, r.targets, off, loss, dlogits=d2)
            torch.cuda.synchronize()
            got.append([t.clone() for t in (stats, loss, *d, *d2)])
        with pytest.raises(fo.FoError) as e:
            c.poll()
        assert e.value.status == fo.FO_ERR_TIMEOUT
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_contexts_of_four_threads(ctx):
    """Each thread its own context and stream, losses of several shapes at once: the bits of one after the other."""
    import threading

    import overlapped_tensor_gemm_gb300 as fo
    rows = [Rows(*s, seed=20 + i) for i, s in enumerate([(64, [4096, 4096]), (300, [515, 64, 100]), (9, [32000]), (130, [96])])]
    adv = [torch.rand(r.m, device="cuda") for r in rows]

    def step(c, i):
        r = rows[i]
        stats, d = torch.empty(4, device="cuda"), r.outputs(BF)
        c.policy_loss(r.logits, r.targets, adv[i], stats, dlogits=d, entropy_coef=0.1)
        return [stats] + d
    want = [[t.clone() for t in step(ctx, i)] for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with fo.Context(0) as c, torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = step(c, i)
                torch.cuda.current_stream().synchronize()
                c.poll()
                wrong.extend((i, k) for k, (x, y) in enumerate(zip(got, want[i])) if not torch.equal(x, y))
        except Exception as e:  # noqa: BLE001
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_one_column_is_certain(ctx):
    """Rows of one finite column: log-probability, entropy and gradient are 0 to the bit, lse the column itself."""
    z = torch.full((3, 40), -float("inf"), device="cuda")
    z[:, 7] = torch.tensor([0.0, -3.5, 88.25], device="cuda")
    y = torch.full((3,), 7, dtype=torch.int32, device="cuda")
    logp, lse, ent = (torch.empty(3, device="cuda") for _ in range(3))
    ctx.token_logprobs([z], y, logp, lse=lse, entropy=ent)
    stats, d = torch.empty(4, device="cuda"), torch.empty_like(z)
    ctx.policy_loss([z], y, torch.ones(3, device="cuda"), stats, dlogits=[d], entropy_coef=0.5)
    assert (logp == 0).all() and (ent == 0).all() and torch.equal(lse, z[:, 7]) and (d == 0).all()


@pytest.mark.parametrize("call", ["token_logprobs", "token_logprobs_backward", "preference_loss"])
def test_every_call_tells_of_a_target_behind_the_vocabulary(ctx, call):
    import overlapped_tensor_gemm_gb300 as fo
    r = Rows(7, [20, 12], seed=21, masked=0.0, dtype=F32)
    r.targets[5] = 2 ** 31 - 1
    logp, d, one = torch.full((7,), 3.0, device="cuda"), r.outputs(BF), torch.ones(7, device="cuda")
    if call == "token_logprobs":
        ctx.token_logprobs(r.logits, r.targets, logp)
    elif call == "token_logprobs_backward":
        ctx.token_logprobs_backward(r.logits, r.targets, one, one, d)
    else:
        off = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
        ctx.preference_loss(r.logits, r.targets, off, torch.empty(1, device="cuda"), logp=logp, dlogits=d)
    torch.cuda.synchronize()
    with pytest.raises(fo.FoError) as e:
        ctx.poll()
    assert e.value.status == fo.FO_ERR_RANGE and "row 5" in str(e.value)
    assert call == "token_logprobs_backward" or logp[5] == 0
    assert call == "token_logprobs" or all((x[5] == 0).all() for x in d)
