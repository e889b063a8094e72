"""Norms around a block (fo_norm_residual and its backward) and rotary positions (fo_rope and its
backward) against the fp64 oracle.

Tolerances, element by element: half a step of the output's type relative to the value
(bf16 2^-8, fp32 2^-24), plus fp32 arithmetic: an operation chain of at most DEPTH roundings
(a row sum: 16 products per thread, 5 shuffles, at most 32 warps; then square root, division and
a few products) relative to the sum of the magnitudes that enter the element.  Sums over tokens
add one rounding per token."""
import numpy as np
import pytest
import torch

from helpers import guarded
from oracle import training as tr

pytestmark = pytest.mark.gpu

DEPTH = 128
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _close(got, ref, mag, dtype, what, more=0):
    got = got.double().cpu().numpy()
    tol = U[dtype] * np.abs(ref) + (DEPTH + more) * 2.0 ** -24 * mag
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got.size, np.abs(got - ref)[bad].max(), tol[bad].max())


def _randn(g, shape, dtype, std=1.0, mean=0.0, pitch=True):
    """Values of `dtype` on the GPU (rows 16-byte aligned, padding NaN) and their fp64 copy."""
    v = (torch.randn(shape, generator=g) * std + mean).to(dtype)
    if len(shape) == 1 or not pitch:
        return v.cuda(), v.double().numpy()
    per = 16 // v.element_size()
    base = torch.full((shape[0], (shape[1] + per - 1) // per * per + per), float("nan"), dtype=dtype, device="cuda")
    base[:, :shape[1]] = v.cuda()
    return base[:, :shape[1]], v.double().numpy()


CASES = [  # P, m, H, residual, activations, parameters, post, gate, pre, alpha
    (1, 1, 1, BF, BF, BF, True, "row", True, 1.0),
    (2, 5, 24, F32, BF, BF, True, "row", True, 0.5),
    (3, 7, 257, BF, BF, F32, False, "token", True, 1.0),
    (1, 300, 1001, F32, F32, F32, True, "token", False, 1.25),
    (4, 65, 512, BF, F32, BF, True, None, True, 1.0),
    (2, 129, 4096, BF, BF, BF, True, "row", True, 0.75),
    (1, 40, 8192, F32, BF, F32, False, "row", True, 1.0),
    (1, 9, 16384, BF, BF, BF, True, "row", True, 1.0),
    (1, 3, 16383, F32, F32, BF, True, "token", True, 1.0),
    (8, 33, 128, BF, BF, BF, True, None, False, 2.0),
]


def _inputs(case, seed):
    P, m, H, tr_, ta, tp, post, gate, pre, alpha = case
    g = torch.Generator().manual_seed(seed)
    mats = lambda dt, std: list(zip(*[_randn(g, (m, H), dt, std) for _ in range(P)]))  # noqa: E731
    vec = lambda on, mean: _randn(g, (H,), tp, 0.25, mean) if on else (None, None)     # noqa: E731
    w_post, w_pre = vec(post, 1.0), vec(pre, 1.0)
    if gate == "token":
        gt = mats(tp, 0.5)
        gt = (list(gt[0]), gt[1])
    else:
        gt = vec(gate is not None, 0.5)
    return mats, w_post, w_pre, gt


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(x).replace("torch.", "") for x in c))
def test_norm_forward(ctx, case):
    P, m, H, t_res, t_act, _, post, gate, pre, alpha = case
    mats, w_post, w_pre, gt = _inputs(case, 100 + H)
    (R, r64), (Y, y64) = mats(t_res, 2.0), mats(t_act, 1.0)
    RO = [guarded((m, H), t_res) for _ in range(P)]
    X = [guarded((m, H), t_act) for _ in range(P)] if pre else None
    ctx.norm_residual(R, Y, RO, X, w_post=w_post[0], gate=gt[0], w_pre=w_pre[0], residual_scale=alpha, eps=1e-5)
    torch.cuda.synchronize()
    for p in range(P):
        g64 = gt[1][p] if gate == "token" else gt[1]
        ro, x, mag = tr.norm_residual(r64[p], y64[p], w_post[1], g64, w_pre[1], alpha, 1e-5)
        _close(RO[p], ro, mag, t_res, f"R_out {p}")
        if pre:
            scale = np.abs(w_pre[1]) / np.sqrt((ro * ro).mean(-1, keepdims=True) + 1e-5)
            # the row's rms carries the row's relative error: magnitudes of the largest element count
            _close(X[p], x, mag * scale + np.abs(x) * (mag * np.abs(ro)).sum(-1, keepdims=True)
                   / ((ro * ro).sum(-1, keepdims=True) + 1e-30), t_act, f"X {p}")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(str(x).replace("torch.", "") for x in c))
@pytest.mark.parametrize("rest", [True, False])
def test_norm_backward(ctx, case, rest):
    P, m, H, t_res, t_act, t_par, post, gate, pre, alpha = case
    if not pre and not rest:
        rest = True
    mats, w_post, w_pre, gt = _inputs(case, 200 + H)
    (R, r64), (Y, y64) = mats(t_res, 2.0), mats(t_act, 1.0)
    dX, dx64 = mats(t_act, 1.0) if pre else (None, [None] * P)
    dRO, dr64 = mats(t_res, 1.0) if rest else (None, [None] * P)
    dR, dY = [guarded((m, H), t_res) for _ in range(P)], [guarded((m, H), t_act) for _ in range(P)]
    vec = lambda on, dt: guarded((1, H), dt)[0] if on else None  # noqa: E731
    d_post, d_pre = vec(post, F32), vec(pre, t_par)
    d_gate = [guarded((m, H), t_par) for _ in range(P)] if gate == "token" else vec(gate is not None, F32)
    how = dict(w_post=w_post[0], gate=gt[0], w_pre=w_pre[0], residual_scale=alpha, eps=1e-5)
    out = dict(dw_post=d_post, dgate=d_gate, dw_pre=d_pre)
    ctx.norm_residual_backward(list(R), list(Y), None if dX is None else list(dX), None if dRO is None else list(dRO),
                               dR, dY, **how, **out)
    torch.cuda.synchronize()
    total, tmag = {}, {}
    for p in range(P):
        g64 = gt[1][p] if gate == "token" else gt[1]
        g, mag = tr.norm_residual_backward(r64[p], y64[p], dx64[p], dr64[p], w_post[1], g64, w_pre[1], alpha, 1e-5)
        _close(dR[p], g["r"], mag["r"], t_res, f"dR {p}")
        _close(dY[p], g["y"], mag["y"], t_act, f"dY {p}")
        if gate == "token":
            _close(d_gate[p], g["gate"], mag["gate"], t_par, f"dgate {p}")
        for k in ("w_post", "w_pre", "gate"):
            if k in g and np.ndim(g[k]) == 1:
                total[k] = total.get(k, 0) + g[k]
                tmag[k] = tmag.get(k, 0) + mag[k]
    for k, got, dt in (("w_post", d_post, F32), ("w_pre", d_pre, t_par), ("gate", d_gate, F32)):
        if k in total:
            _close(got, total[k], tmag[k], dt, "d" + k, more=P * m)
    # the same inputs give the same bits
    again = {k: (torch.empty_like(v) if v is not None and not isinstance(v, list) else v) for k, v in out.items()}
    ctx.norm_residual_backward(list(R), list(Y), None if dX is None else list(dX), None if dRO is None else list(dRO),
                               dR, dY, **how, **again)
    for k, v in out.items():
        if v is not None and not isinstance(v, list):
            assert torch.equal(v, again[k]), k


@pytest.mark.parametrize("case", [
    (1, 307, 8192, BF, BF, BF, True, "row", True, 1.0), (2, 3, 8192, BF, BF, F32, True, "row", True, 0.5),
    (2, 12, 512, BF, BF, BF, True, "row", True, 1.0), (1, 40, 1024, F32, F32, F32, True, "row", True, 1.5),
    (1, 41, 1024, F32, BF, F32, True, "row", True, 1.0), (1, 21, 8192, F32, BF, BF, True, "row", True, 1.0),
    (1, 17, 6144, F32, F32, F32, True, "row", True, 0.5), (2, 9, 5120, BF, BF, BF, True, "row", True, 1.0),
    (1, 11, 5128, BF, BF, BF, True, "row", True, 1.0), (1, 7, 9000, BF, F32, BF, True, "row", True, 1.0),
    (3, 5, 4096, BF, F32, BF, True, "row", True, 1.0), (1, 19, 8192, BF, BF, F32, False, None, True, 1.0),
    (2, 8, 2048, F32, BF, BF, False, "row", True, 0.5), (1, 31, 4096, BF, BF, BF, True, None, True, 1.0),
    (1, 12, 8192, F32, BF, BF, False, None, True, 1.0),
], ids=lambda c: "x".join(str(x).replace("torch.", "") for x in c))
def test_norm_of_a_whole_block(ctx, case):
    """Every operand given, rows that fill their threads (and one count of rows that does not)."""
    test_norm_forward(ctx, case)
    test_norm_backward(ctx, case, True)


def test_norm_without_a_block_and_in_place(ctx):
    g = torch.Generator().manual_seed(5)
    R, r64 = _randn(g, (37, 320), F32)
    w, w64 = _randn(g, (320,), BF, 0.2, 1.0)
    X = guarded((37, 320), BF)
    ctx.norm_residual([R], None, None, [X], w_pre=w)
    _, x, mag = tr.norm_residual(r64, None, w_pre=w64)
    _close(X, x, 2 * np.abs(x), BF, "X")
    dX, dx64 = _randn(g, (37, 320), BF)
    dR, dw = guarded((37, 320), F32), torch.empty(320, device="cuda")
    ctx.norm_residual_backward([R], None, [dX], None, [dR], None, w_pre=w, dw_pre=dw)
    got, mag = tr.norm_residual_backward(r64, None, dx64, None, w_pre=w64)
    _close(dR, got["r"], mag["r"], F32, "dR")
    _close(dw, got["w_pre"], mag["w_pre"], F32, "dw", more=37)
    # R_out over R, X over Y; dR over dR_out, dY over dX: the same bits as apart
    Y, _ = _randn(g, (37, 320), BF)
    apart = [guarded((37, 320), F32), guarded((37, 320), BF)]
    ctx.norm_residual([R], [Y], [apart[0]], [apart[1]], w_post=w, w_pre=w)
    r2, y2 = R.clone(), Y.clone()
    ctx.norm_residual([r2], [y2], [r2], [y2], w_post=w, w_pre=w)
    assert torch.equal(r2, apart[0]) and torch.equal(y2, apart[1])
    grads = [torch.empty(320, device="cuda") for _ in range(4)]
    ctx.norm_residual_backward([R], [Y], [dX], [dR], [apart[0]], [apart[1]], w_post=w, w_pre=w, dw_post=grads[0],
                               dw_pre=grads[1])
    r2, y2 = dR.clone(), dX.clone()
    ctx.norm_residual_backward([R], [Y], [y2], [r2], [r2], [y2], w_post=w, w_pre=w, dw_post=grads[2], dw_pre=grads[3])
    assert torch.equal(r2, apart[0]) and torch.equal(y2, apart[1])
    assert torch.equal(grads[0], grads[2]) and torch.equal(grads[1], grads[3])


def test_norm_after_a_call_that_timed_out(ctx):
    """The abort word of a timed-out call ends other kernels' waits; a norm waits for its own copies only."""
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator().manual_seed(6)
    m, h = 256, 1
    qkv = [torch.randn((m, 128), generator=g).to(BF).cuda() for _ in range(3)]
    O = [torch.empty((m, 128), dtype=BF, device="cuda") for _ in range(2)]
    with fo.Context(0) as c:
        c.qsplit_attn([qkv[0]] * 2, [qkv[1]] * 2, [qkv[2]] * 2, O, heads=h, head_dim=128, fault="skip_hop",
                      timeout_us=20000)
        R, r64 = _randn(g, (300, 4096), F32)
        w, w64 = _randn(g, (4096,), BF, 0.2, 1.0)
        X = guarded((300, 4096), BF)
        c.norm_residual([R], None, None, [X], w_pre=w)
        torch.cuda.synchronize()
        _, x, _ = tr.norm_residual(r64, None, w_pre=w64)
        _close(X, x, 2 * np.abs(x), BF, "X")
        with pytest.raises(fo.FoError) as e:
            c.poll()
        assert e.value.status == fo.FO_ERR_TIMEOUT


def test_norm_no_rows(ctx):
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    ctx.norm_residual([e], [e.clone()], [e.clone()], [e.clone()], w_post=w, w_pre=w)
    dw = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    ctx.norm_residual_backward([e], [e.clone()], [e.clone()], [e.clone()], [e.clone()], [e.clone()], w_post=w, w_pre=w,
                               dw_post=dw[0], dw_pre=dw[1])
    torch.cuda.synchronize()
    assert (dw[0] == 0).all() and (dw[1] == 0).all()  # sums over no tokens


ROPE = [  # P, m, heads, head_dim, rot_dim, layout, dtype, scaling, start, scattered
    (1, 1, 1, 2, 2, "half", BF, {}, 0, False),
    (1, 1, 40, 128, 128, "half", BF, {}, 77, False),
    (2, 37, 3, 64, 64, "interleaved", BF, {}, (1 << 31) - 40, False),
    (1, 200, 5, 96, 64, "half", F32, dict(scaling="linear", factor=4.0), 1 << 20, True),
    (3, 65, 2, 128, 48, "interleaved", F32, dict(scaling="banded", factor=8.0, original_length=8192), 100000, False),
    (1, 129, 7, 80, 20, "half", BF, dict(scaling="ramped", factor=16.0, original_length=4096), 0, True),
    (2, 50, 3, 26, 14, "interleaved", BF, {}, 1 << 33, False),
    (1, 700, 4, 512, 512, "half", F32, {}, 3, False),
    (1, 33, 2, 18, 10, "half", F32, {}, -1000, True),
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c[:7]))
@pytest.mark.parametrize("backward", [False, True])
def test_rope(ctx, case, backward):
    import overlapped_tensor_gemm_gb300 as fo
    P, m, h, d, rot, layout, dt, how, start, scattered = case
    g = torch.Generator().manual_seed(rot)
    X, x64 = zip(*[_randn(g, (m, h * d), dt) for _ in range(P)])
    Y = [guarded((m, h * d), dt) for _ in range(P)]
    pos = None
    where = [start + 1000 * p + np.arange(m) for p in range(P)]
    if scattered:
        pos = [(start + torch.randint(0, 5000, (m,), generator=g)).to(torch.int32).cuda() for _ in range(P)]
        where = [t.cpu().numpy().astype(np.int64) for t in pos]
    table = fo.RopeTable(rot, base=10000.0, **how)
    call = ctx.rope_backward if backward else ctx.rope
    args = dict(head_dim=d, layout=layout, positions=pos, start=start, rank_stride=1000)
    call(list(X), Y, table, **args)
    torch.cuda.synchronize()
    kw = {k: v for k, v in how.items() if k in ("scaling", "factor")}
    if "original_length" in how:
        kw.update(length=how["original_length"], low=1.0, high=32.0 if how["scaling"] == "ramped" else 4.0)
    freq, amp = tr.rope_frequencies(rot, 10000.0, **kw)
    # angles: the table's fractions are exact to 2^-54 of a turn (64-bit pow) times the position, in the oracle's
    # radians as in the library's turns; cos and sin to 4 roundings, two products and a sum
    off = 16 * 2.0 ** -53 * max(abs(start) + 10000, 1)
    for p in range(P):
        want = tr.rope(x64[p].reshape(m, h, d), where[p], freq, amp, layout == "interleaved",
                       -1.0 if backward else 1.0).reshape(m, h * d)
        mag = tr.rope(np.abs(x64[p]).reshape(m, h, d), np.zeros(m), np.zeros(rot // 2), 1.0).reshape(m, h, d)
        a, b = ((slice(0, rot, 2), slice(1, rot, 2)) if layout == "interleaved"
                else (slice(0, rot // 2), slice(rot // 2, rot)))
        both = amp * (mag[..., a] + mag[..., b])
        mag[..., a] = mag[..., b] = both
        got = Y[p].double().cpu().numpy()
        tol = U[dt] * np.abs(want) + (8 * 2.0 ** -24 + off) * mag.reshape(m, h * d)
        assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
        if rot < d:  # what does not turn is copied
            assert torch.equal(Y[p].reshape(m, h, d)[..., rot:], X[p].reshape(m, h, d)[..., rot:])
    # in place: the same bits
    Z = [torch.empty((m, x.stride(0)), dtype=dt, device="cuda")[:, :h * d].copy_(x) for x in X]
    call(Z, Z, table, **args)
    for p in range(P):
        assert torch.equal(Z[p], Y[p])


def test_rope_on_columns_of_a_wider_matrix(ctx):
    # the query and key heads of a QKV matrix turned in place; the value heads stay
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((50, 6 * 64), generator=g).to(BF).cuda()
    keep = qkv.clone()
    table = fo.RopeTable(64)
    view = qkv[:, :4 * 64]
    ctx.rope([view], [view], table)
    assert torch.equal(qkv[:, 4 * 64:], keep[:, 4 * 64:])
    want = guarded((50, 4 * 64), BF)
    ctx.rope([keep[:, :4 * 64]], [want], table)
    assert torch.equal(view, want)


def test_streams_graphs_and_devices(ctx):
    import overlapped_tensor_gemm_gb300 as fo
    g = torch.Generator().manual_seed(8)
    R, _ = _randn(g, (64, 256), BF)
    Y, _ = _randn(g, (64, 256), BF)
    w = torch.ones(256, dtype=BF, device="cuda")
    ro, x, out = torch.empty_like(R), torch.empty_like(R), torch.empty_like(R)
    table = fo.RopeTable(64)

    def step(stream=None):
        ctx.norm_residual([R], [Y], [ro], [x], w_post=w, w_pre=w, stream=stream)
        ctx.rope([x], [out], table, start=9, stream=stream)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    step(stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    R.copy_(torch.randn((64, 256), generator=g).to(BF))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    with pytest.raises(ValueError):
        ctx.rope([x.cpu()], [out], table)
    with pytest.raises(ValueError):
        ctx.norm_residual([R], [Y], [ro], [x], w_post=w.cpu(), w_pre=w)
