"""The AdamW step over many tensors, the gradients' norm and 8-bit states against the fp64 oracle.

Tolerances, u = 2^-24: m and v are sums of two products (4 roundings of their terms); the update divides by an
approximate square root (2^-22), with corrections rounded to fp32: 32 u of its size, and 4 u of each term of the
weight.  8-bit states are compared as codes: the same code, but where the random part of a step is so close to
deciding otherwise that fp32's error does."""
import numpy as np
import pytest
import torch

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


class Set:
    """Tensors of the given sizes between guards of 7 (bytes: 77); kinds: (parameter type, gradient type,
    master, bits) in turn."""

    def __init__(self, sizes, kinds, seed=0, zero=False):
        import overlapped_tensor_gemm_gb300 as fo
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.kinds = sizes, [kinds[i % len(kinds)] for i in range(len(sizes))]
        self._guards = []
        names = ("w", "g", "master", "m", "v", "m_scale", "v_range")
        for x in names:
            setattr(self, x, [])
        for n, (pt, gt, master, bits) in zip(sizes, self.kinds):
            nb = -(-n // 256)
            wide = torch.exp2(torch.randn(nb, generator=g)).repeat_interleave(256)[:n]
            w = torch.randn(n, generator=g) * 0.05
            m, v = torch.randn(n, generator=g) * 1e-3 * wide, (1e-3 * wide) ** 2 * torch.exp2(torch.randn(n, generator=g))
            if zero:
                m, v = 0 * m, 0 * v
            elif n > 5:
                v[n // 2] = m[n // 2] = 0.0
            self.w.append(self._place(w.to(pt)))
            self.g.append(self._place((torch.randn(n, generator=g) * 1e-3 * wide).to(gt)))
            self.master.append(self._place(w) if master else None)
            if bits == 32:
                self.m.append(self._place(m))
                self.v.append(self._place(v))
                self.m_scale.append(None)
                self.v_range.append(None)
                continue
            word = torch.zeros(n, dtype=torch.int64).numpy().astype(np.uint64)
            q, scale, code, low, gap, _, _ = ls.pack(m.double().numpy(), v.double().numpy(), word)
            self.m.append(self._place(torch.from_numpy(q).float().to(torch.float8_e4m3fn)))
            self.v.append(self._place(torch.from_numpy(code).to(torch.uint8)))
            self.m_scale.append(self._place(torch.from_numpy(scale).float()))
            self.v_range.append(self._place(torch.from_numpy(np.stack([low, gap], 1).reshape(-1)).float()))
        self.group = fo.AdamWTensors(self.w, self.g, self.m, self.v, master=self.master, m_scale=self.m_scale,
                                     v_range=self.v_range)

    def _place(self, t):
        """t on the GPU, 64 bytes into a buffer that ends 64 bytes and a bit behind it"""
        raw = t.contiguous().view(torch.uint8) if t.numel() else torch.empty(0, dtype=torch.uint8)
        base = torch.full((raw.numel() + 128,), 77, dtype=torch.uint8, device="cuda")
        base[64:64 + raw.numel()] = raw.cuda()
        self._guards.append((base, raw.numel()))
        return base[64:64 + raw.numel()].view(t.dtype)

    def check_guards(self):
        for base, n in self._guards:
            assert (base[:64] == 77).all() and (base[64 + n:] == 77).all()

    def values(self, i):
        """w (as the step reads it), gradient, m, v in 64 bits"""
        up = lambda t: t.double().cpu().numpy()  # noqa: E731
        w = up(self.w[i] if self.master[i] is None else self.master[i])
        if self.kinds[i][3] == 32:
            return w, up(self.g[i]), up(self.m[i]), up(self.v[i])
        low, gap = up(self.v_range[i]).reshape(-1, 2).T
        m, v = ls.unpack(up(self.m[i]), up(self.m_scale[i]), up(self.v[i]), low, gap)
        return w, up(self.g[i]), m, v

    def state(self):
        return [t.clone() for x in ("w", "master", "m", "v", "m_scale", "v_range") for t in getattr(self, x) if t is not None]


KINDS = [(BF, BF, True, 32), (F32, F32, False, 32), (BF, F32, False, 32), (BF, BF, True, 8), (F32, BF, False, 8),
         (BF, F32, False, 8), (F32, F32, False, 8), (BF, F32, True, 8), (BF, BF, False, 32), (F32, BF, False, 32),
         (BF, BF, False, 8), (BF, F32, True, 32)]
SIZES = [1, 3, 4, 127, 128, 129, 255, 256, 257, 511, 1000, 2048, 5003, 40001, 0, 2, 70000, 300007, 9, 31]
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-7, weight_decay=0.1)


def _check_step(s, before, step, factor, stochastic=False, seed=0, err_factor=0.0):
    """Every tensor against the oracle's step from `before` (values of every tensor)."""
    c64 = lambda x: float(np.float32(x))  # noqa: E731
    lr, eps, wd = (c64(HYPER[x]) for x in ("lr", "eps", "weight_decay"))
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    for i, (n, (pt, gt, master, bits)) in enumerate(zip(s.sizes, s.kinds)):
        if n == 0:
            continue
        w, g, m, v = before[i]
        rw, rm, rv = ls.adamw(w, g, m, v, step, lr, b1, b2, eps, wd, factor)
        # v of 8 bits is 2^x with x rounded to fp32 and an exponential of 2^-22
        dec = 64 * u if bits == 8 else 0.0
        em = 4 * u * (np.abs(b1 * m) + np.abs((1 - b1) * g * factor)) + np.abs((1 - b1) * g * factor) * err_factor
        ev = 6 * u * rv + dec * v + 2 * err_factor * (1 - b2) * (g * factor) ** 2
        rel_v = np.where(rv > 0, ev / np.where(rv > 0, rv, 1), 0)
        update = np.abs(rm / (1 - b1 ** step)) / (np.sqrt(rv / (1 - b2 ** step)) + eps)
        e_up = update * (rel_v + 32 * u) + em / (1 - b1 ** step) / (np.sqrt(rv / (1 - b2 ** step)) + eps)
        ew = 4 * u * (np.abs(w) * (1 + lr * wd) + lr * update) + lr * e_up
        up = lambda t: t.double().cpu().numpy()  # noqa: E731

        def near(got, ref, tol, what):
            bad = ~(np.abs(got - ref) <= tol)
            assert not bad.any(), (i, n, s.kinds[i], what, int(bad.sum()), got[bad][:3], ref[bad][:3], tol[bad][:3])
        if master:
            near(up(s.master[i]), rw, ew, "master")
        word = ls.words(seed, step, i, n)
        if pt == BF and not master and stochastic:
            # one of the two bf16 values around the new weight
            step_w = np.exp2(np.floor(np.log2(np.maximum(np.abs(rw), 1e-38))) - 7)
            near(up(s.w[i]), rw, step_w + ew, "w, stochastic")
        else:
            near(up(s.w[i]), rw, HALF[pt] * np.abs(rw) + ew * (1 + HALF[pt]), "w")
        if bits == 32:
            near(up(s.m[i]), rm, em, "m")
            near(up(s.v[i]), rv, ev, "v")
            continue
        q, scale, code, low, gap, near_m, near_v = ls.pack(rm, rv, word)
        got_scale, got_range = up(s.m_scale[i]), up(s.v_range[i]).reshape(-1, 2)
        top = np.abs(ls._blocks(rm, 0)).max(1)
        near(got_scale, scale, (8 * u * top + ls._blocks(em, 0).max(1)) / 448, "m_scale")
        near(got_range[:, 0], low, (np.abs(low) + 8) * 8 * u + ls._blocks(rel_v, 0).max(1) * 2, "low")
        near(got_range[:, 1], gap, (np.abs(low) + 32) * 16 * u / 254 + ls._blocks(rel_v, 0).max(1) * 4 / 254, "gap")
        # codes: a neighbour only where the deciding part is nearer than the error in steps
        rep = lambda x: np.repeat(x, 256)[:n]  # noqa: E731
        x = np.abs(rm) / np.where(rep(scale) > 0, rep(scale), 1)
        e_steps = (em / np.where(rep(scale) > 0, rep(scale), 1) + 16 * u * (x + 2.0 ** -6)) / ls.e4m3_step(x) + 1e-9
        got_q = up(s.m[i])
        same = got_q == q
        close = np.abs(got_q - q) <= ls.e4m3_step(q) * 1.001
        bad = ~(same | (close & (near_m <= e_steps)))
        assert not bad.any(), (i, "m codes", int(bad.sum()), got_q[bad][:3], q[bad][:3], near_m[bad][:3], e_steps[bad][:3])
        y_err = ((np.abs(rep(low)) + 32) * 8 * u + 4 * rel_v + 2e-7) / np.where(rep(gap) > 0, rep(gap), 1.0) + 1e-6
        y_err = np.where(rep(gap) > 0, y_err, 300.0) + 254 * y_err * 0.02
        got_c = up(s.v[i])
        bad = ~((got_c == code) | ((np.abs(got_c - code) <= 1 + y_err) & (near_v <= 2 * y_err) & (got_c > 0) & (code > 0)))
        assert not bad.any(), (i, "v codes", int(bad.sum()), got_c[bad][:3], code[bad][:3], near_v[bad][:3], y_err[bad][:3])


@pytest.mark.parametrize("step", [1, 2, 1000])
@pytest.mark.parametrize("stochastic", [False, True])
def test_one_step_of_every_kind(ctx, step, stochastic):
    s = Set(SIZES * 2, KINDS, seed=step, zero=step == 1)
    before = [s.values(i) if n else None for i, n in enumerate(s.sizes)]
    ctx.adamw_step(s.group, step=step, stochastic=stochastic, seed=0x123456789ABCDEF, **HYPER)
    torch.cuda.synchronize()
    ctx.poll()
    s.check_guards()
    _check_step(s, before, step, 1.0, stochastic, 0x123456789ABCDEF)


def test_gradient_scale_and_clipping(ctx):
    s = Set(SIZES, KINDS, seed=5)
    norm = torch.empty(1, device="cuda")
    ctx.grad_norm(s.group, norm)
    want = np.sqrt(sum((g.double() ** 2).sum().item() for g in s.g))
    # 512 fp32 squares in a row, their root halves the error; the rest is fp64
    assert abs(norm.item() - want) <= want * (256 + 8) * u
    before = [s.values(i) if n else None for i, n in enumerate(s.sizes)]
    scale, limit = 0.125, 0.05 * want
    ctx.adamw_step(s.group, step=3, norm=norm, max_norm=limit, grad_scale=scale, seed=11, **HYPER)
    _check_step(s, before, 3, scale * limit / (scale * want), seed=11, err_factor=270 * u)
    before = [s.values(i) if n else None for i, n in enumerate(s.sizes)]
    ctx.adamw_step(s.group, step=4, norm=norm, max_norm=2 * want, grad_scale=-0.5, seed=12, **HYPER)  # not clipped
    _check_step(s, before, 4, -0.5, seed=12)
    s.check_guards()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_everything(ctx, value):
    s = Set([300, 1000], KINDS[:4], seed=6)
    s.g[1][77] = value
    was = s.state()
    norm = torch.zeros(1, device="cuda")
    ctx.grad_norm(s.group, norm)
    ctx.adamw_step(s.group, step=2, norm=norm, max_norm=1.0, **HYPER)
    torch.cuda.synchronize()
    assert not torch.isfinite(norm).any()
    for a, b in zip(was, s.state()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_rate_and_step_from_memory_in_a_replayed_graph(ctx):
    s, t = Set(SIZES, KINDS, seed=7), Set(SIZES, KINDS, seed=7)
    lr, step = torch.empty(1, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    norm, norm2 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    how = {k: v for k, v in HYPER.items() if k != "lr"}
    lr.fill_(0.0), step.fill_(1)
    ctx.grad_norm(t.group, norm2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.grad_norm(s.group, norm)
        ctx.adamw_step(s.group, lr, step, norm=norm, max_norm=1.0, seed=5, stochastic=True, **how)
    for k in (1, 2, 30, 1001):
        lr.fill_(1e-3 * k), step.fill_(k)
        graph.replay()
        ctx.grad_norm(t.group, norm2)
        ctx.adamw_step(t.group, float(np.float32(1e-3 * k)), k, norm=norm2, max_norm=1.0, seed=5, stochastic=True, **how)
    torch.cuda.synchronize()
    ctx.poll()
    assert torch.equal(norm, norm2)
    # the corrections by repeated squaring and by pow agree to fp64 rounding, seen where fp32 rounds it
    for a, b in zip(s.state(), t.state()):
        if a.dtype in (BF, F32):
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=1e-9)
            assert (a != b).sum() <= 0.02 * a.numel()


def test_a_step_below_one_from_memory(ctx):
    import overlapped_tensor_gemm_gb300 as fo
    s = Set([300], KINDS[3:4], seed=8)
    was = s.state()
    ctx.adamw_step(s.group, 1e-3, torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    with pytest.raises(fo.FoError) as e:
        ctx.poll()
    assert e.value.status == fo.FO_ERR_RANGE and "step 0" in str(e.value)
    for a, b in zip(was, s.state()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unpack(ctx, dtype):
    s = Set(SIZES, KINDS, seed=9)
    out = [[None if k[3] == 32 else torch.full((n,), 7.0, dtype=dtype, device="cuda") for n, k in zip(s.sizes, s.kinds)]
           for _ in range(2)]
    ctx.adamw_unpack(s.group, *out)
    torch.cuda.synchronize()
    for i, n in enumerate(s.sizes):
        if s.kinds[i][3] == 32 or n == 0:
            continue
        _, _, m, v = s.values(i)
        for got, ref in zip((out[0][i], out[1][i]), (m, v)):
            err = np.abs(got.double().cpu().numpy() - ref)
            assert (err <= (HALF[dtype] + 64 * u) * np.abs(ref) + 2.0 ** -149).all(), i


def test_many_tensors_and_none(ctx):
    """1300 tensors (several launches a kind), the same bits as in groups of their own; an empty group."""
    import overlapped_tensor_gemm_gb300 as fo
    sizes = [1 + (i * 37) % 600 for i in range(1300)]
    s = Set(sizes, [KINDS[0], KINDS[1]], seed=10)
    before = [s.values(i) for i in range(len(sizes))]
    norm = torch.zeros(1, device="cuda")
    ctx.grad_norm(s.group, norm)
    ctx.adamw_step(s.group, step=7, **HYPER)
    torch.cuda.synchronize()
    want = np.sqrt(sum((g.double() ** 2).sum().item() for g in s.g))
    assert abs(norm.item() - want) <= want * 264 * u
    for i in range(0, 1300, 101):
        s.sizes, s.kinds = [sizes[i]], [s.kinds[i]] + s.kinds[1:]
        one = Set.__new__(Set)
        one.__dict__.update(sizes=[sizes[i]], kinds=[KINDS[i % 2]], **{x: [getattr(s, x)[i]] for x in
                                                                       ("w", "g", "master", "m", "v", "m_scale", "v_range")})
        _check_step(one, [before[i]], 7, 1.0)
        s.sizes = sizes
    none = fo.AdamWTensors([], [], [], [])
    ctx.grad_norm(none, norm)
    ctx.adamw_step(none, 0.1, 1)
    ctx.adamw_unpack(none, [], [])
    torch.cuda.synchronize()
    assert norm.item() == 0


def test_tensors_behind_2_32_elements(ctx):
    """One tensor of 2^32 + 1000 bf16 elements with 8-bit states: its last elements like a small tensor's."""
    import overlapped_tensor_gemm_gb300 as fo
    n = 2 ** 32 + 1000
    w = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    tail = torch.randn(1000, device="cuda").to(BF)
    w[-1000:], g[-1000:] = 1.0, tail
    m, v, scale, rng = fo.adamw_states([w], 8)
    ctx.adamw_step(fo.AdamWTensors([w], [g], m, v, m_scale=scale, v_range=rng), 0.25, 1, weight_decay=0.0)
    norm = torch.zeros(1, device="cuda")
    ctx.grad_norm(fo.AdamWTensors([w], [g], m, v, m_scale=scale, v_range=rng), norm)
    torch.cuda.synchronize()
    want = 1.0 - 0.25 * torch.sign(tail.float())  # the first step is the sign
    assert torch.allclose(w[-1000:].float(), want, atol=2.0 ** -7)
    assert (w[:1000] == 0).all() and (w[2 ** 31:2 ** 31 + 1000] == 0).all() and (m[0][:100000].view(torch.uint8) == 0).all()
    ref = tail.double().norm().item()
    assert abs(norm.item() - ref) <= ref * 264 * u


def test_stochastic_weights_are_right_in_the_mean(ctx):
    """bf16 weights of 1 that move by 2^-10 a step: rounded to the nearest they stay, at random they move on."""
    import overlapped_tensor_gemm_gb300 as fo
    n, steps = 20000, 64
    moved = []
    for stochastic in (False, True):
        w, g = torch.full((n,), 1.5, dtype=BF, device="cuda"), torch.ones(n, dtype=BF, device="cuda")
        m, v, _, _ = fo.adamw_states([w])
        group = fo.AdamWTensors([w], [g], m, v)
        for k in range(1, steps + 1):
            ctx.adamw_step(group, 2.0 ** -10, k, weight_decay=0.0, stochastic=stochastic, seed=3)
        moved.append(1.5 - w.double().mean().item())
    assert moved[0] == 0
    # each step adds at most (2^-7)^2 / 4 of variance to an element; five standard deviations of the mean
    assert abs(moved[1] - steps * 2.0 ** -10) <= 5 * (2.0 ** -8) * np.sqrt(steps / n) + 1e-6


@pytest.mark.parametrize("kinds", [KINDS[0:2], KINDS[3:5], KINDS[8:10], KINDS[10:11]],
                         ids=["32-bit", "8-bit", "32-bit, bf16", "8-bit, bf16"])
def test_long_tensors_between_short_ones(ctx, kinds):
    """Several blocks of a tensor for every warp, then another tensor's: what is loaded ahead is the right block's."""
    s = Set([2500001, 2500001, 700, 3, 1, 257, 2000256, 2000256], kinds, seed=14)
    before = [s.values(i) for i in range(len(s.sizes))]
    norm = torch.zeros(1, device="cuda")
    ctx.grad_norm(s.group, norm)
    ctx.adamw_step(s.group, step=5, stochastic=True, seed=99, norm=norm, **HYPER)
    torch.cuda.synchronize()
    s.check_guards()
    _check_step(s, before, 5, 1.0, True, 99)
    want = np.sqrt(sum((g.double() ** 2).sum().item() for g in s.g))
    assert abs(norm.item() - want) <= want * 264 * u
