"""The two ends of a training step with the projection between them, as a program would run them: Flash-AG output
projection with the vocabulary sharded over the ranks, the loss and its gradient over the logits, the projection's
backward, the gradients' norm, the update -- against fp64 autograd of the same bf16 weights, eagerly and captured.

Tolerances.  The logits are rounded to bf16 (2^-9 of each, size about 1.3), so a token's log-probability is off by
about 2^-9 * 1.3 in a 2-norm sense and a probability by as much relative: 0.004; the gradient is rounded once more
(2^-9) and summed by the projection's backward in fp32, rounded to bf16 (2^-9).  In quadrature under 0.006 relative to
the 2-norm; 0.02 is asked for."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
P, m, K, V = 2, 128, 256, 512   # ranks, tokens per rank, hidden, vocabulary per rank
HYPER = dict(beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.05)


class Model:
    def __init__(self, bits, seed):
        import overlapped_tensor_gemm_gb300 as fo
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.X = [rnd(m, K).to(BF) for _ in range(P)]
        self.master = [rnd(V, K) * 0.08 for _ in range(P)]
        self.W = [w.to(BF) for w in self.master]
        self.w_norm = 1 + 0.1 * rnd(K)        # (a parameter in 32 bits beside them)
        self.g_norm = 1e-3 * rnd(K)
        self.logits = [torch.empty((P * m, V), dtype=BF, device="cuda") for _ in range(P)]
        self.dX = [torch.empty((m, K), dtype=BF, device="cuda") for _ in range(P)]
        self.dW = [torch.empty((V, K), dtype=BF, device="cuda") for _ in range(P)]
        self.y = torch.randint(0, P * V, (P * m,), generator=g, device="cuda", dtype=torch.int32)
        self.y[::5] = -1
        self.adv, self.old, self.ref = rnd(P * m), -7 + 0.3 * rnd(P * m), -7 + 0.3 * rnd(P * m)
        self.off = torch.tensor([0, 60, 100, 190, 256], dtype=torch.int32, device="cuda")
        self.stats, self.loss, self.norm = (torch.zeros(n, device="cuda") for n in (4, 1, 1))
        params = self.W + [self.w_norm]
        self.m, self.v, self.m_scale, self.v_range = fo.adamw_states(params[:P], bits)
        m1, v1, _, _ = fo.adamw_states(params[P:])
        none = [None] * (P + 1)
        self.group = fo.AdamWTensors(params, self.dW + [self.g_norm], self.m + m1, self.v + v1,
                                     master=self.master + [None],
                                     m_scale=self.m_scale + [None] if bits == 8 else none,
                                     v_range=self.v_range + [None] if bits == 8 else none)
        self.lr, self.step = torch.full((1,), 1e-2, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")

    def forward(self, ctx):
        ctx.ag_gemm(self.X, self.W, self.logits)

    def make_loss(self, ctx, loss):
        if loss == "policy":
            ctx.policy_loss(self.logits, self.y, self.adv, self.stats, old_logp=self.old, ref_logp=self.ref,
                            dlogits=self.logits, kl_coef=0.05, entropy_coef=0.01)
        else:
            ctx.preference_loss(self.logits, self.y, self.off, self.loss, ref_logp=self.ref, dlogits=self.logits,
                                beta=0.3)

    def backward(self, ctx):
        ctx.col_linear_backward(self.X, self.W, self.logits, self.dX, self.dW)

    def update(self, ctx):
        ctx.grad_norm(self.group, self.norm)
        ctx.adamw_step(self.group, self.lr, self.step, norm=self.norm, max_norm=0.5, seed=9, **HYPER)

    def train(self, ctx, loss):
        self.forward(ctx)
        self.make_loss(ctx, loss)
        self.backward(ctx)
        self.update(ctx)

    def exact(self, loss):
        """(loss, dX, dW, norm) in 64 bits"""
        X = torch.cat(self.X).double().requires_grad_()
        W = torch.cat(self.W).double().requires_grad_()
        lp = torch.log_softmax(X @ W.T, 1)
        on = self.y >= 0
        logp = lp.gather(1, self.y.clamp(min=0).long()[:, None])[:, 0]
        if loss == "policy":
            ratio = torch.exp(logp - self.old.double())
            adv, x = self.adv.double(), self.ref.double() - logp
            per = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.05 * (torch.expm1(x) - x)
            per = per + 0.01 * (lp.exp() * lp).sum(1)
            value = per[on].mean()
        else:
            ratio = torch.where(on, logp - self.ref.double(), 0.0)
            b = self.off.tolist()
            s = [ratio[lo:hi].sum() for lo, hi in zip(b[:-1], b[1:])]
            value = -sum(torch.nn.functional.logsigmoid(0.3 * (s[i] - s[2 + i])) for i in range(2)) / 2
        dX, dW = torch.autograd.grad(value, [X, W])
        norm = torch.sqrt((dW ** 2).sum() + (self.g_norm.double() ** 2).sum())
        return value.detach(), dX, dW, norm


def _near(got, want, rel, what):
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= rel, (what, off)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_a_step_against_autograd(loss, bits):
    import overlapped_tensor_gemm_gb300 as fo
    model = Model(bits, 3)
    value, dX, dW, norm = model.exact(loss)
    was = torch.cat(model.master).double()
    with fo.Context(0) as ctx:
        model.train(ctx, loss)
        torch.cuda.synchronize()
        ctx.poll()
    got = (model.stats[0] if loss == "policy" else model.loss[0]).double()
    assert abs(got - value) <= 0.02 * abs(value) + 0.01
    _near(torch.cat(model.dX), dX, 0.02, "dX")
    _near(torch.cat(model.dW), dW, 0.02, "dW")
    assert abs(model.norm.double() - norm) <= 0.02 * norm
    # the update from the gradients that the step had: the first step of zero states
    g = torch.cat(model.dW).double() * min(1.0, 0.5 / model.norm.item())
    change = g / (g.abs() + 1e-6) + 0.05 * was
    # (a first step's root and quotient: 32 * 2^-24; the clipping factor and the master's own rounding)
    assert ((torch.cat(model.master).double() - (was - 1e-2 * change)).abs()
            <= 1e-2 * (1e-5 * change.abs() + 1e-5) + 2.0 ** -23 * was.abs()).all()
    assert torch.equal(torch.cat(model.W), torch.cat(model.master).to(BF))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_captured_losses_and_updates_are_the_eager_ones(loss, bits):
    """Loss and update as two graphs that share the context's workspaces, the ring operations between them (their
    flags carry a number of the call, so they are not replayed) eager; beside them eager steps on the same context."""
    import overlapped_tensor_gemm_gb300 as fo
    a, b, warm = Model(bits, 4), Model(bits, 4), Model(bits, 5)
    with fo.Context(0) as ctx:
        warm.train(ctx, loss)  # (workspaces are had outside the capture)
        torch.cuda.synchronize()
        graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        with torch.cuda.graph(graphs[0]):
            a.make_loss(ctx, loss)
        with torch.cuda.graph(graphs[1]):
            a.update(ctx)
        for k in range(1, 5):
            for mod in (a, b):
                mod.step.fill_(k)
                mod.lr.fill_(1e-2 / k)
            a.forward(ctx)
            graphs[0].replay()
            a.backward(ctx)
            graphs[1].replay()
            b.train(ctx, loss)
        torch.cuda.synchronize()
        ctx.poll()
    for x, y in zip(a.W + a.master + a.dX + [a.w_norm, a.norm], b.W + b.master + b.dX + [b.w_norm, b.norm]):
        assert torch.equal(x, y)
    assert not torch.equal(a.W[0], Model(bits, 4).W[0])
