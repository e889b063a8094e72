"""Policy loss: terms that do not enter the loss, and values whose exponentials leave fp32."""
import numpy as np
import pytest
import torch

from oracle import losses as ls

pytestmark = pytest.mark.gpu

F32 = torch.float32
u = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


def _rows():
    g = torch.Generator().manual_seed(3)
    z = torch.randn((6, 52), generator=g) * 2
    y = torch.randint(0, 52, (6,), generator=g, dtype=torch.int32)
    return z, y, ls.token_stats(z.double().numpy(), y.numpy())[0]


def _run(ctx, z, y, adv, old, ref, **k):
    stats, d = torch.empty(4, device="cuda"), torch.empty_like(z, device="cuda")
    vec = lambda x: None if x is None else torch.from_numpy(np.asarray(x)).float().cuda()  # noqa: E731
    ctx.policy_loss([z.cuda()], y.cuda(), vec(adv), stats, old_logp=vec(old), ref_logp=vec(ref), dlogits=[d], **k)
    torch.cuda.synchronize()
    ctx.poll()
    return stats.double().cpu().numpy(), d.double().cpu().numpy()


def _check(ctx, z, y, adv, old, ref, kl_coef=0.0, entropy_coef=0.0):
    """Against the oracle on the fp32 values of the vectors; a logp of at most 12 is off by less than 64 u,
    and each of a dozen operations adds a rounding of a number of the losses' size."""
    c64 = lambda x: None if x is None else np.asarray(x, np.float32).astype(np.float64)  # noqa: E731
    with np.errstate(over="ignore", invalid="ignore"):
        want, _, grad, a, _ = ls.policy_loss(z.double().numpy(), y.numpy(), c64(adv), c64(old), c64(ref), None,
                                             1 - float(np.float32(1) - np.float32(0.2)),
                                             float(np.float32(1) + np.float32(0.2)) - 1, kl_coef, entropy_coef)
    stats, d = _run(ctx, z, y, adv, old, ref, kl_coef=kl_coef, entropy_coef=entropy_coef)
    assert np.isfinite(stats[[0, 2, 3]]).all() and np.isfinite(d).all()
    size = 1 + np.abs(want[0]) + np.abs(a).max()
    assert (np.abs(stats[[0, 2, 3]] - want[[0, 2, 3]]) <= 128 * u * size * 12).all(), (stats, want)
    assert (np.abs(d - grad) <= 128 * u * size).all()
    return stats, want


def test_a_ratio_beyond_fp32_without_an_advantage(ctx):
    """exp(100) times an advantage of 0 is 0."""
    z, y, lp = _rows()
    old = lp + 0.1
    old[2] = lp[2] - 100.0
    adv = np.array([1.0, -0.5, 0.0, 0.25, 0.0, 2.0])
    _check(ctx, z, y, adv, old, None)


def test_a_ratio_beyond_fp32_is_clipped(ctx):
    z, y, lp = _rows()
    old = lp + 0.1
    old[2] = lp[2] - 100.0
    _check(ctx, z, y, np.array([1.0, -0.5, 0.75, 0.25, 0.0, 2.0]), old, None)


def test_a_reference_that_is_only_watched(ctx):
    """Without a coefficient the KL term is a statistic: where it leaves fp32, loss and gradient do not follow."""
    z, y, lp = _rows()
    ref = lp - 0.2
    ref[1] = lp[1] + 100.0
    adv = np.array([1.0, -0.5, 0.3, 0.25, 0.1, 2.0])
    stats, _ = _check(ctx, z, y, adv, lp + 0.05, ref)
    assert stats[1] == np.inf
    ref[1] = lp[1] - 0.2
    stats, want = _check(ctx, z, y, adv, lp + 0.05, ref)
    assert abs(stats[1] - want[1]) <= 128 * u
