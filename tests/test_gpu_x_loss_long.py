"""Losses of so many rows that a team of CTAs takes more than 64 of them: the second and third batch of targets
and inputs, and every barrier, ring slot and place for the warps' parts used again and again, against the fp64
oracle on every row.  Tolerances are those of the losses' other tests."""
import functools

import pytest
import torch

import test_gpu_u_losses as losses

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
MANY = (25000, [70, 33])       # 82 rows for each of 304 teams, 164 for each of 152
WIDE = (5200, [9000, 0, 7601])   # clusters: over 64 rows a team, one in twenty of them counted


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_token_logprobs(ctx, dtype):
    losses.test_token_logprobs(ctx, MANY, dtype)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
def test_token_logprobs_backward(ctx, types):
    losses.test_token_logprobs_backward(ctx, MANY, types)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("how", losses.POLICY, ids=str)
def test_policy_loss(ctx, how, types):
    losses.test_policy_loss(ctx, MANY, how, types)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge"])
@pytest.mark.parametrize("how", [(0.0, False, 0.0, True), (0.1, True, 0.25, True)], ids=str)
def test_preference_loss(ctx, how, kind):
    losses.test_preference_loss(ctx, MANY, how, kind)


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF)], ids=str)
def test_policy_loss_by_clusters(ctx, types, monkeypatch):
    monkeypatch.setattr(losses, "Rows", functools.partial(losses.Rows, masked=0.95))
    losses.test_policy_loss(ctx, WIDE, losses.POLICY[1], types)


def test_policy_loss_by_clusters_bf16(ctx, monkeypatch):
    monkeypatch.setattr(losses, "Rows", functools.partial(losses.Rows, masked=0.95))
    losses.test_policy_loss(ctx, (2600, [20000, 13001]), losses.POLICY[0], (BF, BF))
