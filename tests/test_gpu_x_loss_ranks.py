"""Losses whose first rank has no columns: which rank comes first says nothing about whether a gradient is
wanted.  Tolerances are those of the losses' other tests."""
import pytest
import torch

import test_gpu_u_losses as losses

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(7, [0, 8, 3, 9]), (5, [0, 0, 40]), (33, [0, 257, 0]), (6, [0, 3000, 5]), (130, [0, 96, 0, 33])]
IDS = ["x".join(map(str, [m] + c)) for m, c in SHAPES]
ALIKE = [(BF, BF), (F32, F32)]
MIXED = [(BF, F32), (F32, BF)]


@pytest.fixture(scope="module")
def ctx():
    import overlapped_tensor_gemm_gb300 as fo
    c = fo.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_token_logprobs(ctx, shape, dtype):
    losses.test_token_logprobs(ctx, shape, dtype)


@pytest.mark.parametrize("types", ALIKE + MIXED, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_token_logprobs_backward(ctx, shape, types):
    losses.test_token_logprobs_backward(ctx, shape, types)


@pytest.mark.parametrize("types", ALIKE + MIXED, ids=str)
@pytest.mark.parametrize("how", losses.POLICY, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_policy_loss(ctx, shape, how, types):
    losses.test_policy_loss(ctx, shape, how, types)


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("how", [(0.0, False, 0.0, True), (0.1, True, 0.25, True)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_preference_loss(ctx, shape, how, kind):
    losses.test_preference_loss(ctx, shape, how, kind)


@pytest.mark.parametrize("types", ALIKE, ids=str)
def test_rows_that_do_not_fit_shared_memory(ctx, types, monkeypatch):
    """Vocabularies of a million behind an empty rank: rows are read twice."""
    rows = losses.Rows
    monkeypatch.setattr(losses, "Rows", lambda m, cols, **k: rows(m, [0] + cols, **k))
    losses.test_rows_that_do_not_fit_shared_memory(ctx, types, 5)
