"""Distillation: values and calls at which a row's place in memory, or another call, must not matter."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import post_weight_quantization_17_b200 as G  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = G.Context(1, 1)
    yield c
    c.close()


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("V, offset", [(1001, 0), (1001, 1), (5, 0), (5, 1), (1, 0), (200003, 1)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_infinite_and_nan_logits_anywhere_in_a_row(ctx, dt, V, offset, value):
    """NaN in the loss, in lse and in the whole gradient, wherever in a row of odd length the value stands:
    among its aligned vectors or at one of its ends."""
    at = sorted({0, V - 1, V // 2, min(3, V - 1), max(0, V - 3)})
    T, K = len(at) + 1, 1
    store = torch.randn(T * V + offset, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dt)
    z = store[offset:].view(T, V)
    for t, i in enumerate(at):
        z[t, i] = value
    val = torch.zeros(T, K, device="cuda")
    idx = torch.full((T, K), V // 3, dtype=torch.int32, device="cuda")
    loss, lse, dl = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    dz = torch.zeros_like(z)
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, dloss=dl, dlogits=dz)
    G.gptq_sync_status(ctx)
    assert loss[:-1].isnan().all() and lse[:-1].isnan().all() and dz[:-1].isnan().all()
    assert torch.isfinite(loss[-1]) and torch.isfinite(lse[-1]) and torch.isfinite(dz[-1]).all()
