"""The adapter calls where their documentation allows more than a plain training step or a decoding batch
shows: parts of a backward pass, values without a number, calls side by side."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import post_weight_quantization_17_b200 as G  # noqa: E402
from tests._lora import Case  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = G.Context(1, 1, workspace_bytes=64 << 20)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("part", ["dX", "dA", "dB"])
@pytest.mark.parametrize("bad", [3, -2, 2 ** 31 - 1])
def test_bad_ids_are_reported_by_every_gradient_alone(ctx, dtype, part, bad):
    c = Case(300, 70, 96, 4, -1, 5, 3, dtype, "mixed", 41)
    c.adapter[257] = bad
    out = {"dX": torch.empty_like(c.X), "dA": torch.empty(3, 5, 96, device="cuda"),
           "dB": torch.empty(3, 5, 70, device="cuda")}[part]
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), torch.zeros(300, 5, device="cuda"), **{part: out})
    with pytest.raises(G.GPTQError) as e:
        G.gptq_sync_status(ctx)
    assert e.value.code == G.GPTQ_ERR_ARG
