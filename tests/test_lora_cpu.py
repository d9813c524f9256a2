"""Host logic of the adapter and distillation calls: argument refusals that need no device, and the
workspace size.  No GPU needed."""
import types

import pytest
import torch

import post_weight_quantization_17_b200 as G


def test_null_context_is_an_argument_error():
    L = G._lib
    assert L.gptq_lora_matmul(None, None, 0, 1, 32, None, 1, 4, 128, None, 1, None, None, None, 1, 8, None,
                              None, None, None, 0, None) == G.GPTQ_ERR_ARG
    assert L.gptq_lora_backward(None, None, None, 0, 1, 32, None, 1, 4, 128, None, 1, None, None, None, 1, 8,
                                None, None, None, None, None, None, None, 0) == G.GPTQ_ERR_ARG
    assert L.gptq_distill_topk(None, None, 0, 1, 8, 8, None, None, 1, 1.0, None, None, None, None, None, None,
                               0) == G.GPTQ_ERR_ARG
    assert L.gptq_distill_topk_backward(None, None, 0, 1, 8, 8, None, None, 1, 1.0, None, None, None, None,
                                        None, 0) == G.GPTQ_ERR_ARG


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_workspace_covers_the_low_rank_products(dtype):
    small = G.gptq_lora_workspace_bytes(0, 1, 1, 4, 1, 1, dtype)
    assert small >= 256
    for T, m, d, bits, n, R in ((1, 4096, 4096, 4, 8, 16), (4096, 11008, 4096, 4, 8, 64), (7, 33, 100, 3, 2, 5)):
        ws = G.gptq_lora_workspace_bytes(T, m, d, bits, n, R, dtype)
        assert ws >= 4 * T * R + 256
        assert ws <= G.gptq_lora_workspace_bytes(2 * T + 64, m, d, bits, n, R, dtype)


def test_workspace_of_refused_sizes_is_the_status_block():
    for bad in ((-1, 8, 8, 4, 1, 1), (1, 0, 8, 4, 1, 1), (1, 8, 0, 4, 1, 1), (1, 8, 8, 0, 1, 1), (1, 8, 8, 9, 1, 1),
                (1, 8, 8, 4, 0, 1), (1, 8, 8, 4, 1, 0), (1, 8, 8, 4, 1, 1025), (1, 8, 8, 4, 65536, 1),
                (2 ** 40, 8, 8, 4, 1, 1), (1, 2 ** 40, 8, 4, 1, 1)):
        assert G.gptq_lora_workspace_bytes(*bad) == 256


def test_host_tensors_are_refused():
    """The binding refuses tensors that are not on the context's device before it calls the library."""
    ctx = types.SimpleNamespace(device=torch.device("cuda", 0), handle=None)
    z = torch.zeros
    layer = (z(4, 4, dtype=torch.int32), 32, 4, -1, z(4, 1), z(4, 1, dtype=torch.int32), z(2, dtype=torch.int32),
             z(1, 8, 32), z(1, 8, 4), z(1))
    with pytest.raises(ValueError, match="packed"):
        G.gptq_lora_matmul(ctx, z(2, 32), *layer, z(2, 4))
    with pytest.raises(ValueError, match="packed"):
        G.gptq_lora_backward(ctx, z(2, 4), z(2, 32), *layer, z(2, 8), dX=z(2, 32))
    with pytest.raises(ValueError, match="logits"):
        G.gptq_distill_topk(ctx, z(2, 9), z(2, 3), z(2, 3, dtype=torch.int32), 1.0, z(2), z(2))
    with pytest.raises(ValueError, match="go together"):
        G.gptq_distill_topk(ctx, z(2, 9), z(2, 3), z(2, 3, dtype=torch.int32), 1.0, z(2), z(2), dloss=z(2))
