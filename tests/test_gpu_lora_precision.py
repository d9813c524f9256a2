"""What the adapter calls keep of their operands, by inputs on which a lost part would show: worst-case
bounds over long sums (tests/_lora.py) leave room for it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import post_weight_quantization_17_b200 as G  # noqa: E402
from tests._lora import U32, Case, within  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    c = G.Context(1, 1, workspace_bytes=64 << 20)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T, m, d, bits, group", [(7, 128, 256, 4, 128), (100, 515, 416, 4, 128), (300, 640, 512, 3, -1),
                                                  (520, 2049, 384, 2, 128)])
def test_dx_comes_from_unrounded_weights(ctx, T, m, d, bits, group, dtype):
    """The weights keep 14 bits (bf16) or 19 (fp16) at the worst, 16 and 22 in the mean, so dX is off by
    its own rounding alone: element by element that and 2^-14 (2^-19) of the sum of magnitudes, and over
    all elements no more than the exact sum rounded is (weights rounded to 16 bits: 1.41 times that)."""
    c = Case(T, m, d, bits, group, 8, 3, dtype, "runs", 31)
    dX = torch.full_like(c.X, float("nan"))
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), None, dX=dX)
    G.gptq_sync_status(ctx)
    (want, bound), _, _ = c.backward(torch.zeros(T, 8, dtype=torch.float64, device="cuda"), False)
    kept = 2.0 ** (-14 if dtype == BF else -19)
    within(dX, want, bound + 1.01 * kept * (c.dY.double().abs() @ c.W.abs()), "dX")
    rounded = (want.to(dtype).double() - want).norm()
    assert (dX.double() - want).norm() <= 1.1 * rounded


@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("factor", [2.0 ** -22, 2.0 ** -12, 2.0 ** 8])
def test_dx_of_fp16_keeps_small_weights(ctx, T, factor):
    """Δ from some 2e-10 up (2^-22 of the usual), where an fp16 weight is far below the smallest normal number;
    the last group's Δ is another 2^20 smaller than the others'."""
    c = Case(T, 384, 320, 4, 128, 8, 2, HF, "none", 32)
    for k in range(3):
        s = factor if k < 2 else factor * 2.0 ** -20
        c.scales[:, k] *= s
        c.W[:, 128 * k:128 * (k + 1)] *= s
    dX = torch.full_like(c.X, float("nan"))
    c.dY.mul_(2.0 ** 14 if factor < 1 else 1.0)
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), None, dX=dX)
    G.gptq_sync_status(ctx)
    (want, bound), _, _ = c.backward(torch.zeros(T, 8, dtype=torch.float64, device="cuda"), False)
    within(dX, want, bound + 1.01 * 2.0 ** -19 * (c.dY.double().abs() @ c.W.abs()), "dX")
