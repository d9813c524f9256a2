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


# The adapter terms, with a base product of zero (Δ = 0): U and G pass the tensor cores as two tf32 numbers,
# off by 2^-22 of each at most.  A sum on them is off by no more than 2 units of fp32 a term (half of it for the
# sums' own additions, which round towards zero), so what a lost low part leaves, up to 2^-11 of a term and
# 2^-12.8 in the mean, lies far outside.
PARTS = 1.01 * 2.0 ** -22


def _without_low_part(u):
    """u rounded to tf32: the mistake that the bounds have to show, planted in the formula."""
    bits = u.float().view(torch.int32)
    return ((bits + 0x1000) & ~0x1FFF).view(torch.float32).double()


def _outside(got, want, bound):
    return float(((got - want).abs() / bound.clamp_min(1e-300)).max()) > 1.0


def _adapters_only(T, m, d, R, n, dtype, pattern, seed):
    c = Case(T, m, d, 4, 128, R, n, dtype, pattern, seed)
    c.scales.zero_()
    c.W.zero_()
    return c


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T, m, d, R, n", [(7, 300, 256, 16, 3), (40, 128, 1024, 16, 3), (300, 2048, 256, 16, 3),
                                           (300, 2048, 256, 64, 2)])
def test_adapter_term_of_y(ctx, T, m, d, R, n, dtype):
    c = _adapters_only(T, m, d, R, n, dtype, "mixed", 33)
    Y, U = torch.empty(T, m, device="cuda"), torch.empty(T, R, device="cuda")
    G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y, U=U)
    G.gptq_sync_status(ctx)
    want = c.up(U, c.B)
    bound = (PARTS + 2 * (R + 8) * U32) * c.up(U.abs(), c.B.abs())
    within(Y, want, bound, "Y")
    assert _outside(c.up(_without_low_part(U), c.B), want, bound)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T, R, n", [(300, 16, 1), (300, 40, 2), (2000, 16, 1)])
def test_adapter_gradients_of_few_outputs(ctx, T, R, n, dtype):
    """m = 8, so that G is good to its last bits; dB takes its U from the caller."""
    m, d = 8, 512
    c = _adapters_only(T, m, d, R, n, dtype, "mixed", 34)
    U = c.low(c.X, c.A)[0].float()
    dA, dB = torch.empty(n, R, d, device="cuda"), torch.empty(n, R, m, device="cuda")
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dA=dA, dB=dB)
    G.gptq_sync_status(ctx)
    g, gmag = c.low(c.dY, c.B)
    # runs of 16 additions that round towards zero, then IEEE additions of the runs, warps and CTAs
    sums = (2 * 16 + T / 64 + 16) * U32
    da, da_bound = c.outer(g, c.X), 2 * (m + 8) * U32 * c.outer(gmag, c.X.abs()) + (PARTS + sums) * c.outer(g.abs(), c.X.abs())
    db, db_bound = c.outer(U, c.dY), (PARTS + sums) * c.outer(U.abs(), c.dY.abs())
    within(dA, da, da_bound, "dA")
    within(dB, db, db_bound, "dB")
    assert _outside(c.outer(_without_low_part(g), c.X), da, da_bound)
    assert _outside(c.outer(_without_low_part(U), c.dY), db, db_bound)


def test_adapter_term_of_dx(ctx):
    """fp16, whose rounding is small enough: over all elements dX is as far from the formula as the formula
    rounded to fp16 (a G without its low part: 1.4 times that)."""
    T, m, d, R = 300, 256, 2048, 16
    c = _adapters_only(T, m, d, R, 3, HF, "mixed", 35)
    dX = torch.empty_like(c.X)
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), None, dX=dX)
    G.gptq_sync_status(ctx)
    g = c.low(c.dY, c.B)[0]
    want = c.up(g, c.A)
    rounded = (want.to(HF).double() - want).norm()
    assert (dX.double() - want).norm() <= 1.1 * rounded
    assert (c.up(_without_low_part(g), c.A).to(HF).double() - want).norm() > 1.1 * rounded


def test_long_sums_do_not_drift(ctx):
    """Positive terms, so that additions which round towards zero all err one way: a run of k of them loses
    half of k units in the last place on average, at most 2^-23 each, of a sum that is half its end.  U: runs
    of 512 features are 32 additions, 32 / 2 · 2^-23; dB: runs of 64 tokens are 16, with their two parts'
    halves; what joins the runs rounds to nearest.  In one run, 49152 features over 16 warps would be 192
    additions and 4096 tokens over 4 warps 256."""
    T, d, m, R = 2400, 49152, 8, 16
    big = G.Context(1, 1, workspace_bytes=G.gptq_lora_workspace_bytes(T, m, d, 4, 1, R, BF))
    try:
        c = _adapters_only(T, m, 128, R, 1, BF, "one", 36)
        c.d = d
        g = torch.Generator(device="cuda").manual_seed(5)
        c.X = torch.rand(T, d, device="cuda", generator=g).to(BF)
        c.A = torch.rand(1, R, d, device="cuda", generator=g).to(BF)
        c.packed = torch.zeros(m, d // 8, dtype=torch.int32, device="cuda")
        c.scales, c.zeros = torch.zeros(m, d // 128, device="cuda"), torch.zeros(m, d // 128, dtype=torch.int32, device="cuda")
        Y, U = torch.empty(T, m, device="cuda"), torch.empty(T, R, device="cuda")
        G.gptq_lora_matmul(big, c.X, *c.layer(), Y, U=U)
        G.gptq_sync_status(big)
        want = c.low(c.X, c.A)[0]
        drift = float((U.double() / want - 1).mean())
        assert abs(drift) <= 17 * 2.0 ** -23, drift
        del c, Y
    finally:
        big.close()
    T, d, m = 4096, 8, 148 * 128      # columns for a CTA on every SM: each takes all the tokens
    c = _adapters_only(T, 128, d, R, 1, BF, "one", 37)
    c.m = m
    c.dY = torch.rand(T, m, device="cuda", generator=g).to(BF)
    c.B = torch.zeros(1, R, m, dtype=BF, device="cuda")
    c.packed = torch.zeros(m, 1, dtype=torch.int32, device="cuda")
    c.scales, c.zeros = torch.zeros(m, 1, device="cuda"), torch.zeros(m, 1, dtype=torch.int32, device="cuda")
    U = torch.rand(T, R, device="cuda", generator=g)
    dB = torch.empty(1, R, m, device="cuda")
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), U, dB=dB)
    G.gptq_sync_status(ctx)
    drift = float((dB.double() / c.outer(U, c.dY) - 1).mean())
    assert abs(drift) <= 9 * 2.0 ** -23, drift
