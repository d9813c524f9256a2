"""The adapter calls where their documentation allows more than a plain training step or a decoding batch
shows: parts of a backward pass, values without a number, calls side by side."""
import ctypes

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


def _same_where_not_finite(got, want, what):
    want = want.to(torch.float64)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN elsewhere"
    inf = want.isinf()
    assert torch.equal(got.double()[inf], want[inf]), f"{what}: other infinities"
    assert torch.isfinite(got[torch.isfinite(want)]).all(), f"{what}: non-finite elsewhere"


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [5, 40, 150, 300])
@pytest.mark.parametrize("where", ["X", "A", "B"])
def test_an_infinity_is_what_the_formula_makes_of_it(ctx, dtype, T, where):
    c = Case(T, 200, 256, 4, 128, 8, 3, dtype, "mixed", 42)
    c.adapter[:3] = torch.arange(3, dtype=torch.int32)
    t = {"X": c.X, "A": c.A[1], "B": c.B[1]}[where]
    t[1, 7] = -torch.inf
    Y, U = torch.zeros(T, 200, device="cuda"), torch.zeros(T, 8, device="cuda")
    G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y, U=U)
    G.gptq_sync_status(ctx)
    y, _, u, _ = c.forward(F32)
    _same_where_not_finite(U, u, "U")
    _same_where_not_finite(Y, y, "Y")


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [5, 40, 150, 300])
@pytest.mark.parametrize("where", ["X", "dY", "A", "B", "U"])
def test_an_infinity_in_the_backward_pass(ctx, dtype, T, where):
    c = Case(T, 200, 256, 4, 128, 8, 3, dtype, "mixed", 43)
    c.adapter[:3] = torch.arange(3, dtype=torch.int32)
    U = c.low(c.X, c.A)[0].float()
    t = {"X": c.X, "dY": c.dY, "A": c.A[1], "B": c.B[1], "U": U}[where]
    t[1, 7] = -torch.inf
    dX = torch.zeros_like(c.X)
    dA, dB = torch.zeros(3, 8, 256, device="cuda"), torch.zeros(3, 8, 200, device="cuda")
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dX=dX, dA=dA, dB=dB)
    G.gptq_sync_status(ctx)
    (dx, _), (da, _), (db, _) = c.backward(U.double(), False)
    _same_where_not_finite(dX, dx, "dX")
    _same_where_not_finite(dA, da, "dA")
    _same_where_not_finite(dB, db, "dB")


@pytest.mark.parametrize("T, m, d, R", [(1, 128, 8192, 8), (24, 640, 4096, 16), (33, 128, 8192, 8), (75, 841, 768, 16),
                                        (110, 1408, 1408, 16), (63, 1462, 1536, 16), (200, 640, 4096, 16), (500, 256, 4096, 8)])
def test_equal_bits_from_any_workspace_that_covers_the_call(T, m, d, R):
    c = Case(T, m, d, 4, 128, R, 3, BF, "mixed", 44)
    asked = G.gptq_lora_workspace_bytes(T, m, d, 4, 3, R, BF)
    got = []
    for more in (0, 1 << 20, 256 << 20):
        ctx = G.Context(1, 1, workspace_bytes=asked + more)
        if not more:   # no more than was asked for, whatever the context would have made of it
            ctx.close()
            ctx.workspace, ctx.handle = torch.empty(asked, dtype=torch.uint8, device="cuda"), ctypes.c_void_p()
            assert G._lib.gptq_create(ctypes.byref(ctx.handle), ctypes.c_void_p(ctx.stream.cuda_stream),
                                      ctypes.c_void_p(ctx.workspace.data_ptr()), asked) == G.GPTQ_OK
        try:
            Y, U, dX = torch.empty(T, m, device="cuda"), torch.empty(T, R, device="cuda"), torch.empty_like(c.X)
            dA, dB = torch.empty(3, R, d, device="cuda"), torch.empty(3, R, m, device="cuda")
            G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y, U=U)
            G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dX=dX, dA=dA, dB=dB)
            G.gptq_sync_status(ctx)
            got.append((Y, U, dX, dA, dB))
        finally:
            ctx.close()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def _refused(call):
    with pytest.raises(G.GPTQError) as e:
        call()
    assert e.value.code == G.GPTQ_ERR_ARG and "overlaps" in str(e.value)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_overlapping_outputs_are_refused(ctx, dtype):
    c = Case(6, 128, 128, 4, 128, 8, 2, dtype, "mixed", 45)
    Y, U = torch.zeros(6, 128, dtype=dtype, device="cuda"), torch.zeros(6, 8, device="cuda")
    dA, dB = torch.zeros(2, 8, 128, device="cuda"), torch.zeros(2, 8, 128, device="cuda")
    _refused(lambda: G.gptq_lora_matmul(ctx, c.X, *c.layer(), c.X))
    _refused(lambda: G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y, U=Y.view(-1)[-48 * (2 if dtype == BF else 1):].view(F32).view(6, 8)))
    _refused(lambda: G.gptq_lora_matmul(ctx, c.X, *c.layer(), c.B.view(-1)[:6 * 128].view(6, 128)))
    back = lambda X, U, **out: G.gptq_lora_backward(ctx, c.dY, X, *c.layer(), U, **out)  # noqa: E731
    _refused(lambda: back(c.X, U, dX=c.dY))
    _refused(lambda: back(c.X, U, dX=c.X, dA=dA))
    _refused(lambda: back(c.X, U, dA=dA, dB=dA))
    _refused(lambda: back(c.X, dB.view(-1)[40:88].view(6, 8), dB=dB))
    rows = torch.zeros(12, 128, dtype=dtype, device="cuda")     # beside one another is fine
    rows[6:] = c.X
    G.gptq_lora_matmul(ctx, rows[6:], *c.layer(), rows[:6], U=U)
    Y2 = torch.zeros(6, 128, dtype=dtype, device="cuda")
    G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y2)
    G.gptq_sync_status(ctx)
    assert torch.equal(rows[:6], Y2)
    want = torch.zeros_like(c.X)
    back(None, U, dX=want, dB=dB)
    back(c.X, U, dX=c.X, dB=dB)                                 # X is not read without dA
    G.gptq_sync_status(ctx)
    assert torch.equal(c.X, want)


def test_stage_times_fit_the_arrays_of_older_programs():
    """gptq_timing_read fills the 13 entries that it always has; newer stages count under the last of them."""
    c, own = Case(80, 128, 256, 4, 128, 8, 2, BF, "runs", 46), G.Context(1, 1, workspace_bytes=32 << 20)
    Y = torch.empty(80, 128, device="cuda")
    n, other = len(G.STAGES), G.STAGES.index("other")
    try:
        G.gptq_timing_enable(own, True)
        seen = {}
        for name in ("gptq_timing_read", "gptq_timing_read_stages"):
            G.gptq_lora_matmul(own, c.X, *c.layer(), Y)
            ms, k = (ctypes.c_double * (n + 3))(*[-7.0] * (n + 3)), (ctypes.c_int64 * (n + 3))(*[-7] * (n + 3))
            args = (own.handle, ms, k) if name == "gptq_timing_read" else (own.handle, n, ms, k)
            assert getattr(G._lib, name)(*args) == G.GPTQ_OK
            seen[name] = list(k)
            end = 13 if name == "gptq_timing_read" else n
            assert all(v == -7.0 for v in ms[end:]) and all(v == -7 for v in k[end:])
        assert seen["gptq_timing_read"][other] == seen["gptq_timing_read_stages"][G.STAGES.index("lora")] > 0
        short = (ctypes.c_double * 1)(), (ctypes.c_int64 * 1)()
        assert G._lib.gptq_timing_read_stages(own.handle, 1, *short) == G.GPTQ_ERR_ARG
    finally:
        own.close()


@pytest.mark.parametrize("T", [20, 300])
def test_captured_fp16_backward(T):
    """The largest Δ of every column group is found anew in each replay: with smaller scales, too."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = Case(T, 256, 384, 4, 128, 8, 3, HF, "mixed", 47)
    ctx = G.Context(1, 1, workspace_bytes=32 << 20, stream=s)
    U = c.low(c.X, c.A)[0].float()
    dX, dA = torch.empty_like(c.X), torch.empty(3, 8, 384, device="cuda")
    torch.cuda.synchronize()
    step = lambda: G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dX=dX, dA=dA)  # noqa: E731
    try:
        with torch.cuda.stream(s):
            step()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            for factor in (1.0, 2.0 ** -12, 2.0 ** 18):
                c.scales.mul_(factor)
                step()
                want = dX.clone(), dA.clone()
                dX.zero_(), dA.zero_()
                graph.replay()
                s.synchronize()
                assert torch.equal(dX, want[0]) and torch.equal(dA, want[1])
        G.gptq_sync_status(ctx)
    finally:
        torch.cuda.synchronize()
        ctx.close()


def test_fp32_gradients_may_be_added_to_the_adapters_themselves(ctx):
    c = Case(40, 96, 128, 4, 128, 8, 2, F32, "mixed", 48)
    U = c.low(c.X, c.A)[0].float()
    dA, dB = torch.empty_like(c.A), torch.empty_like(c.B)
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dA=dA, dB=dB)
    A, B = c.A + dA, c.B + dB
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dA=c.A, dB=c.B, accumulate=True)
    G.gptq_sync_status(ctx)
    assert torch.equal(c.A, A) and torch.equal(c.B, B)
