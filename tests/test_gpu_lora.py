"""The packed layer with low-rank adapters (gptq_lora_matmul, gptq_lora_backward) against the
formulas in fp64, with the bounds that tests/_lora.py derives."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

import post_weight_quantization_17_b200 as G  # noqa: E402
from tests._lora import Case, within  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# T, m, d, bits, group, rank, adapters, dtype, Y, pattern, more
SHAPES = {
    "one_token": (1, 128, 256, 4, 128, 16, 1, BF, BF, "one", {}),
    "one_of_each": (1, 1, 1, 1, -1, 1, 1, F32, F32, "one", {}),
    "decode_mixed": (7, 300, 512, 4, 128, 16, 5, BF, BF, "mixed", {}),
    "decode_f16_odd_rank": (16, 257, 1056, 4, 128, 13, 3, HF, F32, "mixed", {}),
    "decode_none": (9, 129, 384, 4, -1, 8, 2, BF, F32, "none", {}),
    "decode_3bit": (5, 200, 640, 3, 128, 4, 3, HF, HF, "mixed", {}),
    "decode_2bit_g256": (31, 130, 768, 2, 256, 33, 4, BF, BF, "runs", {}),
    "decode_1bit": (3, 64, 256, 1, 128, 8, 2, BF, F32, "mixed", {}),
    "rows_of_odd_length": (6, 77, 333, 4, 128, 8, 3, BF, F32, "mixed", {}),
    "off_16_byte_boundaries": (19, 96, 256, 4, 128, 8, 2, HF, HF, "runs", {"offset": 3}),
    "t33": (33, 260, 512, 4, 128, 16, 4, BF, BF, "mixed", {}),
    "t64": (64, 128, 1024, 4, 128, 64, 9, HF, F32, "mixed", {}),
    "t100_ragged": (100, 515, 416, 4, 128, 24, 3, BF, F32, "runs", {}),
    "t257_many_adapters": (257, 384, 512, 4, 128, 16, 40, BF, BF, "mixed", {}),
    "t300_rank96": (300, 256, 640, 3, -1, 96, 2, HF, HF, "runs", {}),
    "t520_one": (520, 1024, 768, 4, 256, 32, 1, BF, F32, "one", {}),
    "t300_odd_length": (300, 131, 333, 4, 128, 12, 3, BF, BF, "runs", {}),
    "t640_m_odd": (640, 2049, 512, 2, 128, 16, 4, HF, HF, "runs", {"offset": 1}),
    "rank_200": (40, 128, 256, 4, 128, 200, 2, BF, BF, "mixed", {}),
    "t300_300_adapters": (300, 128, 256, 4, 128, 8, 300, BF, F32, "mixed", {}),
    "t8300_many_tokens": (8300, 40, 128, 4, 128, 4, 3, BF, BF, "mixed", {}),
    "t2500_rank40": (2500, 68, 256, 4, 128, 40, 3, HF, HF, "runs", {}),
    "t40_one_row_of_8": (40, 1, 8, 4, 128, 3, 2, HF, F32, "mixed", {}),
    "t40_one_column": (40, 9, 1, 4, -1, 2, 2, BF, BF, "mixed", {}),
    "t24": (24, 200, 384, 4, 128, 16, 24, HF, HF, "mixed", {}),
    "t32_fc2_like": (32, 256, 6144, 4, 128, 32, 8, BF, BF, "mixed", {}),
    "t129_wide_grid": (129, 300, 8192, 4, 128, 16, 2, BF, F32, "runs", {}),
    "any_fp32": (11, 70, 130, 4, 128, 8, 3, F32, F32, "mixed", {}),
    "any_8bit": (9, 65, 96, 8, -1, 5, 2, BF, BF, "mixed", {}),
    "any_g32": (12, 80, 200, 4, 32, 8, 2, HF, F32, "runs", {}),
    "any_group_id": (10, 64, 256, 4, 64, 8, 2, BF, BF, "mixed", {"gid": True}),
}


@pytest.fixture(scope="module")
def ctx():
    c = G.Context(1, 1, workspace_bytes=64 << 20)
    yield c
    c.close()


def _case(name, seed=3):
    T, m, d, bits, group, R, n, dt, yt, pattern, more = SHAPES[name]
    return Case(T, m, d, bits, group, R, n, dt, pattern, seed, **more), yt


def _tensor_path(c):
    return c.dtype != F32 and c.bits <= 4 and c.gid is None and (c.group == -1 or c.group % 128 == 0)


def _guarded(shape, dtype):
    """A tensor in the middle of a larger one, and the check that only it was written."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    out = buf[32:32 + n].view(shape)
    out.fill_(float("nan"))
    return out, lambda: bool((buf[:32] == 7).all() and (buf[32 + n:] == 7).all())


def _forward(ctx, c, yt, keep_u=True):
    Y, fine = _guarded((c.T, c.m), yt)
    U = _guarded((c.T, c.R), F32)[0] if keep_u else None
    G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y, group_id=c.group_id, U=U)
    G.gptq_sync_status(ctx)
    assert fine(), "written outside Y"
    return Y, U


def _backward(ctx, c, U, **kw):
    (dX, f1), (dA, f2), (dB, f3) = (_guarded((c.T, c.d), c.dtype), _guarded((c.n, c.R, c.d), F32),
                                    _guarded((c.n, c.R, c.m), F32))
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U, dX=dX, dA=dA, dB=dB, group_id=c.group_id, **kw)
    G.gptq_sync_status(ctx)
    assert f1() and f2() and f3(), "written outside the gradients"
    return dX, dA, dB


@pytest.mark.parametrize("name", SHAPES)
def test_forward(ctx, name):
    c, yt = _case(name)
    Y, U = _forward(ctx, c, yt)
    want, bound, u, ubound = c.forward(yt)
    within(U, u, ubound, "U")
    within(Y, want, bound, "Y")
    again, _ = _forward(ctx, c, yt, keep_u=False)     # U in the workspace
    assert torch.equal(Y, again)


@pytest.mark.parametrize("name", SHAPES)
def test_backward(ctx, name):
    c, _ = _case(name, 4)
    U = c.low(c.X, c.A)[0].float()
    got = _backward(ctx, c, U)
    want = c.backward(U.double(), _tensor_path(c))
    for what, g, (w, b) in zip(("dX", "dA", "dB"), got, want):
        within(g, w, b, what)
    for a, b in zip(got, _backward(ctx, c, U)):
        assert torch.equal(a, b), "two calls differ"


def test_backward_in_parts_and_accumulating(ctx):
    c, _ = _case("t100_ragged", 5)
    U = c.low(c.X, c.A)[0].float()
    dX, dA, dB = _backward(ctx, c, U)
    only = torch.full_like(dX, float("nan"))
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), None, dX=only)
    assert torch.equal(only, dX)
    acc_a, acc_b = torch.ones_like(dA), torch.ones_like(dB)
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), None, dA=acc_a, accumulate=True)
    G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), U, dB=acc_b, accumulate=True)
    assert torch.equal(acc_a, 1.0 + dA) and torch.equal(acc_b, 1.0 + dB)
    G.gptq_sync_status(ctx)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_against_differences(ctx, dtype):
    """Y is linear in A and in B alone, so L(A + E) - L(A - E) = 2 <dA, E> for L = <Y, dY> without a
    truncation error: what is left is the rounding of the two losses (fp32 Y), and of A ± E, which
    is exact here (E moves A by steps of its own type on a grid of 1/64)."""
    c = Case(24, 160, 256, 4, 128, 8, 2, dtype, "mixed", 6)
    for w in (c.A, c.B):
        w.copy_((w.float() * 64).round() / 64)
    Y, U = _forward(ctx, c, F32)
    _, dA, dB = _backward(ctx, c, U)
    g = torch.Generator(device="cuda").manual_seed(1)
    for w, grad in ((c.A, dA), (c.B, dB)):
        E = torch.randint(-1, 2, w.shape, generator=g, device="cuda").float() / 64
        kept, loss = w.clone(), []
        for sign in (1, -1):
            w.copy_(kept.float() + sign * E)
            y, yb, _, _ = c.forward(F32)
            loss.append(((_forward(ctx, c, F32)[0].double() * c.dY.double()).sum(),
                         (yb * c.dY.double().abs()).sum()))
        w.copy_(kept)
        diff = loss[0][0] - loss[1][0]
        dot = (grad.double() * E.double()).sum()
        (_, _), (_, ab), (_, bb) = c.backward(U.double(), True)
        slack = loss[0][1] + loss[1][1] + 2 * ((ab if w is c.A else bb) * E.double().abs()).sum()
        # dB was formed from the rounded U: 2 <(U - u)ᵀ dY, E>
        slack = slack + 2 * (c.outer(c.forward(F32)[3], c.dY.abs()) * E.double().abs()).sum() \
            if w is c.B else slack
        assert abs(float(diff - 2 * dot)) <= float(slack)


@pytest.mark.parametrize("T", [6, 150])
def test_other_requests_do_not_leak(ctx, T):
    """A token's NaN, an adapter's NaN and infinities stay with that token and that adapter."""
    c = Case(T, 300, 512, 4, 128, 16, 4, BF, "mixed", 8)
    c.adapter[:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    Y, U = _forward(ctx, c, F32)
    grads = _backward(ctx, c, U)
    c.X[1, 5] = float("nan")
    c.dY[1, 7] = float("inf")
    c.A[2] = float("nan")
    c.B[3, 1] = float("inf")
    Y2, U2 = _guarded((c.T, c.m), F32)[0], torch.zeros(c.T, c.R, device="cuda")
    G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y2, U=U2)
    clean = ((c.adapter != 2) & (c.adapter != 3)).nonzero()[:, 0]
    clean = clean[clean != 1]
    assert torch.equal(Y2[clean], Y[clean]) and torch.equal(U2[clean], U[clean])
    assert torch.isnan(Y2[1]).all() and torch.isnan(Y2[c.adapter == 2]).all()
    dX, dA, dB = (torch.zeros_like(g) for g in grads)
    G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), U2, dX=dX, dA=dA, dB=dB)
    assert torch.equal(dX[clean], grads[0][clean])
    assert torch.equal(dA[0], grads[1][0]) and torch.equal(dB[0], grads[2][0])
    assert not torch.isfinite(dX[1]).any() or not torch.isfinite(dX[1]).all()
    G.gptq_sync_status(ctx)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements of Y and of dY: every 997th token against the formulas."""
    T, m, d, R, n = 66000, 33000, 64, 4, 3
    assert T * m > 2 ** 31
    c = Case(8, m, d, 4, -1, R, n, BF, "mixed", 12)
    g = torch.Generator(device="cuda").manual_seed(3)
    c.T = T
    c.X = torch.randn(T, d, device="cuda", generator=g).to(BF)
    c.adapter = torch.randint(-1, n, (T,), device="cuda", generator=g, dtype=torch.int32)
    big = G.Context(1, 1, workspace_bytes=G.gptq_lora_workspace_bytes(T, m, d, 4, n, R, BF))
    try:
        Y, U = torch.empty(T, m, dtype=BF, device="cuda"), torch.empty(T, R, device="cuda")
        G.gptq_lora_matmul(big, c.X, *c.layer(), Y, U=U)
        dX = torch.empty_like(c.X)
        G.gptq_lora_backward(big, Y, c.X, *c.layer(), U, dX=dX)
        G.gptq_sync_status(big)
        rows = torch.arange(T - 1, 0, -997, device="cuda")
        few = Case.__new__(Case)
        few.__dict__.update(c.__dict__)
        few.T, few.X, few.dY, few.adapter = len(rows), c.X[rows], Y[rows], c.adapter[rows]
        want, bound, u, ubound = few.forward(BF)
        within(U[rows], u, ubound, "U")
        within(Y[rows], want, bound, "Y")
        dx, dx_bound = few.backward(u, True)[0]
        within(dX[rows], dx, dx_bound, "dX")
    finally:
        big.close()


def test_empty_batch(ctx):
    c = Case(1, 64, 128, 4, 128, 8, 2, BF)
    none = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    layer = list(c.layer())
    layer[6] = none(0, dt=torch.int32)
    G.gptq_lora_matmul(ctx, none(0, 128), *layer, none(0, 64))
    dA, dB = torch.ones(2, 8, 128, device="cuda"), torch.ones(2, 8, 64, device="cuda")
    args = (none(0, 64), none(0, 128), *layer, none(0, 8, dt=F32))
    G.gptq_lora_backward(ctx, *args, dX=none(0, 128), dA=dA, dB=dB, accumulate=True)
    G.gptq_sync_status(ctx)
    assert (dA == 1).all() and (dB == 1).all()
    G.gptq_lora_backward(ctx, *args, dX=none(0, 128), dA=dA, dB=dB)
    G.gptq_sync_status(ctx)
    assert (dA == 0).all() and (dB == 0).all()


def test_bad_ids_and_zeros_are_reported(ctx):
    c = Case(8, 64, 256, 4, 128, 8, 2, BF, "mixed", 9)
    good = c.adapter.clone()
    for bad in (2, -2, 2 ** 31 - 1, -2 ** 31):
        c.adapter.copy_(good)
        c.adapter[3] = -1
        want, _ = _forward(ctx, c, F32)
        c.adapter[3] = bad                 # counts as no adapter
        Y = torch.empty_like(want)
        G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y)
        with pytest.raises(G.GPTQError) as e:
            G.gptq_sync_status(ctx)
        assert e.value.code == G.GPTQ_ERR_ARG and torch.equal(Y, want)
        for out in (dict(dX=torch.empty_like(c.X)), dict(dB=torch.empty_like(c.B, dtype=F32))):
            G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), torch.zeros(8, 8, device="cuda"), **out)
            with pytest.raises(G.GPTQError) as e:
                G.gptq_sync_status(ctx)
            assert e.value.code == G.GPTQ_ERR_ARG
    for T in (8, 80):
        c = Case(T, 64, 256, 4, 128, 8, 2, HF, "mixed", 9)
        Y, dX = torch.empty(T, 64, device="cuda"), torch.empty_like(c.X)
        calls = [lambda: G.gptq_lora_matmul(ctx, c.X, *c.layer(), Y),
                 lambda: G.gptq_lora_backward(ctx, c.dY, None, *c.layer(), None, dX=dX)]
        c.zeros[5, 1] = 16
        for call in calls:
            call()
            with pytest.raises(G.GPTQError) as e:
                G.gptq_sync_status(ctx)
            assert e.value.code == G.GPTQ_ERR_ARG
        c.zeros[5, 1] = 15
        c.scales[3, 0] = 17.5              # fp16 weights of 255 and more: the backward pass only
        calls[0]()
        G.gptq_sync_status(ctx)
        calls[1]()
        with pytest.raises(G.GPTQError) as e:
            G.gptq_sync_status(ctx)
        assert e.value.code == G.GPTQ_ERR_ARG


def test_refusals(ctx):
    c = Case(8, 64, 256, 4, 128, 8, 2, BF)
    Y, layer = torch.empty(8, 64, dtype=BF, device="cuda"), c.layer()

    def refused(i, value, exc=ValueError):
        bad = list(layer)
        bad[i] = value
        with pytest.raises(exc):
            G.gptq_lora_matmul(ctx, c.X, *bad, Y)

    refused(0, c.packed.cpu())
    refused(0, c.packed[:, :-1].contiguous())
    refused(2, 9)                                      # bits: the words of a row no longer fit
    refused(3, 0, G.GPTQError)
    refused(3, -2, G.GPTQError)
    refused(3, 64, G.GPTQError)                        # scales have too few groups
    refused(5, c.zeros.float())
    refused(6, c.adapter.long())
    refused(6, c.adapter[:-1].contiguous())
    refused(7, c.A.float())
    refused(7, c.A.transpose(1, 2))
    refused(8, c.B[:, :, :-1].contiguous())
    refused(9, c.scaling[:1])
    with pytest.raises(ValueError):
        G.gptq_lora_matmul(ctx, c.X, *layer, torch.empty(8, 64, dtype=HF, device="cuda"))
    with pytest.raises(ValueError):
        G.gptq_lora_matmul(ctx, c.X, *layer, Y, U=torch.empty(8, 9, device="cuda"))
    with pytest.raises(G.GPTQError):
        G.gptq_lora_backward(ctx, c.dY, c.X, *layer, None)                    # nothing to compute
    with pytest.raises(G.GPTQError):
        G.gptq_lora_backward(ctx, c.dY, None, *layer, None, dA=torch.empty_like(c.A, dtype=F32))
    small = G.Context(1, 1)            # and then one whose workspace really is 1 KB
    small.close()
    small.workspace, small.handle = torch.empty(1024, dtype=torch.uint8, device="cuda"), ctypes.c_void_p()
    assert G._lib.gptq_create(ctypes.byref(small.handle), ctypes.c_void_p(small.stream.cuda_stream),
                              ctypes.c_void_p(small.workspace.data_ptr()), 1024) == G.GPTQ_OK
    try:
        with pytest.raises(G.GPTQError) as e:
            G.gptq_lora_matmul(small, c.X.repeat(64, 1), *layer[:6], c.adapter.repeat(64), *layer[7:],
                               Y.repeat(64, 1))
        assert e.value.code == G.GPTQ_ERR_NOMEM
    finally:
        small.close()


@pytest.mark.parametrize("T", [3, 80])
def test_workspace_as_asked_for_suffices(T):
    c = Case(T, 300, 640, 3, 128, 16, 3, BF, "mixed", 10)
    own = G.Context(1, 1, workspace_bytes=G.gptq_lora_workspace_bytes(T, 300, 640, 3, 3, 16, BF))
    try:
        Y, U = _forward(own, c, F32)
        want, bound, _, _ = c.forward(F32)
        within(Y, want, bound, "Y")
        _backward(own, c, U)
    finally:
        own.close()


def test_stage_timing_counts_the_calls(ctx):
    c = Case(80, 256, 512, 4, 128, 16, 2, BF, "runs", 14)
    plain, _ = _forward(ctx, c, F32)
    G.gptq_timing_enable(ctx, True)
    timed, U = _forward(ctx, c, F32)
    _backward(ctx, c, U)
    ms, launches = G.gptq_timing_read(ctx)["lora"]
    G.gptq_timing_enable(ctx, False)
    assert launches >= 5 and ms > 0 and torch.equal(plain, timed)


@pytest.mark.parametrize("T", [4, 200])
def test_captured_and_replayed(T):
    """Forward and backward in one graph, replayed with other inputs."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = Case(T, 384, 512, 4, 128, 16, 3, BF, "runs", 11)
    ctx = G.Context(1, 1, workspace_bytes=64 << 20, stream=s)
    try:
        with torch.cuda.stream(s):
            outs = [torch.empty(T, 384, device="cuda"), torch.empty(T, 16, device="cuda"),
                    torch.empty_like(c.X), torch.empty(3, 16, 512, device="cuda"),
                    torch.empty(3, 16, 384, device="cuda")]

            def step():
                G.gptq_lora_matmul(ctx, c.X, *c.layer(), outs[0], U=outs[1])
                G.gptq_lora_backward(ctx, c.dY, c.X, *c.layer(), outs[1], dX=outs[2], dA=outs[3],
                                     dB=outs[4])

            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            for k in range(2):
                c.X.normal_()
                c.adapter.copy_(torch.roll(c.adapter, 1))
                step()
                want = [o.clone() for o in outs]
                for o in outs:
                    o.fill_(float("nan"))
                graph.replay()
                s.synchronize()
                for a, b in zip(outs, want):
                    assert torch.equal(a, b)
        G.gptq_sync_status(ctx)
    finally:
        torch.cuda.synchronize()
        ctx.close()


def test_two_contexts_at_once():
    """Two streams, each with its own context, work side by side."""
    cases = [Case(40, 384, 512, 4, 128, 16, 3, BF, "mixed", 20 + k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    ctxs = [G.Context(1, 1, workspace_bytes=32 << 20, stream=s) for s in streams]
    outs = [torch.empty(40, 384, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    try:
        for _ in range(20):
            for c, x, o in zip(cases, ctxs, outs):
                G.gptq_lora_matmul(x, c.X, *c.layer(), o)
        torch.cuda.synchronize()
        for c, x, o in zip(cases, ctxs, outs):
            want, bound, _, _ = c.forward(F32)
            within(o, want, bound, "Y")
            G.gptq_sync_status(x)
    finally:
        for x in ctxs:
            x.close()
