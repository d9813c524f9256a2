"""Distillation from a teacher's top logits (gptq_distill_topk, ..._backward) against the formula in
fp64, and the run of the new operators together: adapters trained on a packed layer."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import post_weight_quantization_17_b200 as G  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    c = G.Context(1, 1)
    yield c
    c.close()


def _inputs(T, V, K, dtype, seed, ld=None, full=False, tau=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.full((T, ld or V), 5.0, device="cuda").to(dtype)
    logits = store[:, :V]
    logits.copy_(torch.randn(T, V, device="cuda", generator=g) * 3)
    idx = torch.rand(T, V, device="cuda", generator=g).topk(K, 1).indices.to(torch.int32)
    val = torch.randn(T, K, device="cuda", generator=g) * 2 + 4
    w = 0.5 + torch.rand(T, device="cuda", generator=g)
    dl = torch.randn(T, device="cuda", generator=g)
    tl = torch.logsumexp(val / tau, 1) + 0.3 if full else None
    return logits, val, idx, w, dl, tl


def _formula(logits, val, idx, tau, w, dl, tl):
    """loss, lse, dlogits and their bounds, in fp64.  The bounds count: an exponent's argument is off
    by 4 u times its largest magnitude a (scaling, subtraction, the conversion to a power of two),
    an exponential by 2^-22 more, a sum of V terms held in more than 64 partial sums by
    (V / 64 + 32) u, a logarithm by 2 u of its value and 2^-22."""
    y, V = logits.double() / tau, logits.shape[1]
    v = torch.where(idx >= 0, val.double() / tau, -math.inf)
    L = torch.logsumexp(v, 1) if tl is None else tl.double()
    L = torch.where(torch.isfinite(L), L, 0.0)
    p = torch.exp(v - L[:, None])
    M = p.sum(1, keepdim=True)
    lse = torch.logsumexp(y, 1, keepdim=True)
    at = idx.clamp(min=0).long()
    lp, lq = v - L[:, None], y.gather(1, at) - lse
    live = p > 0
    loss = torch.where(live, p * (lp - lq), 0.0).sum(1)
    q = torch.exp(y - lse)
    dense = torch.zeros_like(y).scatter_add_(1, at, p)
    c = (dl.double() * w.double() * tau)[:, None]
    grad = c * (M * q - dense)
    a = y.masked_fill(~torch.isfinite(y), 0).abs().amax(1, keepdim=True) + lse.abs()
    av = v.masked_fill(~torch.isfinite(v), 0).abs().amax(1, keepdim=True) + L[:, None].abs()
    e_lse = 4 * U32 * (a + 2) + 2.0 ** -21 + (V / 64 + 32) * U32
    e_p = 4 * U32 * (av + 2) + 2.0 ** -20 + (val.shape[1] + 32) * U32    # relative, of p and M
    mag = torch.where(live, p * (lp.abs() + lq.abs() + 1), 0.0).sum(1)
    e_loss = w.double().abs() * tau ** 2 * (mag * (e_p[:, 0] + 8 * U32) + (M * (e_lse + e_p))[:, 0])
    e_grad = c.abs() * (M * q * (e_lse + e_p + 4 * U32 * (a + 2) + 2.0 ** -21) + dense * (e_p + 4 * U32))
    return w.double() * tau ** 2 * loss, lse[:, 0], grad, e_loss, e_lse[:, 0], e_grad


def _near(got, want, bound, dtype, what):
    if dtype != F32:
        half = torch.finfo(dtype).eps / 2
        bound = bound + half * (want.abs() + bound) + (2.0 ** -25 if dtype == HF else 0.0)
    assert torch.isfinite(got).all(), what
    # below 2^-126 an fp32 exponential may flush to zero
    worst = ((got.double() - want).abs() / (bound + 2.0 ** -126)).max()
    assert float(worst) <= 1.0, f"{what}: {float(worst):.3g} times its bound"


CASES = [
    (1, 1, 1, F32, None, False, 1.0), (1, 33, 4, BF, None, False, 2.0), (5, 32000, 16, F32, None, False, 1.0),
    (3, 50257, 32, HF, None, True, 2.0), (4, 1001, 17, BF, 1008, False, 1.0), (2, 128000, 128, BF, None, True, 1.0),
    (300, 517, 8, HF, 519, False, 4.0), (2, 4096, 2048, F32, None, False, 1.0), (7, 255, 255, BF, None, True, 0.5),
    (1, 131073, 5, F32, None, False, 1.0), (2, 262144, 64, BF, None, False, 1.0), (150, 8192, 64, F32, 8195, True, 3.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}")
def test_loss_and_gradient(ctx, case):
    T, V, K, dt, ld, full, tau = case
    z, val, idx, w, dl, tl = _inputs(T, V, K, dt, 7, ld, full, tau)
    e = lambda: torch.full((T,), float("nan"), device="cuda")  # noqa: E731
    loss, lse, loss2, lse2 = e(), e(), e(), e()
    store = torch.full((T, V + 3), 9.0, dtype=dt, device="cuda")
    dz = store[:, :V]
    G.gptq_distill_topk(ctx, z, val, idx, tau, loss, lse, weight=w, teacher_lse=tl)
    G.gptq_distill_topk(ctx, z, val, idx, tau, loss2, lse2, weight=w, teacher_lse=tl, dloss=dl, dlogits=dz)
    G.gptq_sync_status(ctx)
    want = _formula(z, val, idx, tau, w, dl, tl)
    _near(loss, want[0], want[3], F32, "loss")
    _near(lse, want[1], want[4], F32, "lse")
    _near(loss2, want[0], want[3], F32, "loss of the step")
    _near(dz, want[2], want[5], dt, "dlogits")
    assert (store[:, V:] == 9).all(), "written behind a row's end"
    dz2 = torch.full((T, V), float("nan"), dtype=dt, device="cuda")
    G.gptq_distill_topk_backward(ctx, z, val, idx, tau, lse, dl, dz2, weight=w, teacher_lse=tl)
    _near(dz2, want[2], want[5], dt, "dlogits afterwards")
    if ld:
        assert (z.as_strided((T, ld - V), (ld, 1), V) == 5).all()
    # in place, in one pass and afterwards
    one, two = z.clone(), z.clone()
    G.gptq_distill_topk(ctx, one, val, idx, tau, loss2, lse2, weight=w, teacher_lse=tl, dloss=dl, dlogits=one)
    G.gptq_distill_topk_backward(ctx, two, val, idx, tau, lse, dl, two, weight=w, teacher_lse=tl)
    G.gptq_sync_status(ctx)
    _near(one, want[2], want[5], dt, "dlogits in place")
    _near(two, want[2], want[5], dt, "dlogits in place, afterwards")


@pytest.mark.parametrize("dt", [BF, F32])
def test_masked_rows_short_lists_and_infinities(ctx, dt):
    T, V, K = 8, 700, 12
    z, val, idx, w, dl, tl = _inputs(T, V, K, dt, 8)
    idx[1] = -1                            # no entries at all
    idx[2, 5:] = -1                        # a short list
    val[3, 4] = -math.inf                  # a teacher that excludes an entry
    w[4] = 0.0                             # a masked token, its row unreadable
    z[4] = float("nan")
    idx[5, 3] = idx[5, 0]                  # the same index twice
    z[6, :] = torch.where(torch.isin(torch.arange(V, device="cuda"), idx[6]), z[6].float(), -math.inf).to(dt)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dz = torch.empty_like(z)
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, weight=w, dloss=dl, dlogits=dz)
    G.gptq_sync_status(ctx)
    assert loss[4] == 0 and lse[4] == 0 and (dz[4] == 0).all()
    assert loss[1] == 0 and (dz[1] == 0).all()
    z[4] = 0
    want = _formula(z, val, idx, 1.0, w, dl, None)
    _near(loss, want[0], want[3], F32, "loss")
    _near(dz, want[2], want[5], dt, "dlogits")
    z[7, idx[7, 2].item()] = -math.inf     # the student excludes what the teacher lists
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, weight=w, dloss=dl, dlogits=dz)
    assert loss[7] == math.inf and torch.isfinite(dz[7]).all()
    z[0] = -math.inf
    z[5, 9] = float("nan")
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, weight=w, dloss=dl, dlogits=dz)
    assert loss[0].isnan() and loss[5].isnan() and dz[5].isnan().any()
    assert torch.isfinite(loss[[1, 2, 3, 4, 6]]).all()


def test_bad_index_is_reported(ctx):
    z, val, idx, w, dl, _ = _inputs(3, 100, 6, F32, 9)
    loss, lse = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    for bad in (100, -2, 2 ** 31 - 1, -2 ** 31):
        idx2 = idx.clone()
        idx2[1, 2] = bad
        G.gptq_distill_topk(ctx, z, val, idx2, 1.0, loss, lse, weight=w)
        with pytest.raises(G.GPTQError) as e:
            G.gptq_sync_status(ctx)
        assert e.value.code == G.GPTQ_ERR_ARG
        idx2[1, 2] = -1
        want = _formula(z, val, idx2, 1.0, w, dl, None)
        _near(loss, want[0], want[3], F32, "loss")


def test_refusals(ctx):
    z, val, idx, w, dl, _ = _inputs(3, 100, 6, F32, 9)
    loss, lse, dz = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty_like(z)
    ok = dict(logits=z, values=val, indices=idx, tau=1.0, loss=loss, lse=lse, weight=w)

    def refused(exc, **change):
        with pytest.raises(exc):
            G.gptq_distill_topk(ctx, **{**ok, **change})

    refused(ValueError, logits=z.cpu())
    refused(ValueError, logits=z.double())
    refused(ValueError, logits=torch.empty(100, 3, device="cuda").T)
    refused(ValueError, values=val.half())
    refused(ValueError, indices=idx.long())
    refused(ValueError, weight=w[:2])
    refused(ValueError, dlogits=dz)                    # without dloss
    refused(ValueError, dloss=dl, dlogits=dz.half())
    refused(G.GPTQError, loss=None)
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-9):
        refused(G.GPTQError, tau=tau)
    many = torch.zeros(3, 2049, device="cuda")
    refused(G.GPTQError, values=many, indices=many.int())
    none = torch.empty(0, 100, device="cuda")
    e = torch.empty(0, device="cuda")
    G.gptq_distill_topk(ctx, none, torch.empty(0, 6, device="cuda"),
                        torch.empty(0, 6, dtype=torch.int32, device="cuda"), 1.0, e, e)
    G.gptq_sync_status(ctx)


def test_gradient_against_differences(ctx):
    """(L(z + h e) - L(z - h e)) / 2h of the fp32 loss along one direction: the loss is good to its
    bound, and the third derivative of the log-sum-exp along e is at most 2 |e|^3."""
    T, V, K, h = 4, 300, 10, 2.0 ** -5
    z, val, idx, w, dl, _ = _inputs(T, V, K, F32, 10)
    loss, lse, dz = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(z)
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, weight=w, dloss=dl, dlogits=dz)
    e = torch.sign(torch.randn(T, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)))
    diffs, slack = [], 0.0
    for s in (h, -h):
        moved = z + s * e
        got = torch.empty(T, device="cuda")
        G.gptq_distill_topk(ctx, moved, val, idx, 1.0, got, lse, weight=w)
        diffs.append(got.double())
        # z + h e is rounded to fp32: that moves the loss by at most w tau M times the rounding of y
        slack = slack + _formula(moved, val, idx, 1.0, w, dl, None)[3] + 2 * w.double() * 2 * U32 * 32
    num = (diffs[0] - diffs[1]) / (2 * h)
    got = (dz.double() * e.double()).sum(1)
    err = _formula(z, val, idx, 1.0, w, dl, None)[5].sum(1)
    bound = dl.double().abs() * (slack / (2 * h) + w.double() * h * h * 2 / 6) + err
    assert ((num * dl.double() - got).abs() <= bound).all()


def test_offsets_beyond_32_bits(ctx):
    """More than 2^31 logits, the gradient in place: every 997th token against the formula."""
    T, V, K = 17000, 128000, 8
    assert T * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    z = torch.empty(T, V, dtype=BF, device="cuda").normal_(generator=g)
    val = torch.randn(T, K, device="cuda", generator=g)
    idx = (torch.randint(0, V // K, (T, K), device="cuda", generator=g) +
           torch.arange(K, device="cuda") * (V // K)).to(torch.int32)
    w, dl = torch.ones(T, device="cuda"), torch.rand(T, device="cuda", generator=g)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    rows = torch.arange(T - 1, 0, -997, device="cuda")
    want = _formula(z[rows], val[rows], idx[rows], 1.0, w[rows], dl[rows], None)
    G.gptq_distill_topk(ctx, z, val, idx, 1.0, loss, lse, dloss=dl, dlogits=z)
    G.gptq_sync_status(ctx)
    _near(loss[rows], want[0], want[3], F32, "loss")
    _near(z[rows], want[2], want[5], BF, "dlogits")


def test_captured_and_replayed():
    s = torch.cuda.Stream()
    z, val, idx, w, dl, _ = _inputs(6, 5003, 16, BF, 12)
    torch.cuda.synchronize()
    c = G.Context(1, 1, stream=s)
    loss, lse, dz = torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(z)
    step = lambda: G.gptq_distill_topk(c, z, val, idx, 1.0, loss, lse, weight=w, dloss=dl, dlogits=dz)  # noqa: E731
    try:
        with torch.cuda.stream(s):
            step()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
            z.normal_()
            step()
            want = loss.clone(), dz.clone()
            loss.zero_(), dz.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(loss, want[0]) and torch.equal(dz, want[1])
    finally:
        torch.cuda.synchronize()
        c.close()


def test_quantize_train_adapters_and_serve():
    """The operators as they are used together: a layer is quantized by the library, its adapter is
    trained for some steps towards the full-precision layer's top logits, and serves tokens one by
    one.  Every step's loss and gradients are checked against the formulas in fp64 (bf16 logits)."""
    from workloads.synth import CONFIGS, XSource, make_weight
    spec = CONFIGS[2][0].scaled(256, 512, 2048, chunk=1024)
    W = make_weight(spec, 7, "cuda")
    ctx = G.Context(256, 512, workspace_bytes=64 << 20)
    try:
        bufs, _, _ = G.quantize_layer_pipeline(ctx, list(XSource(spec, 7, "cuda").chunks()), W, spec.bits,
                                               spec.group, spec.block)
        g = torch.Generator(device="cuda").manual_seed(13)
        T, V, d, R, K, n = 96, 256, 512, 8, 16, 2
        X = torch.randn(T, d, device="cuda", generator=g).to(BF)
        teacher = X.float() @ W.float().T
        top = teacher.topk(K, 1)
        val, idx = top.values.contiguous(), top.indices.to(torch.int32)
        tl = torch.logsumexp(teacher, 1)
        A = (torch.randn(n, R, d, device="cuda", generator=g) * d ** -0.5).to(BF)
        B = torch.zeros(n, R, V, dtype=BF, device="cuda")
        scaling = torch.tensor([2.0, 1.0], device="cuda")
        adapter = (torch.arange(T, device="cuda") % 3 - 1).to(torch.int32)
        w, dl = torch.ones(T, device="cuda"), torch.full((T,), 1.0 / T, device="cuda")
        layer = (bufs.packed, d, spec.bits, spec.group, bufs.scales, bufs.zeros, adapter, A, B, scaling)
        Y, U = torch.empty(T, V, dtype=BF, device="cuda"), torch.empty(T, R, device="cuda")
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dA, dB, dX = torch.empty(n, R, d, device="cuda"), torch.empty(n, R, V, device="cuda"), torch.empty_like(X)
        What = bufs.W_hat.double()
        for step in range(4):
            G.gptq_lora_matmul(ctx, X, *layer, Y, U=U)
            z = Y.clone()
            G.gptq_distill_topk(ctx, Y, val, idx, 1.0, loss, lse, weight=w, teacher_lse=tl, dloss=dl, dlogits=Y)
            G.gptq_lora_backward(ctx, Y, X, *layer, U, dX=dX, dA=dA, dB=dB)
            G.gptq_sync_status(ctx)
            want = _formula(z, val, idx, 1.0, w, dl, tl)
            _near(loss, want[0], want[3], F32, "loss")
            _near(Y, want[2], want[5], BF, "dlogits")
            for a in range(n):
                t = adapter == a
                Xd, dy, s = X[t].double(), Y[t].double(), float(scaling[a])
                u = s * (Xd @ A[a].double().T)
                zref = Xd @ What.T + u @ B[a].double()
                zmag = Xd.abs() @ What.abs().T + s * (Xd.abs() @ A[a].double().abs().T) @ B[a].double().abs()
                assert ((z[t].double() - zref).abs() <= 2.0 ** -8 * zref.abs() + 1100 * 2.02 * U32 * zmag).all()
                db = u.T @ dy
                dbm = (s * (Xd.abs() @ A[a].double().abs().T)).T @ dy.abs()
                assert ((dB[a].double() - db).abs() <= 2 * (d + T + 16) * U32 * dbm).all()
                gm = s * (dy.abs() @ B[a].double().abs().T)
                da = (s * (dy @ B[a].double().T)).T @ Xd
                assert ((dA[a].double() - da).abs() <= 2 * (V + T + 16) * U32 * (gm.T @ Xd.abs())).all()
            A.sub_((0.5 * dA).to(BF))
            B.sub_((0.5 * dB).to(BF))
        # serving: token by token gives the batch's rows up to the order of fp32 sums
        Yb = torch.empty(T, V, device="cuda")
        G.gptq_lora_matmul(ctx, X, *layer, Yb)
        one = torch.empty(1, V, device="cuda")
        for t in (0, 1, 2, T - 1):
            G.gptq_lora_matmul(ctx, X[t:t + 1], *layer[:6], adapter[t:t + 1], *layer[7:], one)
            mag = X[t].double().abs() @ What.abs().T
            a = int(adapter[t])
            if a >= 0:
                mag = mag + float(scaling[a]) * (X[t].double().abs() @ A[a].double().abs().T) @ B[a].double().abs()
            assert ((one[0].double() - Yb[t].double()).abs() <= 4 * (d + R + 8) * U32 * mag).all()
        G.gptq_sync_status(ctx)
    finally:
        ctx.close()
