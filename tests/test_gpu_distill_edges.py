"""Distillation: values and calls at which a row's place in memory, or another call, must not matter."""
import ctypes
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


def _side_by_side(calls, rounds):
    """(fn, ctypes arguments, context) of `calls`, `rounds` times each from a thread of its own; the error codes.
    The arguments are ready, so that the threads spend their time inside the library."""
    import threading
    errors, gate = set(), threading.Barrier(len(calls))

    def work(fn, args):
        gate.wait()
        for _ in range(rounds):
            rc = fn(*args)
            if rc:
                errors.add(rc)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def _contexts(n, **kw):
    return [G.Context(1, 1, stream=torch.cuda.Stream(), **kw) for _ in range(n)]


def test_long_and_short_rows_from_several_threads():
    """A context each: no call takes away the shared memory that another's rows need."""
    ctxs, calls, kept = _contexts(6), [], []
    for c, V in zip(ctxs, (262144, 100, 100, 100, 100, 100)):
        z = torch.randn(2, V, device="cuda").to(BF)
        val, idx = torch.randn(2, 4, device="cuda"), torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
        loss, lse = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
        kept.append((z, val, idx, loss, lse))
        calls.append((G._lib.gptq_distill_topk,
                      (c.handle, _p(z), G.GPTQ_BF16, 2, V, V, _p(val), _p(idx), 4, ctypes.c_float(1.0), None, None,
                       _p(loss), _p(lse), None, None, 0)))
    torch.cuda.synchronize()
    try:
        assert not _side_by_side(calls, 20000)
    finally:
        for c in ctxs:
            c.close()


def test_adapter_gradients_of_many_and_few_tokens_from_several_threads():
    ctxs, calls, kept = _contexts(6, workspace_bytes=8 << 20), [], []
    for c, T in zip(ctxs, (8192, 8, 8, 8, 8, 8)):
        e = lambda *s, dt=BF: torch.ones(*s, device="cuda", dtype=dt)  # noqa: E731
        t = dict(dY=e(T, 8), packed=e(8, 1, dt=torch.int32), scales=e(8, 1, dt=F32), zeros=e(8, 1, dt=torch.int32),
                 adapter=torch.zeros(T, device="cuda", dtype=torch.int32), A=e(1, 1, 8), B=e(1, 1, 8),
                 scaling=e(1, dt=F32), U=e(T, 1, dt=F32), dB=e(1, 1, 8, dt=F32))
        kept.append(t)
        calls.append((G._lib.gptq_lora_backward,
                      (c.handle, _p(t["dY"]), None, G.GPTQ_BF16, T, 8, _p(t["packed"]), 8, 4, -1, None, 1,
                       _p(t["scales"]), _p(t["zeros"]), _p(t["adapter"]), 1, 1, _p(t["A"]), _p(t["B"]),
                       _p(t["scaling"]), _p(t["U"]), None, None, _p(t["dB"]), 0)))
    torch.cuda.synchronize()
    try:
        assert not _side_by_side(calls, 20000)
    finally:
        for c in ctxs:
            c.close()
