"""Measured cases of three operators that use a quantized layer after it is packed: the projection
over packed codes with low-rank adapters of many requests (forward), its backward pass for training
the adapters, and the distillation loss from a teacher's stored top logits with its gradient.

`own = False` computes each operator in plain torch, in fp32; `own = True` calls the library."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _proj(name, op, T, m, d, bits, group, rank, n, requests, x, y="", save_u=False):
    """requests: how many requests the T tokens belong to; 0: every token is a request of its own."""
    return dict(name=name, op=op, T=T, m=m, d=d, bits=bits, group=group, rank=rank, n=n,
                requests=requests, x=x, y=y or x, save_u=save_u)


def _loss(name, T, V, K, x, tau, mode, full):
    """mode: "loss" (validation), "step" (loss and gradient at once, the tokens' upstream gradients
    known) or "backward" (the gradient afterwards, from the kept log-sum-exp).
    full: the teacher's log-sum-exp over its whole vocabulary was stored with its top logits."""
    return dict(name=name, op="distill", T=T, V=V, K=K, x=x, tau=tau, mode=mode, full=full)


def listed():
    return [
        # one request decoding one token through a 7B attention projection: latency
        _proj("decode 1 q_proj", "forward", 1, 4096, 4096, 4, 128, 16, 8, 0, "bf16"),
        # a batch of 24 decoding requests, each with an adapter of its own, 7B MLP up projection
        _proj("decode 24 up_proj", "forward", 24, 11008, 4096, 4, 128, 16, 32, 0, "f16"),
        # eight decoding requests on the 175B fc2 layer: bound by its 302 MB of codes
        _proj("decode 8 fc2", "forward", 8, 12288, 49152, 4, 128, 32, 8, 0, "bf16"),
        # short ragged prompts of a dozen requests, 3-bit down projection, fp32 result
        _proj("mixed 301 down_proj 3-bit", "forward", 301, 4096, 11008, 3, 128, 8, 16, 12, "f16", "f32"),
        # one long prompt chunk of 4 requests; keeps U for a backward pass
        _proj("prompt 2048 q_proj", "forward", 2048, 4096, 4096, 4, 128, 16, 4, 4, "bf16", save_u=True),
        # the largest prompt batch, high-rank adapters
        _proj("prompt 4096 up_proj", "forward", 4096, 11008, 4096, 4, 128, 64, 8, 8, "bf16"),
        # adapter training: a small ragged micro-batch, an ordinary one, the largest
        _proj("backward 199 q_proj", "backward", 199, 4096, 4096, 4, 128, 8, 2, 3, "bf16"),
        _proj("backward 2048 q_proj", "backward", 2048, 4096, 4096, 4, 128, 16, 1, 1, "bf16"),
        _proj("backward 4096 down_proj", "backward", 4096, 4096, 11008, 4, 128, 32, 4, 4, "f16"),
        # a validation pass over a few tokens, fp32 logits
        _loss("distill eval 5 x 32000", 5, 32000, 16, "f32", 1.0, "loss", False),
        # the gradient alone, an odd vocabulary and the teacher's full mass
        _loss("distill backward 1024 x 50257", 1024, 50257, 32, "f16", 2.0, "backward", True),
        # the largest training step
        _loss("distill step 4096 x 128000", 4096, 128000, 128, "bf16", 1.0, "step", False),
    ]


MOST_FLOPS = 2.0 * 4096 * 11008 * 4096
MOST_LOGITS = 4096 * 128000


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "distill"])
    if op == "distill":
        V = _log(rng, 1000, 128000)
        T = min(_log(rng, 1, 4096), MOST_LOGITS // V)
        c = _loss("", T, V, min(_log(rng, 1, 256), V), rng.choice(["bf16", "f16", "f32"]),
                  rng.choice([1.0, 2.0, 4.0]), rng.choice(["loss", "step", "step", "backward"]),
                  rng.random() < 0.5)
    else:
        m = _log(rng, 512, 12288)
        d = 32 * _log(rng, 16, 384) if rng.random() < 0.75 else 8 * _log(rng, 64, 1536)
        T = _log(rng, 1, 4096) if op == "forward" else _log(rng, 64, 4096)
        T = max(1, min(T, int(MOST_FLOPS / (2.0 * m * d))))
        requests = rng.choice([0, 1, 3, 8]) if T < 64 else rng.choice([1, 2, 5, 16])
        bits = rng.choice([4, 4, 4, 3, 2])
        x = rng.choice(["bf16", "f16"])
        c = _proj("", op, T, m, d, bits, rng.choice([128, 128, 256, -1]), rng.choice([4, 8, 13, 16, 32, 64]),
                  rng.randint(1, 16), requests, x, rng.choice([x, "f32"]) if op == "forward" else x,
                  op == "forward" and rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------- inputs

def _words(d, bits):
    return -(-(d * bits) // 32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    s = _prepare_distill(case, g) if case["op"] == "distill" else _prepare_proj(case, g)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _prepare_proj(case, g):
    T, m, d, bits, R, n = (case[k] for k in ("T", "m", "d", "bits", "rank", "n"))
    dt, f32 = DTYPES[case["x"]], torch.float32
    ng = 1 if case["group"] == -1 else -(-d // case["group"])
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=g)       # noqa: E731
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g)     # noqa: E731
    # random words are valid codes; the bits of the last word behind the row's end are not read
    packed = torch.randint(-2 ** 31, 2 ** 31, (m, _words(d, bits)), dtype=torch.int64, device="cuda",
                           generator=g).to(torch.int32)
    # weights of about N(0, 0.02): a min-max grid of 2^bits steps around its middle
    scales = (0.5 + rand(m, ng)) * (0.12 / 2 ** bits)
    mid = 2 ** (bits - 1)
    zeros = torch.randint(mid - 1, mid + 1, (m, ng), dtype=torch.int32, device="cuda", generator=g)
    # activations with a few outlier features
    X = randn(T, d) * torch.where(rand(d) < 0.01, 8.0, 1.0)
    A, B = randn(n, R, d) / math.sqrt(d), randn(n, R, m) * (0.4 / math.sqrt(R))
    scaling = 0.5 + rand(n)
    if case["requests"]:    # contiguous requests of ragged lengths, some without an adapter
        cuts = torch.sort(torch.randint(0, T, (case["requests"] - 1,), device="cuda", generator=g)).values
        which = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
        of = torch.randint(0, n, (case["requests"],), device="cuda", generator=g)
        of = torch.where((rand(case["requests"]) < 0.15) & (torch.arange(case["requests"], device="cuda") > 0), -1, of)
        adapter = of[which]
    else:                   # every token is another request's
        adapter = torch.randint(0, n, (T,), device="cuda", generator=g)
        adapter = torch.where((rand(T) < 0.1) & (torch.arange(T, device="cuda") > 0), -1, adapter)
    s = dict(packed=packed, scales=scales, zeros=zeros, X=X.to(dt), A=A.to(dt), B=B.to(dt),
             scaling=scaling.to(f32), adapter=adapter.to(torch.int32))
    if case["op"] == "backward":
        s["dY"] = (randn(T, m) * 0.01).to(dt)
        s["U"] = _low_rank(s["X"], s["A"], s)[1]
    return s


def _prepare_distill(case, g):
    T, V, K, tau = case["T"], case["V"], case["K"], case["tau"]
    z = torch.randn(T, V, device="cuda", generator=g) * 2.0
    # the teacher's list: K distinct entries per token, more likely ones first; short lists end in -1
    idx = torch.rand(T, V, device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    values = torch.randn(T, K, device="cuda", generator=g).sort(dim=1, descending=True).values * 1.5 + 6.0
    # the student has learned most of it
    z.scatter_(1, idx.long(), values + torch.randn(T, K, device="cuda", generator=g) * 0.7)
    short = torch.randint(0, 20, (T, 1), device="cuda", generator=g) == 0
    idx = torch.where(short & (torch.arange(K, device="cuda") > K // 2), -1, idx)
    weight = torch.where(torch.rand(T, device="cuda", generator=g) < 0.1, 0.0, 1.0)   # prompt tokens: 0
    s = dict(logits=z.to(DTYPES[case["x"]]), values=values, indices=idx, weight=weight,
             dloss=torch.rand(T, device="cuda", generator=g) + 0.5)
    # the rest of the teacher's vocabulary holds some of its mass
    s["teacher_lse"] = torch.logsumexp(values / tau, 1) + 0.1 * torch.rand(T, device="cuda", generator=g) \
        if case["full"] else None
    if case["mode"] == "backward":
        s["lse"] = torch.where(weight != 0, torch.logsumexp(s["logits"].float() / tau, 1), 0.0)
    return s


def _prepare_own(case, s):
    """The library's context and the caller's output buffers."""
    import post_weight_quantization_17_b200 as G
    T, f32, e = case["T"], torch.float32, lambda *a, **k: torch.empty(*a, device="cuda", **k)
    if case["op"] == "distill":
        s["ctx"] = G.Context(1, 1, workspace_bytes=1 << 20)
        if case["mode"] != "backward":
            s["loss"], s["lse"] = e(T, dtype=f32), e(T, dtype=f32)
        s["dlogits"] = torch.empty_like(s["logits"]) if case["mode"] != "loss" else None
        return
    m, d, bits, R, n = (case[k] for k in ("m", "d", "bits", "rank", "n"))
    dt = DTYPES[case["x"]]
    s["ctx"] = G.Context(1, 1, workspace_bytes=G.gptq_lora_workspace_bytes(T, m, d, bits, n, R, dt))
    if case["op"] == "forward":
        s["Y"] = e(T, m, dtype=DTYPES[case["y"]])
        s["U"] = e(T, R, dtype=f32) if case["save_u"] else None
    else:
        s["dX"], s["dA"], s["dB"] = e(T, d, dtype=dt), e(n, R, d, dtype=f32), e(n, R, m, dtype=f32)


# ---------------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return _run_own(case, s)
    return {"forward": _forward, "backward": _backward, "distill": _distill}[case["op"]](case, s)


def _run_own(case, s):
    import post_weight_quantization_17_b200 as G
    if case["op"] == "forward":
        G.gptq_lora_matmul(s["ctx"], s["X"], s["packed"], case["d"], case["bits"], case["group"], s["scales"],
                           s["zeros"], s["adapter"], s["A"], s["B"], s["scaling"], s["Y"], U=s["U"])
        return {"Y": s["Y"], "U": s["U"]}
    if case["op"] == "backward":
        G.gptq_lora_backward(s["ctx"], s["dY"], s["X"], s["packed"], case["d"], case["bits"], case["group"],
                             s["scales"], s["zeros"], s["adapter"], s["A"], s["B"], s["scaling"], s["U"],
                             dX=s["dX"], dA=s["dA"], dB=s["dB"])
        return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}
    if case["mode"] == "backward":
        G.gptq_distill_topk_backward(s["ctx"], s["logits"], s["values"], s["indices"], case["tau"], s["lse"],
                                     s["dloss"], s["dlogits"], weight=s["weight"],
                                     teacher_lse=s["teacher_lse"])
        return {"dlogits": s["dlogits"]}
    step = case["mode"] == "step"
    G.gptq_distill_topk(s["ctx"], s["logits"], s["values"], s["indices"], case["tau"], s["loss"], s["lse"],
                        weight=s["weight"], teacher_lse=s["teacher_lse"], dloss=s["dloss"] if step else None,
                        dlogits=s["dlogits"])
    return {"loss": s["loss"], "lse": s["lse"], "dlogits": s["dlogits"]}


def _weights(case, s):
    """The dequantized weights, Δ (c - z), in fp32."""
    d, bits, packed = case["d"], case["bits"], s["packed"]
    if bits in (2, 4):
        shifts = torch.arange(0, 32, bits, device="cuda", dtype=torch.int32)
        codes = ((packed[:, :, None] >> shifts) & (2 ** bits - 1)).flatten(1)[:, :d]
    else:                   # codes that may straddle two words
        at = torch.arange(d, device="cuda") * bits
        low, up = at // 32, torch.clamp(at // 32 + 1, max=packed.shape[1] - 1)
        wide = packed.long() & 0xFFFFFFFF
        codes = ((wide[:, low] | (wide[:, up] << 32)) >> (at % 32)) & (2 ** bits - 1)
    column = torch.arange(d, device="cuda") // (d if case["group"] == -1 else case["group"])
    return s["scales"][:, column] * (codes - s["zeros"][:, column]).float()


def _spread(u, s):
    """[T, R] of each token's own adapter -> [T, n R], zero at the other adapters."""
    n = s["A"].shape[0]
    mine = s["adapter"][:, None] == torch.arange(n, device="cuda")
    return torch.where(mine[:, :, None], u[:, None, :], 0.0).flatten(1)


def _low_rank(x, w, s):
    """scaling[a] x w[a]^T for every token's own adapter a (w [n, R, features]): spread and as [T, R]."""
    n, R, f = w.shape
    every = (x.float() @ w.float().reshape(n * R, f).T).reshape(-1, n, R) * s["scaling"][:, None]
    mine = s["adapter"][:, None] == torch.arange(n, device="cuda")
    every = torch.where(mine[:, :, None], every, 0.0)
    return every.flatten(1), every.sum(1)


def _forward(case, s):
    wide, U = _low_rank(s["X"], s["A"], s)
    Y = s["X"].float() @ _weights(case, s).T + wide @ s["B"].float().flatten(0, 1)
    return {"Y": Y.to(DTYPES[case["y"]]), "U": U if case["save_u"] else None}


def _backward(case, s):
    wide, _ = _low_rank(s["dY"], s["B"], s)
    dX = s["dY"].float() @ _weights(case, s) + wide @ s["A"].float().flatten(0, 1)
    dA = (wide.T @ s["X"].float()).reshape(s["A"].shape)
    dB = (_spread(s["U"], s).T @ s["dY"].float()).reshape(s["B"].shape)
    return {"dX": dX.to(s["X"].dtype), "dA": dA, "dB": dB}


def _distill(case, s):
    tau, idx, w, mode = case["tau"], s["indices"].long(), s["weight"], case["mode"]
    y = s["logits"].float() / tau
    v = torch.where(idx >= 0, s["values"] / tau, -math.inf)
    if case["full"]:
        logp = v - s["teacher_lse"][:, None]
    else:
        most = v.max(1, keepdim=True).values
        logp = v - most - (v - most).exp().sum(1, keepdim=True).log()
    p, at = logp.exp(), idx.clamp(min=0)
    out = {}
    if mode == "backward":
        lse = s["lse"][:, None]
    else:
        top = y.max(1, keepdim=True).values
        lse = top + (y - top).exp().sum(1, keepdim=True).log()
        kl = torch.where(p > 0, p * (logp - (y.gather(1, at) - lse)), 0.0).sum(1)
        out = {"loss": torch.where(w != 0, w * tau * tau * kl, 0.0),
               "lse": torch.where(w != 0, lse[:, 0], 0.0), "dlogits": None}
    if mode != "loss":
        dz = (y - lse).exp() * p.sum(1, keepdim=True)
        dz.scatter_add_(1, at, -p)
        dz *= (s["dloss"] * w * tau)[:, None]
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------------- work and exact

def work(case):
    T, size = case["T"], {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "distill":
        V, K, e = case["V"], case["K"], size[case["x"]]
        passes = 1 if case["mode"] == "loss" else 2    # logits read once; gradients written once
        return {"bytes": T * V * e * passes + 8.0 * T * K + 16.0 * T, "flops": 4.0 * T * V * passes}
    m, d, R, n, e = case["m"], case["d"], case["rank"], case["n"], size[case["x"]]
    ng = 1 if case["group"] == -1 else -(-d // case["group"])
    used = min(n, case["requests"] or T)
    layer = m * _words(d, case["bits"]) * 4.0 + 8.0 * m * ng + used * R * (d + m) * e
    if case["op"] == "forward":
        return {"bytes": layer + T * d * e + T * m * size[case["y"]] + (4.0 * T * R if case["save_u"] else 0),
                "flops": 2.0 * T * m * d + 2.0 * T * R * (d + m)}
    return {"bytes": layer + T * m * e + 2.0 * T * d * e + 4.0 * T * R + 4.0 * n * R * (d + m),
            "flops": 2.0 * T * m * d + 4.0 * T * R * (d + m)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_distill(case, s) if case["op"] == "distill" else _exact_proj(case, s)


def _exact_proj(case, s):
    """Row blocks of the layer, tokens grouped by adapter, all in fp64."""
    T, m, d, bits, f64 = case["T"], case["m"], case["d"], case["bits"], torch.float64
    group = d if case["group"] == -1 else case["group"]
    forward, n = case["op"] == "forward", case["n"]
    X, ids = s["X"].to(f64), s["adapter"]
    tokens = [torch.nonzero(ids == a)[:, 0] for a in range(n)]
    left = X if forward else s["dY"].to(f64)
    out = torch.zeros(T, m if forward else d, dtype=f64, device="cuda")
    for r0 in range(0, m, 1024):
        rows = s["packed"][r0:r0 + 1024]
        stream = torch.stack([(rows >> b) & 1 for b in range(32)], 2).flatten(1)[:, :d * bits]
        code = sum(stream[:, b::bits] << b for b in range(bits)).to(f64)
        delta = s["scales"][r0:r0 + 1024].to(f64).repeat_interleave(group, 1)[:, :d]
        zero = s["zeros"][r0:r0 + 1024].to(f64).repeat_interleave(group, 1)[:, :d]
        W = delta * (code - zero)
        if forward:
            out[:, r0:r0 + 1024] = left @ W.T
        else:
            out += left[:, r0:r0 + 1024] @ W
    first, second = (s["A"], s["B"]) if forward else (s["B"], s["A"])
    low = torch.zeros(T, case["rank"], dtype=f64, device="cuda")
    dA = torch.zeros(s["A"].shape, dtype=f64, device="cuda")
    dB = torch.zeros(s["B"].shape, dtype=f64, device="cuda")
    for a, t in enumerate(tokens):
        low[t] = float(s["scaling"][a]) * (left[t] @ first[a].to(f64).T)
        out[t] += low[t] @ second[a].to(f64)
        if not forward:
            dA[a] = low[t].T @ X[t]
            dB[a] = s["U"][t].to(f64).T @ left[t]
    if forward:
        return {"Y": out, "U": low if case["save_u"] else None}
    return {"dX": out, "dA": dA, "dB": dB}


def _exact_distill(case, s):
    """The teacher as a dense distribution over the vocabulary, in blocks of tokens, in fp64."""
    T, V, tau, f64 = case["T"], case["V"], case["tau"], torch.float64
    loss, lse = torch.zeros(T, dtype=f64, device="cuda"), torch.zeros(T, dtype=f64, device="cuda")
    grad = None if case["mode"] == "loss" else torch.zeros(T, V, dtype=f64, device="cuda")
    for t0 in range(0, T, 256):
        sl = slice(t0, t0 + 256)
        w, idx = s["weight"][sl].to(f64), s["indices"][sl].long()
        logq = torch.log_softmax(s["logits"][sl].to(f64) / tau, 1)
        v = s["values"][sl].to(f64) / tau
        v[idx < 0] = -math.inf
        total = s["teacher_lse"][sl].to(f64) if case["full"] else torch.logsumexp(v, 1)
        p = torch.exp(v - total[:, None])
        have = idx >= 0
        dense = torch.zeros_like(logq)
        row = torch.arange(idx.shape[0], device="cuda")[:, None].expand_as(idx)
        dense[row[have], idx[have]] = p[have]
        loss[sl] = w * tau ** 2 * (torch.xlogy(dense, dense) - dense * logq).sum(1)
        lse[sl] = torch.where(w != 0, torch.logsumexp(s["logits"][sl].to(f64) / tau, 1), 0.0)
        if grad is not None:
            step = (s["dloss"][sl].to(f64) * w * tau)[:, None]
            grad[sl] = step * (p.sum(1, keepdim=True) * logq.exp() - dense)
    return {"dlogits": grad} if case["mode"] == "backward" else {"loss": loss, "lse": lse, "dlogits": grad}
