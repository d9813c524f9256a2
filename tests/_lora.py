"""Inputs, the fp64 formulas and the error bounds of the adapter projection's tests."""
import numpy as np
import torch

from oracle import gptq_oracle as O

U32 = 2.0 ** -24


def adapters_of(T, n, pattern, seed):
    """The adapter of every token: "runs" (ragged requests in a row), "mixed" (every token another
    request's), "one", "none"."""
    rng = np.random.default_rng(seed)
    if pattern == "none":
        return np.full(T, -1, np.int32)
    if pattern == "one":
        return np.full(T, n - 1, np.int32)
    if pattern == "mixed":
        return rng.integers(-1, n, T).astype(np.int32)
    cuts = np.sort(rng.integers(0, T + 1, 4))
    return rng.integers(-1, n, 5).astype(np.int32)[np.searchsorted(cuts, np.arange(T), side="right")]


class Case:
    """One layer with adapters and a batch, on the GPU; `offset`: elements by which the 16-bit
    tensors miss a 16-byte boundary."""

    def __init__(self, T, m, d, bits, group, R, n, dtype, pattern="runs", seed=0, gid=False,
                 offset=0):
        rng = np.random.default_rng(seed)
        self.T, self.m, self.d, self.bits, self.group, self.R, self.n = T, m, d, bits, group, R, n
        self.dtype = dtype
        ng = 1 if group == -1 else -(-d // group)
        self.codes = rng.integers(0, 2 ** bits, (m, d))
        scales = rng.uniform(1e-3, 2e-2, (m, ng)).astype(np.float32)
        zeros = rng.integers(0, 2 ** bits, (m, ng)).astype(np.int32)
        self.gid = rng.integers(0, ng, d).astype(np.int32) if gid else None
        column = self.gid if gid else (np.zeros(d, int) if group == -1 else np.arange(d) // group)
        self.W = torch.from_numpy(scales[:, column].astype(np.float64) *
                                  (self.codes - zeros[:, column])).cuda()
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).cuda()  # noqa: E731
        self.packed = i32(O.pack(self.codes, bits).astype(np.uint32))
        self.scales, self.zeros = torch.from_numpy(scales).cuda(), i32(zeros)
        self.group_id = i32(self.gid) if gid else None
        self.adapter = i32(adapters_of(T, n, pattern, seed + 1))

        def t(*shape, scale=1.0):
            a = torch.from_numpy(rng.normal(0, scale, shape).astype(np.float32)).to(dtype)
            buf = torch.zeros(a.numel() + offset, dtype=dtype, device="cuda")
            out = buf[offset:].view(shape)
            out.copy_(a)
            return out

        self.X, self.dY = t(T, d), t(T, m, scale=0.1)
        self.A, self.B = t(n, R, d, scale=d ** -0.5), t(n, R, m, scale=0.1)
        self.scaling = torch.from_numpy(rng.uniform(0.5, 2, n).astype(np.float32)).cuda()

    def layer(self):
        return (self.packed, self.d, self.bits, self.group, self.scales, self.zeros, self.adapter,
                self.A, self.B, self.scaling)

    def low(self, x, w):
        """scaling[a] x w[a]^T and the same of absolute values, in fp64."""
        out = torch.zeros(self.T, self.R, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        for a in range(self.n):
            t = torch.nonzero(self.adapter == a)[:, 0]
            s, xd, wd = float(self.scaling[a]), x[t].double(), w[a].double()
            out[t], mag[t] = s * (xd @ wd.T), s * (xd.abs() @ wd.abs().T)
        return out, mag

    def up(self, u, w):
        out = torch.zeros(self.T, w.shape[2], dtype=torch.float64, device="cuda")
        for a in range(self.n):
            t = torch.nonzero(self.adapter == a)[:, 0]
            out[t] = u[t].double() @ w[a].double()
        return out

    def outer(self, u, x):
        out = torch.zeros(self.n, self.R, x.shape[1], dtype=torch.float64, device="cuda")
        for a in range(self.n):
            t = torch.nonzero(self.adapter == a)[:, 0]
            out[a] = u[t].double().T @ x[t].double()
        return out

    # Each result's bound: fp32 sums of n terms are within 2 (n + 8) u of the sum of magnitudes
    # (twice the recursive-summation bound, for the tensor cores' own adds), a factor that is itself
    # such a sum adds its own length; rounding to a type adds half its step.
    def forward(self, y_dtype):
        """(Y, bound of Y, U, bound of U) in fp64."""
        u, umag = self.low(self.X, self.A)
        y = self.X.double() @ self.W.T + self.up(u, self.B)
        mag = self.X.double().abs() @ self.W.abs().T + self.up(umag, self.B.abs())
        err = 2 * (self.d + self.R + 8) * U32 * mag
        half = 0.0 if y_dtype == torch.float32 else torch.finfo(y_dtype).eps / 2
        return y, err + half * (y.abs() + err), u, 2 * (self.d + 8) * U32 * umag

    def backward(self, u, tensor):
        """((dX, bound), (dA, bound), (dB, bound)); u: the U that the call was given.  tensor: Ŵ is
        rounded to the 16-bit type (half a step, and 2^-17 of it for the rounding's own products)."""
        g, gmag = self.low(self.dY, self.B)
        dx = self.dY.double() @ self.W + self.up(g, self.A)
        base = self.dY.double().abs() @ self.W.abs()
        err = 2 * (self.m + self.R + 8) * U32 * (base + self.up(gmag, self.A.abs()))
        half = 0.0 if self.dtype == torch.float32 else torch.finfo(self.dtype).eps / 2
        if tensor:
            err = err + half * 1.01 * base
        dx_bound = err + half * (dx.abs() + err)
        if self.dtype == torch.float16:
            dx_bound = dx_bound + 2.0 ** -25
        da = self.outer(g, self.X)
        da_bound = 2 * (self.T + self.m + 8) * U32 * self.outer(gmag, self.X.abs())
        db = self.outer(u, self.dY)
        db_bound = 2 * (self.T + 8) * U32 * self.outer(u.abs(), self.dY.abs())
        return (dx, dx_bound), (da, da_bound), (db, db_bound)


def within(got, want, bound, what):
    assert torch.isfinite(got).all(), f"{what}: unwritten or non-finite values"
    over = ((got.double() - want).abs() / bound.clamp_min(1e-300))
    over = torch.where((got.double() - want) == 0, torch.zeros_like(over), over)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its bound at {int(over.argmax())}"
    return worst
