"""Inputs, 64-bit definitions and error bounds of the adapter-layer tests.

Bounds count roundings.  A storage rounding is at most finfo(t).eps / 2 of the
value (bf16 2^-8); an fp32 sum of n products is within n * 2^-23 of the sum of
magnitudes (twice the round-to-nearest bound, so that it holds for an
accumulator that truncates); a rank vector that enters a product as two bf16
parts is within 2^-16 of its value (2^-8 of a remainder that is at most 2^-8), as three within
2^-24 (the fp32 gradients).
"""
import torch

F64 = torch.float64
U32 = 2.0 ** -23
SPLIT = 2.0 ** -16
SPLIT3 = 2.0 ** -24


def normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, dtype=torch.float32) * std).to(dtype)


class Layer:
    """A seeded layer: tensors on the CPU, moved to `device`; x, y and dy as
    windows of wider rows (`extra` columns).  stale: A and B hold other values
    past each slot's rank (a slot used before for a larger adapter), not zeros."""

    def __init__(self, T, K, N, R, L, seed=0, extra=0, ragged=True, bias=False, runs=False,
                 device="cuda", stale=False):
        g = torch.Generator().manual_seed(1000 + seed)
        self.T, self.K, self.N, self.R, self.L, self.S = T, K, list(N), R, L, len(N)
        n = sum(N)
        # a gradient row is read in 16-byte units when every slice is whole ones
        ldn = n + (extra if extra % 8 == 0 or any(v % 8 for v in N) else 8)
        wide = lambda rows, cols, ld, std: normal(g, (rows, ld), std)[:, :cols]
        mv = lambda t: self._window(t, device)
        self.x = mv(wide(T, K, K + 8 * (extra > 0), 1.0))
        self.W = mv(wide(n, K, K + 16 * (extra > 0), 0.1))
        self.dy = mv(wide(T, n, ldn, 1.0))
        self.ldn = ldn
        self.A = [normal(g, (L, R, K), 0.1).to(device) for _ in N]
        self.B = [normal(g, (L, m, R), 0.1).to(device) for m in N]
        self.bias = normal(g, (n,), 1.0).to(device) if bias else None
        idx = torch.randint(-1, L + 1, (T,), generator=g)      # -1 and L: no adapter
        if runs:
            idx = idx.repeat_interleave(97)[:T]
        self.idx = idx.to(torch.int32).to(device)
        rank = torch.randint(0, R + 1, (L,), generator=g) if ragged else torch.full((L,), R)
        if L > 1:
            rank[0], rank[1] = R, 0
        for s in range(0 if stale else self.S):
            keep = (torch.arange(R) < rank[:, None]).to(device)
            self.A[s] *= keep[:, :, None]
            self.B[s] *= keep[:, None, :]
        self.rank = rank.to(torch.int32).to(device)
        self.scale = (torch.rand((L,), generator=g) + 0.5).to(device)

    @staticmethod
    def _window(t, device):
        base = t._base if t._base is not None else t
        return base.to(device)[:, :t.shape[1]]

    def members(self):
        """(slot, true rank, token indexes) of every slot that has tokens."""
        rank = self.rank.tolist()
        for i in range(self.L):
            m = torch.nonzero(self.idx == i).flatten()
            if rank[i] > 0 and len(m):
                yield i, rank[i], m

    def offsets(self):
        off = 0
        for s, n in enumerate(self.N):
            yield s, off, n
            off += n

    def forward(self):
        """y, buf and the error bounds of both, 64 bits."""
        x, W = self.x.to(F64), self.W.to(F64)
        y, M = x @ W.T, x.abs() @ W.abs().T
        if self.bias is not None:
            y, M = y + self.bias.to(F64), M + self.bias.to(F64).abs()
        buf = torch.zeros((self.S, self.T, self.R), dtype=F64, device=x.device)
        bmag = torch.zeros_like(buf)
        D = torch.zeros_like(M)
        for i, r, m in self.members():
            for s, off, n in self.offsets():
                a, b = self.A[s][i, :r].to(F64), self.B[s][i, :, :r].to(F64)
                u, um = x[m] @ a.T, x[m].abs() @ a.abs().T
                buf[s, m, :r], bmag[s, m, :r] = u, um
                sc = float(self.scale[i])
                y[m, off:off + n] += sc * (u @ b.T)
                D[m, off:off + n] += sc * (um @ b.abs().T)
        # sums of K and of 2 R products, the scale's rounding, the split; then one bf16 rounding
        acc = (self.K + 2 * self.R + 8) * U32 * (M + 2 * D) + SPLIT * D
        return y, y.abs() * 2.0 ** -8 + 1.01 * acc, buf, (self.K + 8) * U32 * bmag

    def backward(self, with_w=True, buf=None):
        """dx, dA, dB and their bounds, 64 bits; buf: the u the call was given
        (exact there), or None (computed, with its own error)."""
        x, dy = self.x.to(F64), self.dy.to(F64)
        W = self.W.to(F64)
        n_all = sum(self.N)
        dx = dy @ W if with_w else torch.zeros_like(x)
        M = dy.abs() @ W.abs() if with_w else torch.zeros_like(x)
        D = torch.zeros_like(x)
        dA = [torch.zeros(a.shape, dtype=F64, device=x.device) for a in self.A]
        dB = [torch.zeros(b.shape, dtype=F64, device=x.device) for b in self.B]
        eA, eB = [torch.zeros_like(t) for t in dA], [torch.zeros_like(t) for t in dB]
        for i, r, m in self.members():
            sc = float(self.scale[i])
            for s, off, n in self.offsets():
                a, b = self.A[s][i, :r].to(F64), self.B[s][i, :, :r].to(F64)
                d = dy[m, off:off + n]
                v, vm = sc * (d @ b), sc * (d.abs() @ b.abs())
                dx[m] += v @ a
                D[m] += vm @ a.abs()
                dA[s][i, :r] = v.T @ x[m]
                # v: a sum of n products, scaled, split; then a sum over the tokens
                eA[s][i, :r] = ((n + 2 * len(m) + 40) * U32 + SPLIT3) * (vm.T @ x[m].abs())
                if buf is None:
                    u, um, k = x[m] @ a.T, x[m].abs() @ a.abs().T, self.K
                else:
                    u = buf[s, m, :r].to(F64)
                    um, k = u.abs(), 0
                dB[s][i, :, :r] = sc * (d.T @ u)
                eB[s][i, :, :r] = ((k + 2 * len(m) + 40) * U32 + SPLIT3) * sc * (d.abs().T @ um)
        acc = (2 * n_all + 2 * self.R * self.S + 40) * U32 * (M + D) + SPLIT * D
        return dx, dx.abs() * 2.0 ** -8 + 1.01 * acc, dA, eA, dB, eB


def within(got, ref, tol, what):
    err = (got.to(F64) - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} past the bound; worst error "
        f"{float(err[bad].max()):.3e} at {torch.nonzero(bad)[0].tolist()}")
