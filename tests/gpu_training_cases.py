"""Inputs, buffers and comparisons shared by the GPU tests of the gated block,
the cross entropy and the clipping."""
import numpy as np
import torch

from lora_adapter_amd import binding as B

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"bf16": B.LORA_BF16, "f32": B.LORA_F32}
# the largest relative error of one rounding
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 2.0 ** -24
ACTS = {"silu": B.LORA_ACT_SILU, "gelu": B.LORA_ACT_GELU, "gelu_tanh": B.LORA_ACT_GELU_TANH}


def f64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A buffer between two guards, all of it one pattern at first."""

    def __init__(self, *shape, dtype=torch.float32, pad=1024):
        n = int(np.prod(shape))
        self.whole = torch.empty(n + 2 * pad, dtype=dtype, device="cuda")
        self.whole.view(torch.uint8).fill_(0x6b)
        self.t = self.whole[pad:pad + n].view(*shape)
        self.before = self.whole.clone()
        self.pad, self.n = pad, n

    def check(self, what=""):
        for a, b in ((0, self.pad), (self.pad + self.n, self.n + 2 * self.pad)):
            assert torch.equal(self.whole[a:b].view(torch.uint8), self.before[a:b].view(torch.uint8)), \
                f"written outside the buffer: {what}"


def workspace(n):
    return torch.full((n,), 0x77, dtype=torch.uint8, device="cuda")


def near(got, ref, tol, what=""):
    """Element for element; infinities equal, NaN in the same places."""
    got = f64(got) if torch.is_tensor(got) else got
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), (what, "NaN", int((np.isnan(got) != nan).sum()))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), (what, "infinities")
    ok = ~(nan | inf)
    tol = np.broadcast_to(tol, ref.shape)
    off = np.abs(got[ok] - ref[ok])
    bad = off > tol[ok]
    i = int(np.argmax(off / np.maximum(tol[ok], 1e-300))) if bad.any() else 0
    assert not bad.any(), (what, int(bad.sum()), "worst", float(got[ok][i]), float(ref[ok][i]), float(tol[ok][i]))


def tables(rng, N, lo, hi, extra=3):
    """Ranks and a scattered page table; the last `extra` pages have no owner."""
    rank = rng.integers(lo, hi + 1, size=N).astype(np.int32)
    start = np.zeros(N + 1, np.int32)
    start[1:] = np.cumsum(rank)
    total = int(start[-1])
    ids = rng.permutation(total + extra)[:total].astype(np.int32)
    return rank, start, ids, total + extra


class Block:
    """A gated block: two pools on one page table, routing, rows and weights."""

    def __init__(self, T, K, d, F, dtype="bf16", N=6, lo=1, hi=16, seed=0, mask=False, runs=False, empty=True):
        rng = np.random.default_rng(seed)
        self.T, self.K, self.d, self.F, self.dtype, self.N = T, K, d, F, dtype, N
        dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).to("cuda") if t is None else \
            torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(t)
        self.rank, self.start, self.page_ids, self.P = tables(rng, N, lo, hi)
        self.R = max(1, int(self.rank.max()))
        ids = np.sort(rng.integers(0, N, size=(T, K)), axis=0) if runs else rng.integers(0, N, size=(T, K))
        ids = ids.astype(np.int32)
        if empty:
            ids[rng.random((T, K)) < 0.1] = -1
            ids[min(3, T - 1)] = -1                       # a row without any adapter
        self.ids = ids
        self.gates = np.ones((T, K), np.float32) if K == 1 else rng.random((T, K)).astype(np.float32)
        self.mask = (rng.random((T, d)) < 0.9).astype(np.uint8) if mask else None
        self.keep = float(np.float32(1 / 0.9)) if mask else 1.0
        t = DT[dtype]
        n = lambda *s, std=1.0: dev(rng.standard_normal(s) * std, t)
        self.X, self.dH = n(T, d), n(T, F)
        self.W = [n(F, d, std=d ** -0.5) for _ in range(2)]
        self.A = [n(self.P, d, std=0.125) for _ in range(2)]
        self.Bp = [n(self.P, F, std=0.2) for _ in range(2)]
        self.scale = [(0.5 + rng.random(N)).astype(np.float32) for _ in range(2)]
        self.d_rank, self.d_start, self.d_page_ids = dev(self.rank), dev(self.start), dev(self.page_ids)
        self.d_ids, self.d_gates = dev(self.ids), dev(self.gates)
        self.d_mask = None if self.mask is None else dev(self.mask)
        self.pools = [B.Pool(CODE[dtype], d, F, a, b, self.d_rank, self.d_start, self.d_page_ids, dev(s))
                      for a, b, s in zip(self.A, self.Bp, self.scale)]
        self.plan = workspace(B.lora_plan_bytes(T, K, N))
        nw = B.lora_apply_workspace_bytes(T, K, d, F, self.R, CODE[dtype])
        self.ws = [workspace(nw) for _ in range(2)]

    def out(self, n):
        return Guarded(self.T, n, dtype=DT[self.dtype])

    def forward(self, act, H, g=None, u=None, stream=None, ws=None, plan=None):
        w = ws or self.ws
        B.lora_gated_forward(self.d_ids, self.d_gates, self.T, self.K, self.X, *self.W, ACTS[act], H, g, u,
                             self.d_mask, self.keep, *self.pools, self.plan if plan is None else plan, *w, stream)

    def slots(self, p):
        """Per active slot: token, pages and coefficient."""
        for t in range(self.T):
            for k in range(self.K):
                a = int(self.ids[t, k])
                if a >= 0 and self.rank[a] > 0 and self.gates[t, k] != 0:
                    yield (t, self.page_ids[self.start[a]:self.start[a + 1]],
                           float(self.gates[t, k]) * float(self.scale[p][a]) * self.keep)

    def projection(self, p, with_error=True):
        """g (or u) in 64 bits and the error a float32 sum of it may have."""
        X, W, A, Bp = f64(self.X), f64(self.W[p]), f64(self.A[p]), f64(self.Bp[p])
        m = np.ones_like(X) if self.mask is None else self.mask.astype(np.float64)
        y = X @ W.T
        e = (self.d + 8) * EPS * (np.abs(X) @ np.abs(W).T)
        for t, pages, c in self.slots(p):
            z = X[t] * m[t]
            un, ua = c * (A[pages] @ z), abs(c) * (np.abs(A[pages]) @ np.abs(z))
            y[t] += un @ Bp[pages]
            # U is a sum of d terms, its coefficient has two roundings; then r terms, and U as two bf16
            e[t] += (self.d + 8 + pages.size) * EPS * (ua @ np.abs(Bp[pages])) + \
                2.0 ** -16 * (np.abs(un) @ np.abs(Bp[pages]))
        return y, e
