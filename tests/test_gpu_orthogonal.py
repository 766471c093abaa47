"""Orthogonalised updates on the GPU against the 64-bit oracle.

Tolerances are oracle.orthogonal.tolerance (derived there).  The momentum's
arithmetic is made exact by the inputs (a momentum of 1/2 and few significant
bits), so that N is the same on both sides; a weight then carries its own
fp32 operations, and a bf16 page one rounding of at most 2^-8 of it.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import orthogonal as NS

pytestmark = pytest.mark.gpu

COEF = B.NS_COEF
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


class Fleet:
    """Adapters of the given ranks over scattered pages, three of them spare."""

    def __init__(self, ranks, d_in, d_out, dtype="f32", seed=0):
        rng = np.random.default_rng(seed)
        self.rng, self.ranks = rng, np.asarray(ranks, np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.ranks)]).astype(np.int32)
        total = int(self.start[-1])
        self.n_pages = total + 3
        self.ids = rng.permutation(self.n_pages)[:total].astype(np.int32)
        self.d = (d_in, d_out)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.t = [dev(self.ranks), dev(self.start), dev(self.ids if total else np.zeros(1, np.int32)),
                  torch.ones(len(ranks), device="cuda")]
        td = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.pages = [torch.from_numpy(self.values(d)).cuda().to(td) for d in self.d]
        self.pool = B.Pool(B.LORA_BF16 if dtype == "bf16" else B.LORA_F32, d_in, d_out, *self.pages, self.t[0],
                           self.t[1], self.t[2][:total], self.t[3])

    def values(self, d):
        """Eight significant bits, rows of unlike powers of two."""
        v = self.rng.integers(-128, 129, size=(self.n_pages, d)).astype(np.float32)
        return v * (2.0 ** self.rng.integers(-12, -4, size=(self.n_pages, 1))).astype(np.float32)

    def rows(self, a):
        return self.ids[self.start[a]:self.start[a + 1]]


def run_ortho(fl, src, ads, max_rank, steps=5, coef=COEF, eps=EPS, stream=None):
    d = src.shape[1]
    out = torch.full_like(src, 7.0)
    ork = torch.full((len(ads),), -5, dtype=torch.int32, device="cuda")
    ad = torch.tensor(ads, dtype=torch.int32, device="cuda")
    ws = torch.full((B.lora_orthogonalise_workspace_bytes(len(ads), max_rank, d),), 0xff, dtype=torch.uint8,
                    device="cuda")
    B.lora_orthogonalise(fl.pool, ad, len(ads), max_rank, src, out, d, steps, coef, eps, ws, ork, stream)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64), ork.cpu().numpy().tolist()


@pytest.mark.parametrize("d", [64, 192, 1088])
@pytest.mark.parametrize("ranks", [[1], [1, 2, 5], [16, 3, 16], [17, 32, 8], [33, 64, 1, 16]])
def test_orthogonalise(ranks, d):
    fl = Fleet(ranks, d, d, seed=sum(ranks) + d)
    src = torch.from_numpy(fl.values(d)).cuda()
    ads = list(range(len(ranks)))[::-1]
    out, ork = run_ortho(fl, src, ads, max(ranks))
    assert ork == [ranks[a] for a in ads]
    seen = np.zeros(fl.n_pages, bool)
    for a in ads:
        N = src.cpu().numpy()[fl.rows(a)].astype(np.float64)
        off = np.abs(out[fl.rows(a)] - NS.newton_schulz(N, 5, COEF, EPS))
        tol = NS.tolerance(N, 5, COEF, EPS)
        assert np.all(off <= tol), (a, float(np.max(off / tol)))
        seen[fl.rows(a)] = True
    assert (out[~seen] == 7).all()                    # spare pages


@pytest.mark.parametrize("ranks,d,steps", [([65], 64, 5), ([100, 3, 64, 128], 576, 5), ([200, 16], 1088, 3),
                                           ([96], 192, 1), ([81, 33], 192, 2)])
def test_orthogonalise_ranks_over_64(ranks, d, steps):
    fl = Fleet(ranks, d, d, seed=sum(ranks) + d)
    src = torch.from_numpy(fl.values(d)).cuda()
    out, ork = run_ortho(fl, src, list(range(len(ranks))), max(ranks), steps)
    assert ork == ranks
    for a in range(len(ranks)):
        N = src.cpu().numpy()[fl.rows(a)].astype(np.float64)
        off = np.abs(out[fl.rows(a)] - NS.newton_schulz(N, steps, COEF, EPS))
        tol = NS.tolerance(N, steps, COEF, EPS)
        assert np.all(off <= tol), (a, float(np.max(off / tol)))


@pytest.mark.parametrize("steps", [1, 2, 32])
def test_other_steps_and_coefficients(steps):
    fl = Fleet([7, 24], 320, 320, seed=steps)
    src = torch.from_numpy(fl.values(320)).cuda()
    coef = (1.5, -0.5, 0.0)
    out, _ = run_ortho(fl, src, [0, 1], 24, steps, coef, 1e-3)
    for a in (0, 1):
        N = src.cpu().numpy()[fl.rows(a)].astype(np.float64)
        off = np.abs(out[fl.rows(a)] - NS.newton_schulz(N, steps, coef, 1e-3))
        if steps < 32:                                # the bound grows with c0^(3 steps)
            assert np.all(off <= NS.tolerance(N, steps, coef, 1e-3))
        else:
            # converged, where perturbations of the r x r matrices die out: orthonormal rows, up to the
            # rounding of Q and N / norm and their fp32 sum (tolerance()'s first term), once for each factor of O O^T
            O, X = out[fl.rows(a)], N / (np.linalg.norm(N) + 1e-3)
            t = (len(O) + 6) * 2.0 ** -24 * (np.abs(NS.left_factor(N, steps, coef, 1e-3)) @ np.abs(X))
            lim = t @ np.abs(O).T
            assert np.all(np.abs(O @ O.T - np.eye(len(O))) <= lim + lim.T + 1e-9)


def test_skipped_entries_touch_nothing():
    ranks = [4, 0, 9, 16, 3, 5]
    fl = Fleet(ranks, 128, 128, seed=4)
    ids = fl.ids.copy()
    ids[fl.start[4]] = fl.n_pages                     # adapter 4: a page out of range
    ids[fl.start[4] + 1] = -1
    start = fl.start.copy()
    fl.t[2].copy_(torch.from_numpy(ids))
    rank = fl.ranks.copy()
    rank[5] = 6                                       # adapter 5: rank and page table differ
    fl.t[0].copy_(torch.from_numpy(rank))
    src = torch.from_numpy(fl.values(128)).cuda()
    ads = [2, -1, 6, 1, 0, 2, 3, 4, 5, 1 << 30, -(1 << 31), 0]
    out, ork = run_ortho(fl, src, ads, 9)
    assert ork == [9, 0, 0, 0, 4, 0, 0, 0, 0, 0, 0, 0]
    live = np.concatenate([fl.rows(0), fl.rows(2)])
    mask = np.zeros(fl.n_pages, bool)
    mask[live] = True
    assert (out[~mask] == 7).all()
    for a in (0, 2):
        N = src.cpu().numpy()[fl.rows(a)].astype(np.float64)
        assert np.all(np.abs(out[fl.rows(a)] - NS.newton_schulz(N, 5, COEF, EPS)) <= NS.tolerance(N, 5, COEF, EPS))


def test_a_pool_without_pages():
    fl = Fleet([0, 0], 64, 64)
    src = torch.zeros(3, 64, device="cuda")
    out, ork = run_ortho(fl, src, [0, 1], 1)
    assert ork == [0, 0] and (out == 7).all()


def test_zero_tiny_huge_and_non_finite():
    fl = Fleet([3, 3, 3, 3, 70, 3], 128, 128, seed=9)
    v = fl.values(128)
    v[fl.rows(0)] = 0
    v[fl.rows(1)] *= np.float32(2.0 ** -90)           # far below eps: the result is tiny too
    v[fl.rows(2)] *= np.float32(2.0 ** 100)
    v[fl.rows(3)[1], 5] = np.nan
    v[fl.rows(4)] = 0
    src = torch.from_numpy(v).cuda()
    out, _ = run_ortho(fl, src, list(range(6)), 70)
    assert (out[fl.rows(0)] == 0).all() and (out[fl.rows(4)] == 0).all()
    assert np.isnan(out[fl.rows(3)]).all()
    for a in (1, 2, 5):
        N = v[fl.rows(a)].astype(np.float64)
        off = np.abs(out[fl.rows(a)] - NS.newton_schulz(N, 5, COEF, EPS))
        assert np.all(off <= NS.tolerance(N, 5, COEF, EPS) + 2.0 ** -149), a


def step_once(fl, ads, max_rank, mom, grad, master, lr, decay, nesterov, mu=0.5, stream=None, ws=None):
    ad = torch.tensor(ads, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.full((B.lora_orthogonal_step_workspace_bytes(len(ads), max_rank, *fl.d),), 0xff,
                        dtype=torch.uint8, device="cuda")
    f = [B.FactorUpdate(fl.pages[i], grad[i], mom[i], master[i], lr[i], decay) for i in (0, 1)]
    B.lora_orthogonal_step(fl.pool, ad, len(ads), max_rank, f[0], f[1], mu, nesterov, 5, COEF, EPS, ws, None, stream)
    return ad, ws, f


@pytest.mark.parametrize("dtype,with_master", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
@pytest.mark.parametrize("ranks,d_in,d_out,nesterov", [([1, 16, 7], 192, 64, True), ([40, 5], 64, 1088, False),
                                                       ([70, 12], 320, 192, True)])
def test_step(ranks, d_in, d_out, nesterov, dtype, with_master):
    fl = Fleet(ranks, d_in, d_out, dtype, seed=sum(ranks))
    dev = lambda a: torch.from_numpy(a).cuda()
    grad = [dev(fl.values(d)) for d in fl.d]
    mom = [dev(fl.values(d)) for d in fl.d]
    master = [dev(fl.values(d)) if with_master else None for d in fl.d]
    lr, decay = (0.03, 0.5), 0.1
    before = [[t.double().cpu().numpy() if t is not None else None for t in (grad[i], mom[i], master[i], fl.pages[i])]
              for i in (0, 1)]
    ads = list(range(1, len(ranks)))                  # adapter 0 is not stepped
    keep = step_once(fl, ads, max(ranks), mom, grad, master, lr, decay, nesterov)
    torch.cuda.synchronize()
    for i in (0, 1):
        g, m0, w0, p0 = before[i]
        m1, p1 = mom[i].double().cpu().numpy(), fl.pages[i].double().cpu().numpy()
        w1 = master[i].double().cpu().numpy() if with_master else None
        done = np.zeros(fl.n_pages, bool)
        for a in ads:
            r = fl.rows(a)
            done[r] = True
            m = 0.5 * m0[r] + g[r]
            assert np.array_equal(m1[r], m)           # exact in fp32
            N = g[r] + 0.5 * m if nesterov else m
            O, tol = NS.newton_schulz(N, 5, COEF, EPS), NS.tolerance(N, 5, COEF, EPS)
            lr32, keep32 = float(np.float32(lr[i])), float(np.float32(1) - np.float32(lr[i]) * np.float32(decay))
            w = (w0 if with_master else p0)[r] * keep32 - lr32 * O
            # the factor, the two products, their difference
            t = lr32 * tol + 2.0 ** -24 * (3 * np.abs((w0 if with_master else p0)[r]) + lr32 * np.abs(O) + np.abs(w))
            if with_master:
                assert np.all(np.abs(w1[r] - w) <= t)
                # the page is the master rounded once
                want = torch.from_numpy(w1[r]).float().to(fl.pages[i].dtype).double().numpy()
                assert np.array_equal(p1[r], want)
            else:
                half = 2.0 ** -8 if dtype == "bf16" else 0.0
                assert np.all(np.abs(p1[r] - w) <= t + half * (np.abs(w) + t))
        assert np.array_equal(m1[~done], m0[~done]) and np.array_equal(p1[~done], p0[~done])
        if with_master:
            assert np.array_equal(w1[~done], w0[~done])


def test_fp32_pages_as_their_own_master():
    got = []
    for own in (False, True):
        fl = Fleet([9, 70], 128, 192, "f32", seed=6)
        dev = lambda a: torch.from_numpy(a).cuda()
        grad, mom = [dev(fl.values(d)) for d in fl.d], [dev(fl.values(d)) for d in fl.d]
        keep = step_once(fl, [0, 1], 70, mom, grad, fl.pages if own else [None, None], (0.1, 0.2), 0.3, True)
        torch.cuda.synchronize()
        got.append([*fl.pages, *mom])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_step_repeats_on_a_stream_and_in_a_graph():
    def state():
        fl = Fleet([16, 9, 70], 192, 320, "bf16", seed=5)
        dev = lambda a: torch.from_numpy(a).cuda()
        return fl, [dev(fl.values(d)) for d in fl.d], [dev(fl.values(d)) for d in fl.d], [dev(fl.values(d)) for d in fl.d]

    def both(fl, mom, master):
        return [t.clone() for t in (*mom, *master, *fl.pages)]

    fl, grad, mom, master = state()
    want = []
    for _ in range(3):
        k = step_once(fl, [0, 1, 2], 70, mom, grad, master, (0.1, 0.1), 0.0, True)
        torch.cuda.synchronize()
        want.append(both(fl, mom, master))
    # another stream
    fl, grad, mom, master = state()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        k = step_once(fl, [0, 1, 2], 70, mom, grad, master, (0.1, 0.1), 0.0, True)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(fl, mom, master), want[0]))
    # a captured step, replayed
    fl, grad, mom, master = state()
    ws = torch.empty(B.lora_orthogonal_step_workspace_bytes(3, 70, *fl.d), dtype=torch.uint8, device="cuda")
    ad = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    f = [B.FactorUpdate(fl.pages[i], grad[i], mom[i], master[i], 0.1, 0.0) for i in (0, 1)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lora_orthogonal_step(fl.pool, ad, 3, 70, f[0], f[1], 0.5, True, 5, COEF, EPS, ws)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(both(fl, mom, master), want[i])), i


def test_many_adapters_and_chunks():
    rng = np.random.default_rng(2)
    ranks = rng.integers(1, 25, size=150).tolist()
    fl = Fleet(ranks, 2112, 64, seed=8)
    src = torch.from_numpy(fl.values(2112)).cuda()
    out, ork = run_ortho(fl, src, list(range(150)), 24)
    assert ork == ranks
    for a in range(0, 150, 13):
        N = src.cpu().numpy()[fl.rows(a)].astype(np.float64)
        assert np.all(np.abs(out[fl.rows(a)] - NS.newton_schulz(N, 5, COEF, EPS)) <= NS.tolerance(N, 5, COEF, EPS))
    # one matrix over many column chunks
    fl = Fleet([16], 8256, 64, seed=8)
    src = torch.from_numpy(fl.values(8256)).cuda()
    out, _ = run_ortho(fl, src, [0], 16)
    N = src.cpu().numpy()[fl.rows(0)].astype(np.float64)
    assert np.all(np.abs(out[fl.rows(0)] - NS.newton_schulz(N, 5, COEF, EPS)) <= NS.tolerance(N, 5, COEF, EPS))
