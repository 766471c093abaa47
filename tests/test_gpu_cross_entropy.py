"""Softmax cross entropy on the GPU against 64 bits.

Tolerances: a logit is a float32 sum of d products, scaled and made relative to
the target's (which is exact to float64): e_v = (d + 8) 2^-24 sum |x w| +
2^-23 (|l_v| + |l_y|) + 2^-22.  The loss moves by sum_{v != y} p_v e_v, and its
own float32 sum of V terms by V 2^-24 relative.  In dX each probability is off
by e_v, by its rounding (half a step of the type) and by the normalisation; the
sum over V by V 2^-24; then one rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import training as R
from tests.gpu_training_cases import CODE, DT, EPS, HALF, Guarded, f64, near, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def make(T, V, d, dtype, seed=0, ignored=0.3, size=1.0):
    rng = np.random.default_rng(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(DT[dtype])
    W = dev(rng.standard_normal((V, d)) * (2 / d) ** 0.5)
    y = rng.integers(0, V, size=T).astype(np.int32)
    lean = 14 * rng.random((T, 1))
    X = dev(size * (rng.standard_normal((T, d)) + lean * f64(W)[y] / 2 ** 0.5))
    y[rng.random(T) < ignored] = -1
    w = (0.5 + rng.random(T)).astype(np.float32)
    return X, W, torch.from_numpy(y).cuda(), torch.from_numpy(w).cuda()


def run(X, W, y, w, scale=1.0, grad=True, stream=None):
    (T, d), V = X.shape, W.shape[0]
    dtype = CODE["bf16" if X.dtype == torch.bfloat16 else "f32"]
    loss, dX = Guarded(T), Guarded(T, d, dtype=X.dtype)
    ws = workspace(B.lora_cross_entropy_workspace_bytes(T, V, d, dtype, grad))
    B.lora_cross_entropy(X, W, dtype, T, V, d, y, w, scale, loss.t, dX.t if grad else None, ws, stream)
    torch.cuda.synchronize()
    loss.check("loss")
    dX.check("dX")
    return loss.t, dX.t


def tolerances(X, W, y, w, scale, loss, dX, P, half):
    """From the oracle's results."""
    d, V = X.shape[1], W.shape[0]
    tl, tx = np.zeros(X.shape[0]), np.zeros_like(X)
    for t in range(X.shape[0]):
        c = int(y[t])
        wt = 1.0 if w is None else float(w[t])
        if c < 0 or c >= V or wt == 0 or not np.isfinite(loss[t]):
            continue
        l = scale * (W @ X[t])
        e = (d + 8) * EPS * abs(scale) * (np.abs(W) @ np.abs(X[t])) + 2 * EPS * (np.abs(l) + abs(l[c])) + 2.0 ** -22
        # of one token's logits only differences that stay small are to first order
        q = P[t].copy()
        q[c] = 0
        shift = q @ e + (V + 4) * EPS * q.sum()
        tl[t] = 1.02 * abs(wt) * shift + 4 * EPS * abs(loss[t]) + 1e-37
        rel = e + half + (V + 8) * EPS
        k = abs(wt * scale)
        tx[t] = 1.02 * k * ((q * (rel + shift)) @ np.abs(W) + q.sum() * (shift + rel.max()) * np.abs(W[c]))
        # exponentials are relative to the target's, and those under 2^-126 of it may be
        # taken as 0 (float32 has no smaller normal numbers): V of them, each off by at
        # most 2 . 2^-126 / Z <= 2 . 2^-126, times k |W|; the largest is the target's or
        # more, so Z >= 1 / 2 on the shift that ref's rounding leaves
        tx[t] += 2 * k * 2.0 ** -126 * np.abs(W).sum(0) * 2
        tx[t] += half * (np.abs(dX[t]) + tx[t]) + 1e-37
    return tl, tx


def check(X, W, y, w, scale=1.0):
    half = HALF["bf16" if X.dtype == torch.bfloat16 else "f32"]
    Xd, Wd, yd = f64(X), f64(W), y.cpu().numpy()
    wd = None if w is None else f64(w)
    loss, dX, P = R.cross_entropy(Xd, Wd, yd, wd, scale)
    tl, tx = tolerances(Xd, Wd, yd, wd, scale, loss, dX, P, half)
    got = run(X, W, y, w, scale)
    near(got[0], loss, tl, "loss")
    near(got[1], dX, tx, "dX")
    only = run(X, W, y, w, scale, grad=False)
    assert torch.equal(torch.nan_to_num(only[0], 7.0), torch.nan_to_num(got[0], 7.0))
    assert bool((only[1].view(torch.uint8) == 0x6b).all())
    return got


@pytest.mark.parametrize("T,V,d", [(1, 1, 64), (1, 2, 64), (1, 1000, 576), (2, 63, 64), (63, 64, 192), (64, 65, 64),
                                   (65, 127, 128), (255, 257, 320), (257, 1000, 256), (300, 5003, 192),
                                   (513, 769, 1088), (40, 20011, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_against_64_bits(T, V, d, dtype):
    check(*make(T, V, d, dtype, seed=T + V))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.25, -1.5, 30.0])
def test_logit_scale(dtype, scale):
    """30: logits over hundreds apart, pieces of rows on shifts of their own."""
    X, W, y, w = make(70, 900, 128, dtype, seed=9)
    check(X, W, y, None, scale)
    check(X, W, torch.where(y < 0, y, (y + 450) % 900), w, scale)     # targets that the states do not lean to


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_targets_far_below_and_far_above(dtype):
    """Logits of +-2000: the target's the largest (loss 0), the smallest, and in
    between; several pieces with shifts, and the row's on the largest."""
    T, V, d = 6, 700, 64
    W = torch.zeros(V, d)
    W[:, 0] = torch.linspace(-2000, 2000, V).bfloat16().float()
    W[:, 1] = torch.randn(V, generator=torch.Generator().manual_seed(1))
    X = torch.zeros(T, d)
    X[:, 0] = torch.tensor([1.0, 1, 1, -1, -1, 0.5])
    X[:, 1] = 1
    y = torch.tensor([V - 1, 0, V // 2, 0, V - 1, 100], dtype=torch.int32)
    check(X.to(DT[dtype]).cuda(), W.to(DT[dtype]).cuda(), y.cuda(), None)


def test_ignored_tokens():
    X, W, y, w = make(300, 500, 128, "bf16", ignored=0.5)
    w[7] = 0
    X[:20] = float("nan")
    y[:20] = -5
    X[30] = float("inf")
    w[30] = 0
    y[40] = 500                                           # past the vocabulary: its loss is NaN
    y[41] = 2 ** 31 - 1
    loss, dX = check(X, W, y, w)
    assert bool(torch.isnan(loss[40:42]).all()) and not bool(dX[40:42].any())
    assert not bool(loss[:20].any()) and not bool(dX[:20].any()) and not bool(dX[30].any())
    # none at all
    y.fill_(-1)
    loss, dX = run(X, W, y, w)
    assert not bool(loss.any()) and not bool(dX.any())


def test_other_tokens_do_not_change_a_token():
    """Rows give the same whatever is ignored around them, bit for bit."""
    X, W, y, w = make(600, 1030, 128, "bf16", ignored=0.0)
    loss, dX = run(X, W, y, w)
    keep = torch.rand(600, generator=torch.Generator().manual_seed(2)).cuda() < 0.4
    loss2, dX2 = run(X, W, torch.where(keep, y, torch.full_like(y, -1)), w)
    assert torch.equal(loss[keep], loss2[keep]) and torch.equal(dX[keep], dX2[keep])
    assert not bool(loss2[~keep].any()) and not bool(dX2[~keep].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan(dtype):
    X, W, y, w = make(80, 400, 64, dtype, ignored=0.0)
    clean = run(X, W, y, w)
    X[3, 5] = float("nan")
    X[9, 0] = float("inf")
    got = run(X, W, y, w)
    ok = torch.ones(80, dtype=torch.bool, device="cuda")
    ok[[3, 9]] = False
    assert torch.equal(got[0][ok], clean[0][ok]) and torch.equal(got[1][ok], clean[1][ok])
    assert bool(torch.isnan(got[0][~ok]).all()) and bool(torch.isnan(got[1][~ok]).all())
    # vocabulary rows that are switched off: logits of -infinity (X positive there)
    X, W, y, w = make(80, 400, 64, dtype, ignored=0.0)
    X[:, 0] = 1.0
    off = torch.zeros(400, dtype=torch.bool, device="cuda")
    off[[0, 77, 399]] = True
    Wz = W.clone()
    Wz[off, 0] = float("-inf")
    y2 = torch.where(off[y.long()], torch.full_like(y, 5), y)
    loss = run(X, Wz, y2, w, grad=False)[0]
    ref = R.cross_entropy(f64(X), f64(W)[~off.cpu().numpy()],
                          (torch.cumsum((~off).int(), 0) - 1)[y2.long()].cpu().numpy(), f64(w))[0]
    near(loss, ref, 2e-5 * np.abs(ref) + 2e-5)
    # such a row as the target: the loss is infinite
    y2[4] = 77
    assert float(run(X, Wz, y2, w, grad=False)[0][4]) == float("inf")


def test_several_blocks_of_tokens():
    """More tokens than one block's exponentials hold, ignored ones among them;
    the reference by torch in 64 bits on the GPU."""
    T, V, d = 1500, 200001, 64
    X, W, y, w = make(T, V, d, "bf16", ignored=0.1)
    assert B.lora_cross_entropy_workspace_bytes(T, V, d, B.LORA_BF16) < (620 << 20)
    loss, dX = run(X, W, y, w)
    Wd = W.double()
    for t0 in range(0, T, 250):
        r = t0 + torch.nonzero(y[t0:t0 + 250] >= 0)[:, 0]
        L = torch.log_softmax(X[r].double() @ Wd.t(), 1)
        k = torch.arange(r.numel(), device="cuda")
        ref = -w[r].double() * L[k, y[r].long()]
        assert float(((loss[r].double() - ref).abs() / (ref.abs() + 1e-3)).max()) < 1e-4
        P = L.exp()
        g = w[r].double()[:, None] * (P @ Wd - Wd[y[r].long()])
        # every probability off by half a step of bf16 and the float32 sums: to first order of |p W|
        tol = w[r].double()[:, None] * ((2.0 ** -8 + 2e-4) * (P @ Wd.abs()) + 2e-4 * Wd[y[r].long()].abs())
        tol = tol + 2.0 ** -8 * (g.abs() + tol)
        assert bool(((dX[r].double() - g).abs() <= tol).all())
    gone = y < 0
    assert not bool(loss[gone].any()) and not bool(dX[gone].any())


def check_on_gpu(X, W, y, w, loss, dX, tokens):
    """The tokens' results against torch in 64 bits on the GPU, bounds as in `tolerances`."""
    dtype = "bf16" if X.dtype == torch.bfloat16 else "f32"
    (_, d), V, Wd, half = X.shape, W.shape[0], W.double(), HALF[dtype]
    t = tokens[y[tokens] >= 0]
    k, c = torch.arange(t.numel(), device="cuda"), y[t].long()
    L = X[t].double() @ Wd.t()
    e = (d + 8) * EPS * (X[t].double().abs() @ Wd.abs().t()) + 2 * EPS * (L.abs() + L[k, c].abs()[:, None]) + 2.0 ** -22
    P = torch.softmax(L, 1)
    wt = w[t].double()
    ref = -wt * torch.log_softmax(L, 1)[k, c]
    g = wt[:, None] * (P @ Wd - Wd[c])
    P[k, c] = 0
    shift = (P * e).sum(1) + (V + 4) * EPS * P.sum(1)
    assert bool(((loss[t].double() - ref).abs() <= 1.02 * wt * shift + 4 * EPS * ref.abs() + 1e-37).all())
    rel = half + (V + 8) * EPS + shift
    tol = (P * (e + rel[:, None])) @ Wd.abs() + (P.sum(1) * (shift + e.max(1)[0] + rel))[:, None] * Wd[c].abs()
    tol = 1.02 * wt[:, None] * tol
    assert bool(((dX[t].double() - g).abs() <= tol + half * (g.abs() + tol) + 1e-37).all())


def made_on_gpu(T, V, d, dtype, ignored):
    gen = torch.Generator("cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    u = lambda: torch.rand(T, generator=gen, device="cuda")
    W, X = (r(V, d) * d ** -0.5).to(DT[dtype]), (2 * r(T, d)).to(DT[dtype])
    y = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    y[u() < ignored] = -1
    return X, W, y, u() + 0.5


@pytest.mark.parametrize("dtype,T", [("bf16", 40000), ("f32", 33100)])
def test_several_blocks_of_wide_tokens(dtype, T):
    """A small vocabulary under wide states: the blocks hold the sums of dX."""
    V, d = 300, 4096
    assert B.lora_cross_entropy_workspace_bytes(T, V, d, CODE[dtype]) < T * d * 4 < 700 << 20
    X, W, y, w = made_on_gpu(T, V, d, dtype, 0.1)
    loss, dX = run(X, W, y, w)
    for t0 in (0, T // 2 - 500, T - 1000):
        check_on_gpu(X, W, y, w, loss, dX, torch.arange(t0, t0 + 1000, device="cuda"))
    gone = y < 0
    assert not bool(loss[gone].any()) and not bool(dX[gone].any())


@pytest.mark.parametrize("dtype,T,V", [("bf16", 300, 1 << 22), ("f32", 70, (1 << 22) - 5), ("bf16", 1 << 20, 3),
                                       ("f32", 1 << 20, 67), ("bf16", 7, 131077)])
def test_largest_vocabulary_and_most_tokens(dtype, T, V):
    X, W, y, w = made_on_gpu(T, V, 64, dtype, 0.2)
    loss, dX = run(X, W, y, w)
    n = min(T, 1000, (1 << 27) // V)
    for t0 in (0, (T - n) // 2, T - n):
        check_on_gpu(X, W, y, w, loss, dX, torch.arange(t0, t0 + n, device="cuda"))
    gone = y < 0
    assert not bool(loss[gone].any()) and not bool(dX[gone].any())
    torch.cuda.empty_cache()


# tiles of 192 x 256 and 256 x 256 with many splits, few, and none; the last columns a quarter of a tile
@pytest.mark.parametrize("T,V,d", [(130, 20011, 4160), (192, 20011, 8256), (700, 8003, 8256), (1150, 3001, 8256),
                                   (700, 3001, 6208), (250, 32003, 6208), (1000, 8003, 6208), (2000, 1001, 6208)])
def test_second_products_tile_shapes(T, V, d):
    X, W, y, w = made_on_gpu(T, V, d, "bf16", 0.05)
    loss, dX = run(X, W, y, w)
    check_on_gpu(X, W, y, w, loss, dX, torch.arange(T, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_is_the_differences_of_the_loss(dtype):
    X, W, y, w = make(20, 300, 64, "f32", ignored=0.2)
    V = torch.randn_like(X)
    dX = run(X, W, y, w)[1]
    h = 1e-2
    up, dn = (f64(run(X + s * V, W, y, w, grad=False)[0]) for s in (h, -h))
    along = (f64(dX) * f64(V)).sum(1)
    # third derivatives of a log-sum-exp: at most the cube of the logits' spread along V
    spread = np.abs(f64(V) @ f64(W).T).max(1)
    assert np.all(np.abs((up - dn) / (2 * h) - along) <= f64(w) * (h * h * spread ** 3 + 4e-6 / h))


def test_bf16_gradient_is_the_differences_of_a_64_bit_loss():
    X, W, y, w = make(60, 300, 128, "bf16", seed=4, ignored=0.2)
    Xd, Wd, yd, wd = f64(X), f64(W), y.cpu().numpy(), f64(w)
    V = np.random.default_rng(5).standard_normal(Xd.shape)
    dX = f64(run(X, W, y, w)[1])
    h = 1e-4
    up, dn = (R.cross_entropy(Xd + s * V, Wd, yd, wd)[0] for s in (h, -h))
    along, (loss, ref, P) = (dX * V).sum(1), R.cross_entropy(Xd, Wd, yd, wd)
    # dX by element as above; third derivatives of a log-sum-exp are at most the cube of the
    # logits' spread along V; the losses' own 2^-52 over h
    tol = (tolerances(Xd, Wd, yd, wd, 1.0, loss, ref, P, HALF["bf16"])[1] * np.abs(V)).sum(1)
    spread = np.abs(V @ Wd.T).max(1)
    assert np.all(np.abs((up - dn) / (2 * h) - along) <= tol + wd * (h * h * spread ** 3) + 1e-14 * (1 + loss) / h)
    listed = yd >= 0
    assert (np.abs(along[listed]) > 4 * tol[listed]).sum() > 10      # the directions say something


def test_captured_and_beside_another_stream():
    X, W, y, w = make(300, 1100, 128, "bf16")
    ref = [t.clone() for t in run(X, W, y, w)]
    with torch.cuda.stream(torch.cuda.Stream()):
        got = run(X, W, y, w)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    loss, dX = torch.empty(300, device="cuda"), torch.empty_like(X)
    ws = workspace(B.lora_cross_entropy_workspace_bytes(300, 1100, 128, B.LORA_BF16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.lora_cross_entropy(X, W, B.LORA_BF16, 300, 1100, 128, y, w, 1.0, loss, dX, ws)
    y0 = y.clone()
    for k in range(3):
        loss.fill_(3)
        dX.fill_(3)
        y.copy_(torch.where(torch.arange(300, device="cuda") % 3 == 0, torch.full_like(y, -1), y0) if k == 1 else y0)
        graph.replay()
        torch.cuda.synchronize()
        want = run(X, W, y, w)
        assert torch.equal(loss, want[0]) and torch.equal(dX, want[1]), k
