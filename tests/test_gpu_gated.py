"""The gated feed-forward block and its backward on the GPU against 64 bits.

Tolerances, per element (e_g, e_u: what a float32 sum in any order and the bf16
split of U may lose, see Block.projection):
  * the activations' slopes are at most 1.13, so act(g) is off by 1.13 e_g,
    and by its own evaluation: the exponential's argument z is rounded a few
    times (its size times 2^-24 each), exponential and reciprocal are within 2
    steps: (4 |z| + 32) 2^-23 relative, twice that for 1 - p;
  * one rounding of the result, half a step.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import training as R
from tests.gpu_training_cases import ACTS, CODE, DT, EPS, HALF, Block, Guarded, f64, near, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def eval_error(act, g):
    """Relative error of act(g)'s own evaluation."""
    return (4 * np.abs(R.activation(act, g)[2]) + 32) * 2.0 ** -23


def expected(b, act):
    (g, eg), (u, eu) = b.projection(0), b.projection(1)
    a, _, _ = R.activation(act, g)
    H, half = a * u, HALF[b.dtype]
    eH = (1.13 * eg + np.abs(a) * eval_error(act, g) + 1e-37) * (np.abs(u) + eu) + np.abs(a) * eu
    return [(H, eH + half * (np.abs(H) + eH)), (g, eg + half * (np.abs(g) + eg)), (u, eu + half * (np.abs(u) + eu))]


def run_forward(b, act, stored=True):
    H, g, u = b.out(b.F), b.out(b.F), b.out(b.F)
    b.forward(act, H.t, g.t if stored else None, u.t if stored else None)
    torch.cuda.synchronize()
    for o in (H, g, u):
        o.check()
    return (H.t, g.t, u.t) if stored else (H.t,)


def check_forward(b, act, stored=True):
    for got, (ref, tol), what in zip(run_forward(b, act, stored), expected(b, act), "Hgu"):
        near(got, ref, tol, what)


def grad_tolerances(b, act, g, u, dH):
    a, slope, z = R.activation(act, g)
    rel = (4 * np.abs(z) + 32) * 2.0 ** -23
    # the slope's terms: p, and x p (1 - p) z' of at most 1 + |z|
    e_slope = rel * (1 + np.abs(z) * np.minimum(1, np.exp(-np.minimum(np.abs(z), 700)) * 4)) * 2
    half = HALF[b.dtype]
    dg, du = dH * u * slope, dH * a
    eg, eu = np.abs(dH * u) * e_slope + 1e-37, np.abs(du) * rel + 1e-37
    return (dg, eg + (half + 3 * EPS) * (np.abs(dg) + eg)), (du, eu + (half + 3 * EPS) * (np.abs(du) + eu))


def expected_dx(b, dg, du, W):
    """dX of the given d_gate, d_up, and its tolerance."""
    y, e = 0, 0
    m = 1.0 if b.mask is None else b.mask.astype(np.float64)
    for p, d in enumerate((dg, du)):
        A, Bp, w = f64(b.A[p]), f64(b.Bp[p]), f64(W[p])
        y = y + d @ w.T
        e = e + (2 * b.F + 8) * EPS * (np.abs(d) @ np.abs(w).T)
        for t, pages, c in b.slots(p):
            mk = 1.0 if b.mask is None else m[t]
            G, Ga = c * (Bp[pages] @ d[t]), abs(c) * (np.abs(Bp[pages]) @ np.abs(d[t]))
            y[t] += mk * (G @ A[pages])
            e[t] += mk * ((b.F + 8 + 2 * pages.size) * EPS * (Ga @ np.abs(A[pages])) +
                          2.0 ** -16 * (np.abs(G) @ np.abs(A[pages])))
    return y, e + HALF[b.dtype] * (np.abs(y) + e)


def run_grad(b, act, g, u, W, dX=True, stream=None):
    dg, du, dx = b.out(b.F), b.out(b.F), b.out(b.d)
    ws = workspace(B.lora_gated_grad_workspace_bytes(b.T, b.K, b.d, b.F, b.R, CODE[b.dtype]))
    B.lora_gated_grad(b.dH, g, u, ACTS[act], *(W if dX else (None, None)), b.d_mask, b.keep, b.T, b.K, b.d_gates,
                      *b.pools, b.plan, b.R, dg.t, du.t, dx.t if dX else None, ws, stream)
    torch.cuda.synchronize()
    for o in (dg, du, dx):
        o.check()
    return dg.t, du.t, dx.t


def check_grad(b, act, dX=True):
    torch.manual_seed(7)
    g = (torch.randn(b.T, b.F, device="cuda") * 2).to(DT[b.dtype])
    u = torch.randn(b.T, b.F, device="cuda").to(DT[b.dtype])
    W = [w.t().contiguous() for w in b.W]
    B.lora_plan(b.d_ids, b.d_gates, b.T, b.K, b.pools[0], b.plan)
    dg, du, dx = run_grad(b, act, g, u, W, dX)
    (rg, tg), (ru, tu) = grad_tolerances(b, act, f64(g), f64(u), f64(b.dH))
    near(dg, rg, tg, "d_gate")
    near(du, ru, tu, "d_up")
    if dX:
        near(dx, *expected_dx(b, f64(dg), f64(du), W), "dX")
    else:
        assert bool((dx.view(torch.uint8) == 0x6b).all())


# ---------------------------------------------------------------- forward

# decode, split K, stream-K and tiles; odd tokens and widths (odd multiples of 64)
FORMS = [(1, 1, 64, 64), (1, 2, 576, 704), (2, 1, 4096, 192), (33, 8, 128, 320), (128, 1, 192, 1088),
         (129, 2, 704, 448), (257, 1, 1024, 1344), (600, 2, 640, 2240), (300, 1, 64, 16448), (4200, 1, 128, 1984)]


@pytest.mark.parametrize("T,K,d,F", FORMS)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward_bf16(T, K, d, F, act):
    check_forward(Block(T, K, d, F, seed=T + F, mask=T % 2 == 1, lo=0, hi=16), act)


@pytest.mark.parametrize("T,K,d,F", [(1, 1, 64, 64), (5, 3, 192, 320), (130, 1, 576, 704), (333, 2, 128, 192)])
@pytest.mark.parametrize("act", list(ACTS))
def test_forward_f32(T, K, d, F, act):
    check_forward(Block(T, K, d, F, "f32", seed=T, mask=T % 2 == 1, lo=0, hi=20), act)


@pytest.mark.parametrize("T,K,d,F,hi,runs", [(4200, 2, 64, 1984, 40, False), (4200, 1, 64, 1984, 70, True),
                                             (4111, 1, 64, 2048, 16, True), (300, 3, 64, 16448, 33, True)])
def test_forward_tiles_of_ranks_and_slots(T, K, d, F, hi, runs):
    """Ranks past 16 and several slots in the tiles' own passes; blocks of one
    adapter and of many."""
    check_forward(Block(T, K, d, F, seed=hi, lo=1, hi=hi, runs=runs, N=9), "gelu", stored=False)


@pytest.mark.parametrize("T,F", [(1, 192), (200, 448), (4200, 1984)])
def test_plan_then_apply_is_the_forward(T, F):
    b = Block(T, 2, 128, F, seed=5, mask=True)
    one = run_forward(b, "silu")
    plan, u = b.plan.clone(), [w.clone() for w in b.ws]
    B.lora_plan(b.d_ids, b.d_gates, b.T, b.K, b.pools[0], b.plan)
    H, g, up = b.out(F), b.out(F), b.out(F)
    B.lora_gated_apply(b.X, *b.W, ACTS["silu"], H.t, g.t, up.t, T, 2, b.d_gates, b.d_mask, b.keep, *b.pools, b.plan,
                       *b.ws)
    torch.cuda.synchronize()
    for x, y in zip(one, (H.t, g.t, up.t)):
        assert torch.equal(x, y)
    # U of both where lora_grad finds it
    at = B.lora_apply_u_offset(T, 2, 128, F, CODE["bf16"])
    n = 4 * int(B.lora_plan_header(b.plan)[B.PH_RPAIRS])
    for x, y in zip(u, b.ws):
        assert torch.equal(x[at:at + n], y[at:at + n])


def test_rows_without_adapters_are_the_base_alone():
    b = Block(4200, 1, 64, 1984, seed=2)
    H = run_forward(b, "silu", stored=False)[0]
    b.d_ids.fill_(-1)
    base = run_forward(b, "silu", stored=False)[0]
    rows = torch.from_numpy(np.flatnonzero((b.ids < 0).all(1) | (b.rank[np.maximum(b.ids[:, 0], 0)] == 0))).cuda()
    assert rows.numel() > 100 and torch.equal(H[rows], base[rows])


@pytest.mark.parametrize("T,F", [(64, 192), (300, 320), (4200, 1984)])
def test_other_rows_are_isolated(T, F):
    """Infinities and NaN of one adapter's factors and of one token reach that
    adapter's rows and that token alone."""
    b = Block(T, 1, 64, F, seed=3, lo=2, hi=16, N=5)
    clean = run_forward(b, "silu")
    bad = 2
    page = int(b.page_ids[b.start[bad]])
    b.Bp[0][page, 5] = float("inf")
    b.Bp[1][page, 7] = float("nan")
    tok = int(np.flatnonzero(b.ids[:, 0] != bad)[1])
    b.X[tok, 3] = float("nan")
    got = run_forward(b, "silu")
    rows = torch.from_numpy((b.ids[:, 0] == bad)).cuda()
    rows[tok] = True
    for x, y in zip(got, clean):
        assert torch.equal(x[~rows], y[~rows])
    H, g, u = got
    mine = torch.from_numpy(np.flatnonzero(b.ids[:, 0] == bad)).cuda()
    assert bool(torch.isnan(u[mine, 7]).all()) and bool((~torch.isfinite(g[mine, 5])).all())
    others = [c for c in range(F) if c not in (5, 7)]
    for x, y in zip(got, clean):
        assert torch.equal(x[mine][:, others], y[mine][:, others])
    assert bool(torch.isnan(g[tok]).all()) and bool(torch.isnan(H[tok]).all())


def test_no_tokens():
    b = Block(1, 1, 64, 64)
    H = b.out(64)
    z = b.X[:0]
    B.lora_gated_forward(b.d_ids, b.d_gates, 0, 1, z, *b.W, 0, H.t[:0], None, None, None, 1.0, *b.pools, b.plan, *b.ws)
    torch.cuda.synchronize()
    H.check()
    assert bool((H.t.view(torch.uint8) == 0x6b).all())


# ---------------------------------------------------------------- backward

@pytest.mark.parametrize("T,K,d,F", [(1, 1, 64, 64), (17, 2, 192, 320), (128, 1, 576, 704), (129, 2, 448, 704),
                                     (300, 1, 320, 1024), (700, 2, 576, 1984), (8200, 1, 1536, 64), (12400, 2, 960, 64)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_grad_bf16(T, K, d, F, act):
    check_grad(Block(T, K, d, F, seed=T, mask=T % 2 == 1 or T > 8000, lo=0, hi=16 if T % 200 else 24, runs=T > 10000),
               act)


@pytest.mark.parametrize("T,K,d,F", [(1, 1, 64, 64), (130, 2, 192, 320), (333, 1, 576, 704)])
@pytest.mark.parametrize("act", list(ACTS))
def test_grad_f32(T, K, d, F, act):
    check_grad(Block(T, K, d, F, "f32", seed=T, mask=T % 2 == 1, lo=0, hi=20), act)


def test_grad_without_dx_and_in_place():
    b = Block(65, 1, 128, 192, seed=4)
    check_grad(b, "gelu", dX=False)
    W = [w.t().contiguous() for w in b.W]
    B.lora_plan(b.d_ids, b.d_gates, b.T, b.K, b.pools[0], b.plan)
    g, u = torch.randn(65, 192, device="cuda").bfloat16(), torch.randn(65, 192, device="cuda").bfloat16()
    apart = run_grad(b, "silu", g, u, W)
    dx = b.out(128)
    ws = workspace(B.lora_gated_grad_workspace_bytes(65, 1, 128, 192, b.R, B.LORA_BF16))
    B.lora_gated_grad(b.dH, g, u, 0, *W, None, 1.0, 65, 1, b.d_gates, *b.pools, b.plan, b.R, g, u, dx.t, ws)
    torch.cuda.synchronize()
    for x, y in zip((g, u, dx.t), apart):
        assert torch.equal(x, y)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad_of_far_arguments(act, dtype):
    """Arguments at which the exponentials over- and underflow: no NaN, and the
    limits of both slopes."""
    b = Block(2, 1, 64, 64, dtype, empty=False)
    B.lora_plan(b.d_ids, b.d_gates, b.T, b.K, b.pools[0], b.plan)
    v = torch.tensor([0.0, -0.0, 1e-30, 12.5, 60, 88.5, 90, 130, 1e4, 1e18, 1e30, 3e38] * 6)[:64]
    g = torch.stack([v, -v]).to(DT[dtype]).cuda()
    u = torch.ones(2, 64, device="cuda", dtype=DT[dtype])
    W = [w.t().contiguous() for w in b.W]
    dg, du, _ = run_grad(b, act, g, u, W, dX=False)
    dH = f64(b.dH)
    big = np.abs(f64(g)) > 20
    with np.errstate(over="ignore"):
        near(f64(dg)[big], np.where(f64(g) > 0, dH, 0.0)[big], (np.abs(dH) * (HALF[dtype] + 1e-5) + 1e-7)[big])
        ref = np.clip(dH * np.maximum(f64(g), 0.0), -np.inf, np.inf)
        fit = big & (np.abs(ref) < 3e38)
        near(f64(du)[fit], ref[fit], (np.abs(ref) * (2 * HALF[dtype] + 1e-5) + 1e-4)[fit])


def test_gradients_are_the_differences_of_the_forward():
    """fp32: <dH, H> of the block moved along a direction of X, against dX."""
    b = Block(40, 2, 128, 192, "f32", seed=11, mask=True, hi=8)
    _, g, u = run_forward(b, "gelu_tanh")
    W = [w.t().contiguous() for w in b.W]
    _, _, dx = run_grad(b, "gelu_tanh", g, u, W)
    V, X, h = torch.randn_like(b.X), b.X.clone(), 2e-3
    got = []
    for s in (h, -h):
        b.X.copy_(X + s * V)
        got.append((f64(run_forward(b, "gelu_tanh", stored=False)[0]) * f64(b.dH)).sum())
    diff, along = (got[0] - got[1]) / (2 * h), (f64(dx) * f64(V)).sum()
    # central differences are off by h^2 / 6 of the third derivative, the sums by 2^-24 of their terms over h
    size = np.abs(f64(dx) * f64(V)).sum()
    assert abs(diff - along) < 2e-3 * size


# ---------------------------------------------------------------- streams and graphs

@pytest.mark.parametrize("T,F", [(3, 192), (300, 448), (4200, 1984)])
def test_captured_and_beside_another_stream(T, F):
    b = Block(T, 1, 128, F, seed=6, mask=True)
    W = [w.t().contiguous() for w in b.W]
    H, g, u = (torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dg, du, dx = torch.empty_like(H), torch.empty_like(H), torch.empty_like(b.X)
    ws = workspace(B.lora_gated_grad_workspace_bytes(T, 1, 128, F, b.R, B.LORA_BF16))

    def step(stream=None):
        b.forward("silu", H, g, u, stream)
        B.lora_gated_grad(b.dH, g, u, 0, *W, b.d_mask, b.keep, T, 1, b.d_gates, *b.pools, b.plan, b.R, dg, du, dx, ws,
                          stream)

    outs = (H, g, u, dg, du, dx)
    step()
    torch.cuda.synchronize()
    ref = [o.clone() for o in outs]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    with torch.cuda.graph(graph):
        step()
    X2 = b.X.flip(0).contiguous()
    for k in range(3):
        for o in outs:
            o.zero_()
        b.X.copy_(X2 if k == 1 else X2.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        if k != 1:
            assert all(torch.equal(o, r) for o, r in zip(outs, ref)), k
        else:
            got = [o.clone() for o in outs]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(o, r) for o, r in zip(outs, got)), k


@pytest.mark.parametrize("T,F", [(3, 192), (200, 448), (4200, 1984)])
def test_buffers_that_touch(T, F):
    """All of a call's larger buffers one behind the other, without a byte between."""
    b = Block(T, 2, 128, F, seed=9, mask=True)
    ref = [t.clone() for t in run_forward(b, "silu")]
    W = [w.t().contiguous() for w in b.W]
    ref += [t.clone() for t in run_grad(b, "silu", ref[1], ref[2], W)]
    one = torch.full((sum(t.numel() * t.element_size() for t in ref) + b.X.numel() * 2 + sum(w.numel() for w in b.ws)
                      + b.plan.numel() + B.lora_gated_grad_workspace_bytes(T, 2, 128, F, b.R, B.LORA_BF16),), 0x77,
                     dtype=torch.uint8, device="cuda")
    at = 0

    def take(n):
        nonlocal at
        at += n
        return one[at - n:at]

    rows = lambda n: take(2 * T * n).view(torch.bfloat16).view(T, n)
    H, X, g, u = rows(F), rows(128), rows(F), rows(F)
    X.copy_(b.X)
    b.X = X
    dg, ws, du, dX = rows(F), [take(w.numel()) for w in b.ws], rows(F), rows(128)
    back = take(B.lora_gated_grad_workspace_bytes(T, 2, 128, F, b.R, B.LORA_BF16))
    b.plan = take(b.plan.numel())
    assert at == one.numel()
    b.forward("silu", H, g, u, ws=ws)
    B.lora_gated_grad(b.dH, g, u, 0, *W, b.d_mask, b.keep, T, 2, b.d_gates, *b.pools, b.plan, b.R, dg, du, dX, back)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((H, g, u, dg, du, dX), ref))
