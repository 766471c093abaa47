"""The gated block, the cross entropy, their gradients, the adapters' gradients,
the clipping and the orthogonalised update in a row, as a training step runs
them; and single calls at sizes that take each tile shape and at rows past
32-bit byte offsets."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import training as R
from tests import test_gpu_cross_entropy as CE
from tests import test_gpu_gated as G
from tests.gpu_training_cases import ACTS, CODE, DT, EPS, HALF, Block, f64, near, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


class Step:
    """One training step of a block's two adapted projections under a frozen head."""

    def __init__(self, T, K, d, F, V, dtype, act="silu", seed=0, lo=1, hi=16):
        self.b = b = Block(T, K, d, F, dtype, seed=seed, mask=True, lo=lo, hi=hi)
        rng = np.random.default_rng(seed + 1)
        dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t)
        self.act, self.V = act, V
        self.head = dev(rng.standard_normal((V, F)) * F ** -0.5, DT[dtype])
        y = rng.integers(0, V, size=T).astype(np.int32)
        y[::4] = -1                                           # a prompt's tokens
        self.y, self.w = dev(y, torch.int32), dev(0.5 + rng.random(T), torch.float32)
        self.Wt = [w.t().contiguous() for w in b.W]
        new = lambda *s: torch.zeros(*s, dtype=DT[dtype], device="cuda")
        z = lambda *s: torch.zeros(*s, device="cuda")
        self.H, self.g, self.u, self.dH, self.dg, self.du = (new(T, F) for _ in range(6))
        self.dX, self.loss = new(T, d), z(T)
        self.grads = [(z(b.P, d), z(b.P, F)) for _ in range(2)]
        self.clipped = [(z(b.P, d), z(b.P, F)) for _ in range(2)]
        self.momentum = [(z(b.P, d), z(b.P, F)) for _ in range(2)]
        self.adapters = torch.arange(b.N, dtype=torch.int32, device="cuda")
        self.norm = z(b.N + 1)
        self.layers = B.GradLayers([(p, *g, *c) for p, g, c in zip(b.pools, self.grads, self.clipped)])
        code = CODE[dtype]
        self.ws_loss = workspace(B.lora_cross_entropy_workspace_bytes(T, V, F, code))
        self.ws_gated = workspace(B.lora_gated_grad_workspace_bytes(T, K, d, F, b.R, code))
        self.ws_grad = workspace(B.lora_grad_workspace_bytes(T, K, b.N, d, F, b.R, code))
        self.ws_clip = workspace(B.lora_clip_grad_workspace_bytes(self.layers, b.N, b.R))
        self.ws_orth = workspace(B.lora_orthogonal_step_workspace_bytes(b.N, b.R, d, F))

    def gradients(self):
        b = self.b
        b.forward(self.act, self.H, self.g, self.u)
        B.lora_cross_entropy(self.H, self.head, CODE[b.dtype], b.T, self.V, b.F, self.y, self.w, 1.0, self.loss,
                             self.dH, self.ws_loss)
        B.lora_gated_grad(self.dH, self.g, self.u, ACTS[self.act], *self.Wt, b.d_mask, b.keep, b.T, b.K, b.d_gates,
                          *b.pools, b.plan, b.R, self.dg, self.du, self.dX, self.ws_gated)
        for p, dY in enumerate((self.dg, self.du)):
            B.lora_grad(b.X, b.d_mask, b.keep, dY, b.T, b.K, b.d_gates, b.pools[p], b.plan, b.ws[p], *self.grads[p],
                        b.R, self.ws_grad)

    def update(self):
        b = self.b
        B.lora_clip_grad(self.layers, self.adapters, b.N, b.R, 0.05, False, self.norm, self.ws_clip)
        for p in range(2):
            f = [B.FactorUpdate(pages, c, m, None, 0.02) for pages, c, m in
                 zip((b.A[p], b.Bp[p]), self.clipped[p], self.momentum[p])]
            B.lora_orthogonal_step(b.pools[p], self.adapters, b.N, b.R, *f, 0.9, False, 3, B.NS_COEF, 1e-7,
                                   self.ws_orth)

    def run(self):
        self.gradients()
        self.update()

    def state(self):
        return [*self.b.A, *self.b.Bp] + [m for pair in self.momentum for m in pair]

    def outputs(self):
        return [self.H, self.loss, self.dH, self.dg, self.du, self.dX, self.norm] + self.state()


@pytest.mark.parametrize("T,K,d,F,V,dtype", [(24, 2, 64, 128, 97, "f32"), (150, 1, 128, 192, 300, "bf16")])
def test_each_stage_against_64_bits(T, K, d, F, V, dtype):
    s = Step(T, K, d, F, V, dtype, seed=3)
    s.run()
    torch.cuda.synchronize()
    b = Block(T, K, d, F, dtype, seed=3, mask=True, lo=1, hi=16)       # the pages before the update
    for got, (ref, tol), what in zip((s.H, s.g, s.u), G.expected(b, s.act), "Hgu"):
        near(got, ref, tol, what)
    X, W, y, w = f64(s.H), f64(s.head), s.y.cpu().numpy(), f64(s.w)
    loss, dH, P = R.cross_entropy(X, W, y, w, 1.0)
    tl, tx = CE.tolerances(X, W, y, w, 1.0, loss, dH, P, HALF[dtype])
    near(s.loss, loss, tl, "loss")
    near(s.dH, dH, tx, "dH")
    (rg, tg), (ru, tu) = G.grad_tolerances(b, s.act, f64(s.g), f64(s.u), f64(s.dH))
    near(s.dg, rg, tg, "d_gate")
    near(s.du, ru, tu, "d_up")
    near(s.dX, *G.expected_dx(b, f64(s.dg), f64(s.du), s.Wt), "dX")
    host = [dict(rank=b.rank, page_start=b.start, page_ids=b.page_ids, n_pages=b.P, A=f64(a), B=f64(c))
            for a, c in s.grads]
    norm, out, _ = R.clip(host, list(range(b.N)), b.R, float(np.float32(0.05)), False)
    near(s.norm, norm, np.abs(norm) * (2.0 ** -24 + 2.0 ** -40) + 1e-45, "norm")
    assert (norm[:-1] > 0.05).any()
    for o, c in zip(out, s.clipped):
        for f, got in zip("AB", c):
            pages = b.page_ids
            near(got[pages.astype(np.int64)], o[f][pages], np.abs(o[f][pages]) * (2.0 ** -23 + 2.0 ** -40) + 2.0 ** -149, f)


@pytest.mark.parametrize("act", list(ACTS))
def test_gradients_are_the_differences_of_the_loss(act):
    """float32: the adapters' gradients of the whole chain along a direction against
    central differences of a 64-bit loss."""
    T, K, d, F, V = 24, 2, 64, 128, 97
    s = Step(T, K, d, F, V, "f32", act, seed=5)
    b = s.b
    s.gradients()
    torch.cuda.synchronize()
    X, W, head, w, y = f64(b.X), [f64(x) for x in b.W], f64(s.head), f64(s.w), s.y.cpu().numpy()
    m = b.mask.astype(np.float64)
    A, Bp = [f64(a) for a in b.A], [f64(x) for x in b.Bp]
    rng = np.random.default_rng(9)
    VA, VB = ([rng.standard_normal(x.shape) for x in q] for q in (A, Bp))

    def forward(h):
        y_ = []
        for p in range(2):
            o = X @ W[p].T
            for t, pages, c in b.slots(p):
                o[t] += (c * ((A[p] + h * VA[p])[pages] @ (X[t] * m[t]))) @ (Bp[p] + h * VB[p])[pages]
            y_.append(o)
        H = R.activation(act, y_[0])[0] * y_[1]
        return y_[0], y_[1], H, R.cross_entropy(H, head, y, w, 1.0)

    h = 1e-4
    diff = (forward(h)[3][0].sum() - forward(-h)[3][0].sum()) / (2 * h)
    got = sum((f64(ga) * VA[p]).sum() + (f64(gb) * VB[p]).sum() for p, (ga, gb) in enumerate(s.grads))
    # The same chain of absolute values: a stage's sums of n terms are off by n 2^-24 of it, what
    # they hand on by as much again, and the probabilities by the logits' error, (F + 8) 2^-24
    # times at most `most`.  Slopes are at most 1.13, |act(g)| at most |g|.
    g, u, H, (_, _, P) = forward(0.0)
    most = (np.abs(H) @ np.abs(head).T).max()
    listed = y >= 0
    dHa = np.where(listed, w, 0)[:, None] * (P @ np.abs(head) + np.abs(head)[np.maximum(y, 0)])
    size = 0.0
    for p, da in enumerate((1.13 * dHa * np.abs(u), dHa * np.abs(g))):
        for t, pages, c in b.slots(p):
            z = np.abs(X[t] * m[t])
            size += abs(c) * ((np.abs(A[p][pages]) @ z) @ (np.abs(VB[p][pages]) @ da[t]))
            size += abs(c) * ((np.abs(Bp[p][pages]) @ da[t]) @ (np.abs(VA[p][pages]) @ z))
    n = 2 * (d + F + V + b.R + T + 64) * (1 + most)
    assert abs(got - diff) < n * EPS * size + 1e-6 * abs(diff)
    assert abs(diff) > 1e-4 * size                      # the direction says something


@pytest.mark.parametrize("T,K,d,F,V,dtype", [(5, 1, 64, 192, 130, "bf16"), (200, 2, 128, 320, 513, "bf16"),
                                             (70, 2, 128, 192, 200, "f32")])
def test_captured_steps_are_the_eager_ones(T, K, d, F, V, dtype):
    """Three steps of a captured graph, the program's own work between them,
    against three eager ones, bit for bit."""
    s = Step(T, K, d, F, V, dtype, seed=8)
    start = [t.clone() for t in s.state()]
    s.run()                                              # (libraries and kernels loaded)
    want = []
    for t, o in zip(s.state(), start):
        t.copy_(o)
    for _ in range(3):
        s.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.outputs()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t, o in zip(s.state(), start):
        t.copy_(o)
    other = Step(T, K, d, F, V, dtype, seed=21)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want[i])), i
        other.run()
    assert not torch.equal(want[0][7], want[1][7])       # the pages moved


# ---------------------------------------------------------------- tile shapes

# (forward of a block) tiles of 128 x 128, 128 x 256, 192 x 256 and 256 x 256
@pytest.mark.parametrize("T,F", [(130, 64), (200, 8256), (300, 11008), (500, 11008)])
@pytest.mark.parametrize("K,d", [(1, 64), (2, 192)])
def test_forward_tile_shapes(T, F, K, d):
    G.check_forward(Block(T, K, d, F, seed=T + K, lo=0, hi=20, mask=K == 2), "silu")


# slots whose terms are kept apart (up to 4, where the workspace has the room) and
# slots taken one after another
@pytest.mark.parametrize("T,K,d,F,dtype", [(200, 2, 1600, 448, "bf16"), (200, 4, 2688, 192, "bf16"), (150, 2, 64, 320, "bf16"),
                                           (140, 5, 1600, 192, "bf16"), (70, 4, 576, 192, "f32"), (70, 8, 576, 192, "f32"),
                                           (70, 2, 64, 192, "f32")])
def test_slots_together_and_in_turn(T, K, d, F, dtype):
    b = Block(T, K, d, F, dtype, seed=T + K, lo=0, hi=12, mask=True)
    G.check_forward(b, "silu")
    G.check_grad(b, "silu")


def test_many_float32_tokens():
    """More windows of 16 pairs than one dimension of a grid holds."""
    T, d, F = 600000, 64, 64
    b = Block(1000, 1, d, F, "f32", seed=12, mask=True)
    n = T // b.T
    ids, gates, mask = b.d_ids.repeat(n, 1), b.d_gates.repeat(n, 1), b.d_mask.repeat(n, 1)
    X = b.X.repeat(n, 1)
    plan = workspace(B.lora_plan_bytes(T, 1, b.N))
    ws = [workspace(B.lora_apply_workspace_bytes(T, 1, d, F, b.R, B.LORA_F32)) for _ in range(2)]
    H = torch.full((T, F), 7.0, device="cuda")
    B.lora_gated_forward(ids, gates, T, 1, X, *b.W, 0, H, None, None, mask, b.keep, *b.pools, plan, *ws)
    torch.cuda.synchronize()
    ref, tol = G.expected(b, "silu")[0]
    for i in (0, n // 2, n - 1):
        near(H[i * b.T:(i + 1) * b.T], ref, tol, i)
    assert torch.equal(H.view(n, b.T, F)[0].expand(n, -1, -1).reshape(T, F), H)


@pytest.mark.parametrize("T,V", [(100, 200), (200, 16500), (300, 22020), (500, 22020)])
def test_cross_entropy_tile_shapes(T, V):
    CE.check(*CE.make(T, V, 64, "bf16", seed=T, ignored=0.1))


@pytest.mark.parametrize("T,N,dtype", [(200, 6000, "bf16"), (150, 1500, "f32")])
def test_forward_of_more_adapters_than_fit_beside_the_product(T, N, dtype):
    """The plan's tables of so many adapters do not fit the product's LDS: a launch of its own."""
    G.check_forward(Block(T, 2, 64, 192, dtype, N=N, lo=0, hi=3, seed=N), "gelu")


# ---------------------------------------------------------------- rows past 2^32 bytes

FAR_T, FAR_D = 33000, 65600
FAR_ROWS = [0, 1, 127, 16384, 32639, 32735, 32736, 32800, 32998, 32999]


def far_rows(n, dtype=torch.bfloat16):
    """[FAR_T][n], zero but for FAR_ROWS."""
    x = torch.zeros(FAR_T, n, dtype=dtype, device="cuda")
    x[FAR_ROWS] = torch.randn(len(FAR_ROWS), n, generator=torch.Generator("cuda").manual_seed(n), device="cuda").to(dtype)
    return x


class FarBlock(Block):
    """A block over FAR_ROWS; the oracle sees those alone."""

    def __init__(self, d, F):
        super().__init__(len(FAR_ROWS), 1, d, F, seed=2, lo=1, hi=8, empty=False)
        ids = torch.full((FAR_T, 1), -1, dtype=torch.int32, device="cuda")
        ids[FAR_ROWS] = self.d_ids
        self.far_ids, self.far_gates = ids, torch.ones(FAR_T, 1, device="cuda")
        self.plan = workspace(B.lora_plan_bytes(FAR_T, 1, self.N))


def test_forward_of_rows_past_32_bits():
    b = FarBlock(FAR_D, 64)
    X = far_rows(FAR_D)
    b.X.copy_(X[FAR_ROWS])
    H, g, u = (torch.full((FAR_T, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ws = [workspace(B.lora_apply_workspace_bytes(FAR_T, 1, FAR_D, 64, b.R, B.LORA_BF16)) for _ in range(2)]
    B.lora_gated_forward(b.far_ids, b.far_gates, FAR_T, 1, X, *b.W, 0, H, g, u, None, 1.0, *b.pools, b.plan, *ws)
    torch.cuda.synchronize()
    for got, (ref, tol), what in zip((H, g, u), G.expected(b, "silu"), "Hgu"):
        near(got[FAR_ROWS], ref, tol, what)
        rest = torch.ones(FAR_T, dtype=torch.bool, device="cuda")
        rest[FAR_ROWS] = False
        assert not bool(got[rest].any())


def test_gradient_of_rows_past_32_bits():
    b = FarBlock(64, FAR_D)
    dH, g, u = far_rows(FAR_D), far_rows(FAR_D), far_rows(FAR_D)
    g.mul_(0.5)
    W = [w.t().contiguous() for w in b.W]
    dg, du = torch.empty_like(dH), torch.empty_like(dH)
    dX = torch.full((FAR_T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace(B.lora_gated_grad_workspace_bytes(FAR_T, 1, 64, FAR_D, b.R, B.LORA_BF16))
    B.lora_plan(b.far_ids, b.far_gates, FAR_T, 1, b.pools[0], b.plan)
    B.lora_gated_grad(dH, g, u, 0, *W, None, 1.0, FAR_T, 1, b.far_gates, *b.pools, b.plan, b.R, dg, du, dX, ws)
    torch.cuda.synchronize()
    b.dH.copy_(dH[FAR_ROWS])
    (rg, tg), (ru, tu) = G.grad_tolerances(b, "silu", f64(g[FAR_ROWS]), f64(u[FAR_ROWS]), f64(dH[FAR_ROWS]))
    near(dg[FAR_ROWS], rg, tg, "d_gate")
    near(du[FAR_ROWS], ru, tu, "d_up")
    near(dX[FAR_ROWS], *G.expected_dx(b, f64(dg[FAR_ROWS]), f64(du[FAR_ROWS]), W), "dX")
    rest = torch.ones(FAR_T, dtype=torch.bool, device="cuda")
    rest[FAR_ROWS] = False
    assert not bool(dX[rest].any())


def test_cross_entropy_of_rows_past_32_bits():
    V = 130
    X = far_rows(FAR_D)
    W = torch.randn(V, FAR_D, generator=torch.Generator("cuda").manual_seed(4), device="cuda").mul_(FAR_D ** -0.5).bfloat16()
    y = torch.full((FAR_T,), -1, dtype=torch.int32, device="cuda")
    y[FAR_ROWS] = torch.arange(len(FAR_ROWS), dtype=torch.int32, device="cuda") * 13
    loss, dX = torch.full((FAR_T,), 7.0, device="cuda"), torch.full_like(X, 7.0)
    ws = workspace(B.lora_cross_entropy_workspace_bytes(FAR_T, V, FAR_D, B.LORA_BF16))
    B.lora_cross_entropy(X, W, B.LORA_BF16, FAR_T, V, FAR_D, y, None, 1.0, loss, dX, ws)
    torch.cuda.synchronize()
    Xd, Wd, yd = f64(X[FAR_ROWS]), f64(W), y[FAR_ROWS].cpu().numpy()
    ref, rx, P = R.cross_entropy(Xd, Wd, yd, None, 1.0)
    tl, tx = CE.tolerances(Xd, Wd, yd, None, 1.0, ref, rx, P, HALF["bf16"])
    near(loss[FAR_ROWS], ref, tl, "loss")
    near(dX[FAR_ROWS], rx, tx, "dX")
    rest = torch.ones(FAR_T, dtype=torch.bool, device="cuda")
    rest[FAR_ROWS] = False
    assert not bool(loss[rest].any()) and not bool(dX[rest].any())


def test_more_elements_than_one_grid_dimension_has_threads():
    """2^20 tokens of 32832: d_gate and d_up in place."""
    T, F = 1 << 20, 32832
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 215 << 30:
        pytest.skip("needs 215 GB of device memory")
    b = Block(1, 1, 64, F, seed=3)
    rows = [0, 524287, T // 2 + 3, T - 2, T - 1]
    dH = torch.zeros(T, F, dtype=torch.bfloat16, device="cuda")
    g, u = torch.ones_like(dH), torch.ones_like(dH)
    for i, r in enumerate(rows):
        for x in (dH, g, u):
            x[r] = torch.randn(F, generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16()
    was = [f64(x[rows]) for x in (g, u, dH)]
    plan = workspace(B.lora_plan_bytes(T, 1, b.N))
    B.lora_gated_grad(dH, g, u, 0, None, None, None, 1.0, T, 1, None, *b.pools, plan, b.R, g, u, None, None)
    torch.cuda.synchronize()
    (rg, tg), (ru, tu) = G.grad_tolerances(b, "silu", *was)
    near(g[rows], rg, tg, "d_gate")
    near(u[rows], ru, tu, "d_up")
    # 0 . u . act'(1) and 0 . act(1) where dH is 0
    for x in (g, u):
        x[rows] = 0
        for i in range(0, T, 1 << 16):
            assert not bool(x[i:i + (1 << 16)].any()), i
    del dH, g, u, x
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- no room for U

@pytest.mark.parametrize("T,K,d,F,dtype", [(5, 1, 128, 192, "bf16"), (200, 2, 1600, 448, "bf16"), (300, 1, 128, 448, "bf16"),
                                           (4200, 1, 128, 1984, "bf16"), (70, 2, 576, 192, "f32")])
@pytest.mark.parametrize("which", [0, 1])
def test_without_room_for_u_the_base_alone(T, K, d, F, dtype, which):
    """One projection's workspace too small for U, or max_rank below the ranks:
    the plan says so and the results are the base products'."""
    b = Block(T, K, d, F, dtype, seed=6, lo=12, hi=16, empty=False)
    small = workspace(B.lora_apply_workspace_bytes(T, K, d, F, 1, CODE[dtype]))
    full = [w.numel() for w in b.ws]
    assert small.numel() < full[0]
    b.ws[which] = small
    H = b.out(F)
    b.forward("silu", H.t)
    torch.cuda.synchronize()
    H.check()
    assert int(b.plan.view(torch.int32)[B.PH_ERR]) & B.DEVERR_CAPACITY
    pairs, b.ids = b.ids, np.full_like(b.ids, -1)
    ref, tol = G.expected(b, "silu")[0]
    near(H.t, ref, tol, "H")
    b.ids = pairs
    g, u = torch.randn_like(b.dH), torch.randn_like(b.dH)
    W = [w.t().contiguous() for w in b.W]
    B.lora_plan(b.d_ids, b.d_gates, T, K, b.pools[0], b.plan)
    assert int(b.plan.view(torch.int32)[B.PH_ERR]) == 0
    b.R = 1
    dg, du, dx = G.run_grad(b, "silu", g, u, W)
    assert int(b.plan.view(torch.int32)[B.PH_ERR]) & B.DEVERR_CAPACITY
    b.ids = np.full_like(b.ids, -1)
    near(dx, *G.expected_dx(b, f64(dg), f64(du), W), "dX")


# ---------------------------------------------------------------- infinities and NaN in pages

@pytest.mark.parametrize("T,K,d,F,dtype", [(5, 2, 128, 192, "bf16"), (150, 2, 64, 320, "bf16"), (200, 2, 1600, 448, "bf16"),
                                           (4200, 2, 128, 1984, "bf16"), (70, 2, 576, 192, "f32"), (70, 5, 128, 192, "f32")])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_pages_that_are_not_finite_stay_with_their_rows(T, K, d, F, dtype, value):
    """Another adapter's rows keep their bits; the adapter's own rows are what float
    arithmetic makes of them, in g, u and dX."""
    b = Block(T, K, d, F, dtype, seed=T + 1, lo=1, hi=12)
    bad = 2
    pages = torch.from_numpy(b.page_ids[b.start[bad]:b.start[bad + 1]].astype(np.int64)).cuda()
    W = [w.t().contiguous() for w in b.W]
    torch.manual_seed(T)
    g0, u0 = torch.randn_like(b.dH), torch.randn_like(b.dH)

    def run():
        _, g, u = G.run_forward(b, "silu")
        return g.clone(), u.clone(), G.run_grad(b, "silu", g0, u0, W)[2].clone()

    clean = run()
    for p in range(2):
        b.Bp[p][pages[0], 5::7] = value
        b.A[p][pages[-1], 3::11] = value
    got = run()
    own = torch.from_numpy(((b.ids == bad) & (b.gates != 0)).any(1)).cuda()
    assert bool(own.any()) and bool((~own).any())
    for a, c, what in zip(got, clean, ("g", "u", "dX")):
        assert torch.equal(a[~own], c[~own]), what
        # G = d.B is not finite for the adapter's pairs, and so is U = X.A: all its columns
        assert not bool(torch.isfinite(a[own]).all(1).any()), what


# ---------------------------------------------------------------- values that are not finite, by kind and place

def signs(v, value):
    """What v . value adds to a finite sum: an infinity's sign, NaN; 0 where |v| is too
    near 0 for its sign to be known in float32."""
    if np.isnan(value):
        return np.full(v.shape, np.nan)
    return np.sign(v) * np.sign(value)


def check_kinds(got, clean, rows, cols, want, what):
    """got equals clean bit for bit but at (rows, cols), where it is want . inf (NaN: NaN)."""
    at = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    at[torch.from_numpy(rows).cuda()[:, None], torch.from_numpy(cols).cuda()] = True
    assert torch.equal(got[~at], clean[~at]), what
    have = f64(got)[rows][:, cols]
    want = np.broadcast_to(want[:, None], have.shape)
    assert not np.isfinite(have).any(), what
    nan = np.isnan(want)
    assert np.isnan(have[nan]).all(), what
    known = ~nan & (want != 0)
    assert np.array_equal(have[known], want[known] * np.inf), what


def own_rows(b, bad, p):
    """The tokens with pairs of adapter `bad`, and those pairs' coefficients added up
    (gates and scales are positive)."""
    rows = np.flatnonzero(((b.ids == bad) & (b.gates != 0)).any(1))
    c = (b.gates * (b.ids == bad)).sum(1)[rows] * float(b.scale[p][bad]) * b.keep
    return rows, c


VALUES = [float("inf"), float("-inf"), float("nan")]


# one slot and several; decode, terms apart and in turn, tiles with ranks up to 16 and past it
@pytest.mark.parametrize("T,K,d,F,dtype,hi", [(5, 1, 128, 192, "bf16", 12), (5, 2, 128, 192, "bf16", 40),
                                              (150, 1, 64, 320, "bf16", 40), (200, 2, 1600, 448, "bf16", 12),
                                              (140, 5, 1600, 192, "bf16", 20), (4200, 1, 128, 1984, "bf16", 12),
                                              (4200, 1, 128, 1984, "bf16", 40), (4200, 2, 128, 1984, "bf16", 20),
                                              (70, 1, 576, 192, "f32", 12), (70, 2, 576, 192, "f32", 40),
                                              (70, 5, 128, 192, "f32", 20)])
@pytest.mark.parametrize("value", VALUES)
def test_b_pages_that_are_not_finite(T, K, d, F, dtype, hi, value):
    b = Block(T, K, d, F, dtype, seed=T + hi, lo=max(1, hi - 6), hi=hi, N=4)
    bad, cols = 2, np.arange(5, F, 37)
    clean = [t.clone() for t in G.run_forward(b, "silu")]
    j = int(b.rank[bad]) - 1
    page = int(b.page_ids[b.start[bad] + j])
    for p in range(2):
        b.Bp[p][page, torch.from_numpy(cols).cuda()] = value
    got = G.run_forward(b, "silu")
    for p, what in enumerate("gu"):
        rows, c = own_rows(b, bad, p)
        assert 0 < rows.size < T
        z, a = f64(b.X)[rows], f64(b.A[p])[page]
        U = c * (z @ a)
        U[np.abs(U) < (d + 8) * EPS * c * (np.abs(z) @ np.abs(a))] = 0
        check_kinds(got[1 + p], clean[1 + p], rows, cols, signs(U, value), what)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[torch.from_numpy(rows).cuda()] = False
    assert torch.equal(got[0][keep], clean[0][keep])


# the split product with terms apart and in turn, whole tiles
@pytest.mark.parametrize("T,K,d,F,dtype,hi", [(5, 1, 128, 192, "bf16", 12), (150, 2, 64, 320, "bf16", 40),
                                              (200, 2, 1600, 448, "bf16", 12), (140, 5, 1600, 192, "bf16", 20),
                                              (8200, 1, 1536, 64, "bf16", 12), (8200, 1, 1536, 64, "bf16", 40),
                                              (12400, 2, 960, 64, "bf16", 20), (70, 1, 576, 192, "f32", 12),
                                              (70, 2, 576, 192, "f32", 40), (70, 5, 128, 192, "f32", 20)])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("value", VALUES)
def test_a_pages_that_are_not_finite(T, K, d, F, dtype, hi, which, value):
    b = Block(T, K, d, F, dtype, seed=T + hi, lo=max(1, hi - 6), hi=hi, N=4)
    bad, cols = 2, np.arange(5, d, 37)
    W = [w.t().contiguous() for w in b.W]
    gen = torch.Generator("cuda").manual_seed(T)
    g, u = (torch.randn(T, F, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    B.lora_plan(b.d_ids, b.d_gates, T, K, b.pools[0], b.plan)
    clean = [t.clone() for t in G.run_grad(b, "silu", g, u, W)]
    j = int(b.rank[bad]) - 1
    page = int(b.page_ids[b.start[bad] + j])
    b.A[which][page, torch.from_numpy(cols).cuda()] = value
    got = G.run_grad(b, "silu", g, u, W)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    rows, c = own_rows(b, bad, which)
    assert 0 < rows.size < T
    z, a = f64(got[which])[rows], f64(b.Bp[which])[page]
    C = c * (z @ a)
    C[np.abs(C) < (F + 8) * EPS * c * (np.abs(z) @ np.abs(a))] = 0
    check_kinds(got[2], clean[2], rows, cols, signs(C, value), "dX")


# ---------------------------------------------------------------- the forward's whole tiles

def whole(b):
    """Whether the forward takes tiles that finish themselves: 256 or more of 256 x 256, and then
    nothing lies before U in the workspace."""
    return B.lora_apply_u_offset(b.T, b.K, b.d, b.F, CODE[b.dtype]) == 0


@pytest.mark.parametrize("T,K,d,F,hi,runs", [(257, 1, 64, 32576, 16, False), (300, 2, 128, 32576, 16, False),
                                             (500, 1, 64, 32576, 70, True), (400, 1, 192, 32576, 33, False),
                                             (511, 3, 64, 32576, 40, True), (300, 8, 64, 32576, 12, False),
                                             (3841, 1, 128, 3904, 16, True), (3900, 2, 64, 3904, 24, False)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward_of_whole_tiles(T, K, d, F, hi, runs, act):
    b = Block(T, K, d, F, seed=T + hi, lo=0, hi=hi, runs=runs, N=9, mask=T % 2 == 1)
    assert whole(b)
    G.check_forward(b, act, stored=act == "silu")


@pytest.mark.parametrize("K,hi", [(1, 12), (1, 40), (2, 20)])
@pytest.mark.parametrize("value", VALUES)
def test_b_pages_that_are_not_finite_in_whole_tiles(K, hi, value):
    b = Block(300, K, 64, 32576, seed=hi, lo=hi - 6, hi=hi, N=4)
    assert whole(b)
    test_b_pages_that_are_not_finite(300, K, 64, 32576, "bf16", hi, value)


@pytest.mark.parametrize("K", [1, 2])
def test_whole_tiles_of_plan_then_apply_and_captured(K):
    """lora_gated_apply on lora_plan's plan, and a captured forward replayed beside other
    work, against lora_gated_forward, bit for bit; U of both where lora_grad finds it."""
    T, d, F = 300, 128, 32576
    b = Block(T, K, d, F, seed=5, mask=True, hi=20)
    assert whole(b)
    one = [t.clone() for t in G.run_forward(b, "silu")]
    n = 4 * int(B.lora_plan_header(b.plan)[B.PH_RPAIRS])
    u = [w[:n].clone() for w in b.ws]
    B.lora_plan(b.d_ids, b.d_gates, T, K, b.pools[0], b.plan)
    H, g, up = b.out(F), b.out(F), b.out(F)
    B.lora_gated_apply(b.X, *b.W, ACTS["silu"], H.t, g.t, up.t, T, K, b.d_gates, b.d_mask, b.keep, *b.pools, b.plan,
                       *b.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((H.t, g.t, up.t), one))
    assert all(torch.equal(x, w[:n]) for x, w in zip(u, b.ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward("silu", H.t, g.t, up.t)
    other = Block(T, K, d, F, seed=6)
    for _ in range(3):
        for o in (H, g, up):
            o.t.zero_()
        G.run_forward(other, "gelu")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((H.t, g.t, up.t), one))


def test_whole_tiles_of_tokens_without_adapters():
    """Tokens without an active slot equal the base product's, wherever they lie; and all of them."""
    b = Block(500, 1, 64, 32576, seed=2, N=5)
    assert whole(b)
    H = G.run_forward(b, "silu")[0].clone()
    idle = torch.from_numpy(np.flatnonzero((b.ids[:, 0] < 0) | (b.rank[np.maximum(b.ids[:, 0], 0)] == 0))).cuda()
    b.ids[:] = -1
    b.d_ids.fill_(-1)
    base = G.run_forward(b, "silu")[0]
    assert idle.numel() > 20 and torch.equal(H[idle], base[idle])
    G.check_forward(b, "silu")


@pytest.mark.parametrize("which", [0, 1])
def test_whole_tiles_without_room_for_u(which):
    assert B.lora_apply_u_offset(300, 1, 64, 32576, B.LORA_BF16) == 0
    b = Block(300, 1, 64, 32576, seed=6, lo=12, hi=16, empty=False)
    b.ws[which] = workspace(B.lora_apply_workspace_bytes(300, 1, 64, 32576, 1, B.LORA_BF16))
    H = G.run_forward(b, "silu")[0]
    assert int(b.plan.view(torch.int32)[B.PH_ERR]) & B.DEVERR_CAPACITY
    b.ids = np.full_like(b.ids, -1)
    near(H, *G.expected(b, "silu")[0], "H")


# ---------------------------------------------------------------- adapters that share pages

class NestedBlock(Block):
    """The pages of adapter 0 are the first of adapter 2's, or the other way round (1, between
    them, is no adapter: its page_start is not consistent, and no token names it); adapter 3
    has some of them too."""

    def __init__(self, T, K, d, F, dtype, r0, r2, seed):
        top, low = max(r0, r2), min(r0, r2)
        super().__init__(T, K, d, F, dtype, N=4, lo=top, hi=top, seed=seed, mask=True)
        self.rank[:] = (r0, 1, r2, low)
        self.start[:] = (0, r0, 0, r2, r2 + low)
        self.ids[self.ids == 1] = 2
        for t, a in ((self.d_rank, self.rank), (self.d_start, self.start), (self.d_ids, self.ids)):
            t.copy_(torch.from_numpy(a))


@pytest.mark.parametrize("T,K,d,F,dtype,r0,r2", [(5, 2, 128, 192, "bf16", 12, 5), (200, 2, 1600, 448, "bf16", 30, 7),
                                                 (140, 5, 1600, 192, "bf16", 12, 5), (300, 1, 64, 32576, "bf16", 12, 9),
                                                 (300, 1, 64, 32576, "bf16", 9, 12), (300, 1, 64, 32576, "bf16", 40, 33),
                                                 (300, 2, 64, 32576, "bf16", 12, 5), (300, 2, 64, 32576, "bf16", 40, 9),
                                                 (70, 2, 576, 192, "f32", 30, 7)])
def test_forward_of_adapters_that_share_pages(T, K, d, F, dtype, r0, r2):
    G.check_forward(NestedBlock(T, K, d, F, dtype, r0, r2, seed=T + r0), "silu")


@pytest.mark.parametrize("T,K,d,F,dtype,r0,r2", [(5, 2, 128, 192, "bf16", 12, 5), (200, 2, 1600, 448, "bf16", 30, 7),
                                                 (8200, 1, 1536, 64, "bf16", 9, 12), (8200, 1, 1536, 64, "bf16", 40, 33),
                                                 (12400, 2, 960, 64, "bf16", 12, 5), (70, 2, 576, 192, "f32", 30, 7)])
def test_gradient_of_adapters_that_share_pages(T, K, d, F, dtype, r0, r2):
    G.check_grad(NestedBlock(T, K, d, F, dtype, r0, r2, seed=T + r0), "silu")


# ---------------------------------------------------------------- the shrinks' forms

# big segments (512 pairs or more, widths of multiples of 128) beside units in one launch or in two,
# units whose rows stay in registers or not; sums of more than 4 and 8 splits
@pytest.mark.parametrize("T,K,d,F,dtype,N", [(600, 1, 128, 128, "bf16", 3), (520, 2, 4096, 128, "bf16", 5),
                                             (600, 1, 4224, 128, "bf16", 3), (530, 2, 6144, 128, "bf16", 30),
                                             (600, 1, 6272, 128, "bf16", 3), (200, 1, 4160, 64, "bf16", 6),
                                             (200, 1, 6208, 64, "bf16", 6), (5, 1, 9280, 128, "bf16", 3),
                                             (100, 2, 6208, 192, "bf16", 6), (70, 1, 2112, 64, "f32", 4),
                                             (70, 2, 1984, 128, "f32", 4)])
@pytest.mark.parametrize("mask", [False, True])
def test_forward_of_wide_rows(T, K, d, F, dtype, N, mask):
    b = Block(T, K, d, F, dtype, N=N, seed=d, mask=mask, lo=0, hi=20)
    G.check_forward(b, "silu")
    # the same by a plan that is there: the shrinks of its order, at decode sizes too
    one = [t.clone() for t in G.run_forward(b, "silu")]
    B.lora_plan(b.d_ids, b.d_gates, T, K, b.pools[0], b.plan)
    H, g, u = b.out(F), b.out(F), b.out(F)
    B.lora_gated_apply(b.X, *b.W, ACTS["silu"], H.t, g.t, u.t, T, K, b.d_gates, b.d_mask, b.keep, *b.pools, b.plan, *b.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x.t, y) for x, y in zip((H, g, u), one))


@pytest.mark.parametrize("T,K,d,F,dtype,N", [(600, 1, 128, 128, "bf16", 3), (520, 2, 128, 4096, "bf16", 5),
                                             (600, 1, 128, 4224, "bf16", 3), (530, 2, 128, 6144, "bf16", 30),
                                             (600, 1, 128, 6272, "bf16", 3), (200, 1, 64, 4160, "bf16", 6),
                                             (200, 1, 64, 6208, "bf16", 6), (8200, 1, 1536, 128, "bf16", 4),
                                             (70, 1, 64, 2112, "f32", 4), (70, 2, 128, 1984, "f32", 4)])
@pytest.mark.parametrize("mask", [False, True])
def test_gradient_of_wide_rows(T, K, d, F, dtype, N, mask):
    G.check_grad(Block(T, K, d, F, dtype, N=N, seed=F, mask=mask, lo=0, hi=20), "silu")


# ---------------------------------------------------------------- ranks and pools at their ends

@pytest.mark.parametrize("T,K,d,F,dtype,N,lo,hi", [(5, 2, 64, 192, "bf16", 3, 1000, 1024), (150, 2, 64, 192, "bf16", 3, 500, 1024),
                                                   (200, 2, 1600, 448, "bf16", 1, 257, 257), (257, 1, 64, 32576, "bf16", 2, 100, 130),
                                                   (257, 2, 64, 32576, "bf16", 1, 33, 33), (70, 2, 128, 192, "f32", 2, 700, 1024),
                                                   (40, 8, 64, 64, "bf16", 1, 1, 1), (8200, 1, 1536, 64, "bf16", 3, 100, 130)])
def test_large_ranks_and_one_adapter(T, K, d, F, dtype, N, lo, hi):
    b = Block(T, K, d, F, dtype, N=N, lo=lo, hi=hi, seed=hi, mask=True)
    if T < 8000:
        G.check_forward(b, "silu")
    if F < 10000:
        G.check_grad(b, "silu")


@pytest.mark.parametrize("T,d,F,dtype", [(5, 128, 192, "bf16"), (200, 128, 192, "bf16"), (300, 64, 32576, "bf16"),
                                         (8200, 1536, 64, "bf16"), (70, 64, 64, "f32")])
def test_pools_without_pages(T, d, F, dtype):
    """Every rank 0 and no page at all: the base products."""
    b = Block(T, 2, d, F, dtype, N=3, lo=0, hi=0, seed=T)
    t = DT[dtype]
    none = [torch.empty(0, n, dtype=t, device="cuda") for n in (d, F)]
    b.pools = [B.Pool(CODE[dtype], d, F, *none, b.d_rank, b.d_start, b.d_page_ids[:0], p.tensors[5]) for p in b.pools]
    assert b.pools[0].desc.n_pages == 0 and not b.pools[0].desc.a_pages
    if T < 8000:
        G.check_forward(b, "silu")
    if F < 10000:
        G.check_grad(b, "silu")


@pytest.mark.parametrize("T,K,d,F,dtype", [(5, 2, 128, 192, "bf16"), (100, 2, 4224, 128, "bf16"), (600, 1, 128, 256, "bf16"),
                                           (300, 2, 64, 32576, "bf16"), (70, 2, 128, 192, "f32")])
def test_the_forwards_plan_serves_later_calls(T, K, d, F, dtype):
    """lora_gated_apply, lora_apply, lora_gated_grad and lora_grad on the plan that
    lora_gated_forward built, against lora_plan's, bit for bit."""
    b = Block(T, K, d, F, dtype, seed=T, mask=True, hi=20)
    W = [w.t().contiguous() for w in b.W]
    gen = torch.Generator("cuda").manual_seed(3)
    g0, u0 = (torch.randn(T, F, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    Y = torch.empty_like(b.dH)
    dA, dB = torch.zeros(b.P, d, device="cuda"), torch.zeros(b.P, F, device="cuda")
    ws = workspace(B.lora_grad_workspace_bytes(T, K, b.N, d, F, b.R, CODE[dtype]))

    def later():
        H, g, u = b.out(F), b.out(F), b.out(F)
        B.lora_gated_apply(b.X, *b.W, ACTS["silu"], H.t, g.t, u.t, T, K, b.d_gates, b.d_mask, b.keep, *b.pools, b.plan,
                           *b.ws)
        dg, du, dx = G.run_grad(b, "silu", g0, u0, W)
        B.lora_apply(b.X, b.W[1], Y, T, K, b.d_gates, b.d_mask, b.keep, b.pools[1], b.plan, b.ws[1])
        B.lora_grad(b.X, b.d_mask, b.keep, dg, T, K, b.d_gates, b.pools[0], b.plan, b.ws[0], dA, dB, b.R, ws)
        torch.cuda.synchronize()
        return [t.clone() for t in (H.t, g.t, u.t, dg, du, dx, Y, dA, dB)]

    first = G.run_forward(b, "silu")
    got = later()
    assert all(torch.equal(x, y) for x, y in zip(first, got))
    B.lora_plan(b.d_ids, b.d_gates, T, K, b.pools[0], b.plan)
    assert all(torch.equal(x, y) for x, y in zip(later(), got))
