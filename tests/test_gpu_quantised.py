"""The layer over an 8-bit base weight on the GPU against the 64-bit oracle.

Codes and scale bytes are compared bit for bit.  Products carry, per element,
  * one rounding of the output: 2^-8 of it (bf16) or 2^-24 (fp32);
  * fp32 sums in any order: n terms are off by at most n 2^-24 of the sum of
    their magnitudes;
  * bf16 layers: the 8-bit MFMA aligns an instruction's products to the
    largest and drops what lies below 2^-14 of it, so a block of 128 loses at
    most 128 x 2^-14 of (largest |x^|) x (largest |w^|) of the block;
  * bf16 layers with the expand in the GEMM's epilogue: U is split into two
    bf16 words, off by less than 2^-16 of each |U B| (and G, for dX).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from lora_adapter_amd import device as D
from lora_adapter_amd import workloads as wl
from oracle import lora_oracle as O
from oracle import quantised as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


def dt_of(w):
    return B.LORA_BF16 if w.dtype == "bf16" else B.LORA_F32


def workload(T, K, d_in, d_out, dtype="bf16", N=12, lo=2, hi=16, seed=3, mask=False, runs=False, empty=True):
    rng = np.random.default_rng(seed)
    rank = rng.integers(lo, hi + 1, size=N).astype(np.int32)
    if runs:
        ids = np.sort(rng.integers(0, N, size=(T, K)), axis=0).astype(np.int32)
    else:
        ids = rng.integers(0, N, size=(T, K)).astype(np.int32)
    if empty:
        ids[rng.random((T, K)) < 0.1] = -1
        ids[min(3, T - 1)] = -1                       # a row without any adapter
    gates = np.ones((T, K), np.float32) if K == 1 else rng.random((T, K)).astype(np.float32)
    return wl.build("q", seed, dtype, T, K, d_in, d_out, rank, ids, gates, x_var=1.0, w_var=0.02,
                    a_var=1 / 64, b_var=0.02, keep_p=0.9 if mask else None, with_dY=True,
                    scale=(0.5 + rng.random(N)).astype(np.float32))


class Layer(D.DeviceLayer):
    def __init__(self, w):
        super().__init__(w)
        self.W8 = B.QuantisedWeight.empty(w.d_out, w.d_in)
        for t in (self.W8.q_t, self.W8.scale, self.W8.q, self.W8.scale_t):
            t.fill_(0x5a)
        B.lora_quantise_weight(self.W_t, dt_of(w), self.W8)
        n = B.lora_apply_quantised_workspace_bytes(w.T, w.K, w.d_in, w.d_out, self.max_rank, dt_of(w))
        self.ws = torch.full((n,), 0x77, dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        B.lora_forward_quantised(self.ids, self.gates, self.T, self.K, self.X, self.W8, self.Y,
                                 self.keep_mask, self.keep_scale, self.pool, self.plan, self.ws, stream)

    def backward(self, stream=None):
        w = self.w
        dA, dB, gws = self.grad_buffers()
        self.run_grad(dA, dB, gws, stream)
        dX = torch.full((w.T, w.d_in), float("nan"), dtype=self.Y.dtype, device="cuda")
        xws = torch.full((B.lora_grad_x_quantised_workspace_bytes(w.T, w.d_in, w.d_out, dt_of(w)),), 0x77,
                         dtype=torch.uint8, device="cuda")
        B.lora_grad_x_quantised(self.dY, self.W8, self.keep_mask, w.T, w.K, self.pool, self.plan, gws,
                                self.max_rank, dX, xws, stream)
        return dA, dB, dX


def terms(w):
    """Per (token, slot): adapter pages' rows, gate x scale x keep."""
    for t in range(w.T):
        for k in range(w.K):
            a = int(w.ids[t, k])
            if a < 0 or w.rank[a] == 0 or w.gates[t, k] == 0:
                continue
            p = w.page_ids[w.page_start[a]:w.page_start[a + 1]]
            yield t, p, float(w.gates[t, k]) * float(w.scale[a]) * (w.keep_scale if w.keep_mask is not None else 1.0)


def product(x8, w8):
    """x^ w^T, and the most its fp32 sum may be off for bf16 and fp32 layers."""
    y = x8 @ w8.T
    mag = np.abs(x8) @ np.abs(w8).T
    n = x8.shape[1]
    lost = 128 * 2.0 ** -14 * (Q.block_amax(x8) @ Q.block_amax(w8).T)
    return y, n * 2.0 ** -24 * mag + lost, n * 2.0 ** -24 * mag


def expected(w):
    """Y and dX with the error each element may have."""
    X, dY = D.as_f64(w.X), D.as_f64(w.dY)
    A, Bp = D.as_f64(w.a_pages), D.as_f64(w.b_pages)
    m = np.ones_like(X) if w.keep_mask is None else w.keep_mask.astype(np.float64)
    W8 = Q.weight_values(*Q.quantise_weight(D.as_f64(w.W_t)), w.d_in)
    out = []
    for rows, wt, side in ((X, W8, 0), (dY, W8.T.copy(), 1)):
        y, eb, ef = product(Q.row_values(*Q.quantise_rows(rows), rows.shape[1]), wt)
        e = eb if w.dtype == "bf16" else ef
        for t, p, c in terms(w):
            if side == 0:
                z, dn, up, mk = X[t] * m[t], A[p], Bp[p], 1.0
            else:
                z, dn, up, mk = dY[t], Bp[p], A[p], m[t]
            u, ua = c * (dn @ z), abs(c) * (np.abs(dn) @ np.abs(z))
            y[t] += mk * (u @ up)
            # U itself is a sum of d terms and two roundings of its coefficient; then r more terms
            e[t] += (z.size + 4 + p.size) * 2.0 ** -24 * (ua @ np.abs(up)) + 2.0 ** -16 * (np.abs(u) @ np.abs(up))
        half = 2.0 ** (-8 if w.dtype == "bf16" else -24)
        out += [y, e + half * (np.abs(y) + e)]
    return out


def check(got, ref, tol, what):
    off = np.abs(D.as_f64(D.to_host(got)) - ref)
    assert np.all(off <= tol), (what, float(np.max(off / tol)))


# ---------------------------------------------------------------- codes

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 64), (3, 128), (5, 192), (7, 576), (33, 1344)])
def test_rows_bit_exact(T, d, dtype):
    rng = np.random.default_rng(T * d)
    x = (rng.standard_normal((T, d)) * 10.0 ** rng.uniform(-6, 6, (T, 1))).astype(np.float32)
    x[0, :64] = 0                                     # a block of zeros when d = 64
    if T > 2:
        x[1, :128] = np.linspace(-448, 448, 128)      # values on and between codes
        x[2] *= 1e-38                                 # fp32 subnormals
    x = wl.f32_to_bf16_bits(x) if dtype == "bf16" else x
    X = D.to_device(x, "cuda")
    c = torch.full((T, B.lora_quantised_row_bytes(d)), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((T, B.lora_quantised_scale_bytes(d)), 0x55, dtype=torch.uint8, device="cuda")
    B.lora_quantise_rows(X, B.LORA_BF16 if dtype == "bf16" else B.LORA_F32, T, d, c, s)
    v, sb = Q.quantise_rows(D.as_f64(x))
    assert np.array_equal(c.view(torch.float8_e4m3fn).float().cpu().numpy(), v)
    assert np.array_equal(s.cpu().numpy()[:, :sb.shape[1]], sb)
    assert not s[:, sb.shape[1]:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("o,i", [(64, 64), (128, 192), (704, 576), (320, 1344)])
def test_weight_bit_exact_in_both_orientations(o, i, dtype):
    rng = np.random.default_rng(o + i)
    W = (rng.standard_normal((o, i)) * 10.0 ** rng.uniform(-3, 3, (o, 1))).astype(np.float32)
    W[:, :64] *= 1e-3
    W = wl.f32_to_bf16_bits(W) if dtype == "bf16" else W
    w = B.QuantisedWeight.empty(o, i)
    for t in (w.q_t, w.q, w.scale, w.scale_t):
        t.fill_(0x55)
    B.lora_quantise_weight(D.to_device(W, "cuda"), B.LORA_BF16 if dtype == "bf16" else B.LORA_F32, w)
    v, s = Q.quantise_weight(D.as_f64(W))
    f = lambda t: t.view(torch.float8_e4m3fn).float().cpu().numpy()
    assert np.array_equal(f(w.q_t), v)
    assert np.array_equal(f(w.q)[:, :o], v.T[:i]) and not w.q[:, o:].any()
    assert np.array_equal(w.scale.cpu().numpy()[:, :s.shape[1]], s) and not w.scale[:, s.shape[1]:].any()
    assert np.array_equal(w.scale_t.cpu().numpy()[:, :s.shape[0]], s.T) and not w.scale_t[:, s.shape[0]:].any()
    # one orientation alone
    w1 = B.QuantisedWeight.empty(o, i, both=False)
    B.lora_quantise_weight(D.to_device(W, "cuda"), B.LORA_BF16 if dtype == "bf16" else B.LORA_F32, w1)
    assert torch.equal(w1.q_t, w.q_t) and torch.equal(w1.scale, w.scale)


def test_non_finite_blocks():
    x = np.ones((2, 256), np.float32)
    x[0, 5], x[1, 200] = np.inf, np.nan
    c = torch.zeros(2, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 4, dtype=torch.uint8, device="cuda")
    B.lora_quantise_rows(torch.from_numpy(x).cuda(), B.LORA_F32, 2, 256, c, s)
    nan = torch.isnan(c.view(torch.float8_e4m3fn).float()).cpu().numpy()
    assert nan[0, :128].all() and not nan[0, 128:].any() and nan[1, 128:].all() and not nan[1, :128].any()
    assert s.cpu().numpy()[:, :2].tolist() == [[255, s[0, 1].item()], [s[1, 0].item(), 255]]


# ---------------------------------------------------------------- the layer

CASES = [  # T, K, d_in, d_out, dtype, extra
    (1, 1, 64, 64, "bf16", {}),
    (1, 1, 1088, 576, "bf16", {}),
    (1, 2, 512, 256, "f32", {}),
    (17, 8, 192, 320, "bf16", {"lo": 1, "hi": 5}),
    (33, 1, 576, 704, "f32", {"mask": True}),
    (64, 1, 1024, 512, "bf16", {"mask": True}),
    (128, 2, 640, 192, "bf16", {}),
    (129, 1, 576, 704, "bf16", {"mask": True}),
    (130, 2, 1344, 320, "f32", {"mask": True, "hi": 40}),
    (300, 2, 640, 1344, "bf16", {"mask": True}),
    (515, 1, 192, 4160, "bf16", {"runs": True, "hi": 80}),
    (1100, 1, 2112, 1088, "bf16", {"runs": True}),
]


@pytest.mark.parametrize("T,K,d_in,d_out,dtype,extra", CASES)
def test_forward_and_backward(T, K, d_in, d_out, dtype, extra):
    w = workload(T, K, d_in, d_out, dtype, **extra)
    L = Layer(w)
    L.forward()
    dA, dB, dX = L.backward()
    torch.cuda.synchronize()
    y, ty, x, tx = expected(w)
    check(L.Y, y, ty, "Y")
    check(dX, x, tx, "dX")
    # the gradients of the factors come from the same plan and U as over a bf16 weight
    L2 = D.DeviceLayer(w)
    L2.run_plan()
    L2.run_apply()
    dA2, dB2, g2 = L2.grad_buffers()
    L2.run_grad(dA2, dB2, g2)
    assert torch.equal(dA.nan_to_num(7), dA2.nan_to_num(7)) and torch.equal(dB.nan_to_num(7), dB2.nan_to_num(7))


@pytest.mark.parametrize("T,d_in,d_out,runs,K,hi", [(4096, 192, 4096, True, 1, 16), (3900, 320, 4160, False, 1, 16),
                                                    (4096, 128, 4096, False, 2, 40),
                                                    (1030, 256, 1536, True, 1, 70)])
def test_fused_tiles(T, d_in, d_out, runs, K, hi):
    """Enough 256 x 256 tiles for the epilogue in the GEMM, forward; the
    backward of the mirrored layer fills them too.  Ranks below, at and over
    the 16 rows of a pass, one slot per token and two."""
    w = workload(T, K, d_in, d_out, N=9, hi=hi, mask=True, runs=runs)
    L = Layer(w)
    L.forward()
    torch.cuda.synchronize()
    y, ty, _, _ = expected(w)
    check(L.Y, y, ty, "Y")
    w = workload(T, K, d_out, d_in, N=9, hi=hi, mask=True, runs=runs)
    L = Layer(w)
    L.forward()
    _, _, dX = L.backward()
    torch.cuda.synchronize()
    _, _, x, tx = expected(w)
    check(dX, x, tx, "dX")


@pytest.mark.parametrize("T,dtype", [(5, "bf16"), (200, "bf16"), (9, "f32")])
def test_forward_is_plan_then_apply_and_repeats(T, dtype):
    w = workload(T, 2, 576, 704, dtype)
    L = Layer(w)
    L.forward()
    Y, U = L.Y.clone(), L.U()
    plan = L.read_plan()
    L.Y.fill_(float("nan"))
    L.ws.fill_(0x11)
    L.run_plan()
    B.lora_apply_quantised(L.X, L.W8, L.Y, L.T, L.K, L.gates, L.keep_mask, L.keep_scale, L.pool, L.plan, L.ws)
    torch.cuda.synchronize()
    assert torch.equal(L.Y, Y) and np.array_equal(L.U(), U)
    for k, v in L.read_plan().items():
        if k != "header":
            assert np.array_equal(v, plan[k]), k


def test_rows_without_adapters_are_the_base_product():
    w = workload(40, 2, 576, 704)
    L = Layer(w)
    L.forward()
    Y = L.Y.clone()
    L.gates.zero_()                                    # every slot off
    L.forward()
    torch.cuda.synchronize()
    off = (w.ids < 0).all(axis=1)
    assert off.any() and torch.equal(L.Y[off], Y[off]) and not torch.equal(L.Y, Y)


def test_nan_row_stays_its_own():
    w = workload(20, 1, 256, 256)
    L = Layer(w)
    L.forward()
    Y = L.Y.clone()
    L.X[7, 130] = float("inf")
    L.gates.zero_()
    L.forward()
    base = L.Y.clone()
    torch.cuda.synchronize()
    assert torch.isnan(base[7]).all() and torch.isfinite(base[:7]).all() and torch.isfinite(base[8:]).all()


def test_an_empty_batch():
    w = workload(4, 1, 128, 128)
    L = Layer(w)
    L.Y.fill_(3)
    B.lora_apply_quantised(L.X, L.W8, L.Y, 0, 1, L.gates, None, 1.0, L.pool, L.plan, L.ws)
    torch.cuda.synchronize()
    assert (L.Y == 3).all()


@pytest.mark.parametrize("T", [3, 150])
def test_another_stream_and_a_graph(T):
    w = workload(T, 1, 576, 704, mask=True)
    L = Layer(w)
    L.forward()
    _, _, dX = L.backward()
    Y, dX = L.Y.clone(), dX.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    dA, dB, gws = L.grad_buffers()
    dX2 = torch.empty_like(dX)
    xws = torch.empty(B.lora_grad_x_quantised_workspace_bytes(w.T, w.d_in, w.d_out, dt_of(w)),
                      dtype=torch.uint8, device="cuda")

    def work():
        L.forward()
        L.run_grad(dA, dB, gws)
        B.lora_grad_x_quantised(L.dY, L.W8, L.keep_mask, w.T, w.K, L.pool, L.plan, gws, L.max_rank, dX2, xws)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    s.synchronize()
    assert torch.equal(L.Y, Y) and torch.equal(dX2, dX)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for i in range(3):
        L.Y.zero_()
        dX2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.Y, Y) and torch.equal(dX2, dX), i


def test_canaries_around_every_output():
    w = workload(150, 2, 576, 704, mask=True)
    L = Layer(w)
    pad = 4096
    ybuf = torch.full((w.T * w.d_out + 2 * pad,), 5.0, dtype=torch.bfloat16, device="cuda")
    L.Y = ybuf[pad:-pad].view(w.T, w.d_out)
    n = L.ws.numel()
    wbuf = torch.full((n + 2 * pad,), 0x3c, dtype=torch.uint8, device="cuda")
    L.ws = wbuf[pad:-pad]
    L.forward()
    torch.cuda.synchronize()
    assert (ybuf[:pad] == 5).all() and (ybuf[-pad:] == 5).all()
    assert (wbuf[:pad] == 0x3c).all() and (wbuf[-pad:] == 0x3c).all()
    y, ty, _, _ = expected(w)
    check(L.Y, y, ty, "Y")


def test_rows_of_more_than_32_bits():
    """2^20 rows of 65 chunks: more threads than one grid dimension holds, and
    byte offsets past 32 bits."""
    T, d = 1 << 20, 32832
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GB of device memory")
    X = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    c = torch.full((T, B.lora_quantised_row_bytes(d)), 0x5a, dtype=torch.uint8, device="cuda")
    s = torch.full((T, B.lora_quantised_scale_bytes(d)), 0x5a, dtype=torch.uint8, device="cuda")
    rows = [0, 65535, 65536, T // 2 + 3, T - 2, T - 1]
    gen = torch.Generator(device="cuda").manual_seed(8)
    for r in rows:
        X[r] = torch.randn(d, generator=gen, device="cuda").bfloat16()
    B.lora_quantise_rows(X, B.LORA_BF16, T, d, c, s)
    torch.cuda.synchronize()
    v, sb = Q.quantise_rows(X[rows].double().cpu().numpy())
    assert np.array_equal(c[rows].view(torch.float8_e4m3fn).float().cpu().numpy(), v)
    assert np.array_equal(s[rows].cpu().numpy()[:, :sb.shape[1]], sb)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[rows] = False
    nb = (d + 127) // 128
    for i in range(0, T, 1 << 16):
        k = rest[i:i + (1 << 16)]
        assert not bool(c[i:i + (1 << 16)][k].any())
        assert bool((s[i:i + (1 << 16), :nb][k] == 1).all()) and not bool(s[i:i + (1 << 16), nb:].any())
    del X, c
    torch.cuda.empty_cache()
