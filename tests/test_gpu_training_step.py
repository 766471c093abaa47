"""The 8-bit base and the orthogonalised update used together: a training loop
of one layer against the 64-bit oracles, and the backward against differences
and adjointness."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from lora_adapter_amd import device as D
from oracle import orthogonal as NS
from oracle import quantised as Q
from tests.test_gpu_quantised import Layer, check, dt_of, expected, terms, workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


@pytest.mark.parametrize("dtype,T", [("bf16", 70), ("bf16", 600), ("f32", 70)])
def test_training_steps(dtype, T):
    """Two steps of forward, backward, update; each forward and backward is
    checked against the oracle on the factors as the last update left them,
    each update against the oracle on the gradients lora_grad left."""
    w = workload(T, 2, 320, 192, dtype, N=6, hi=20, mask=True, seed=21)
    L = Layer(w)
    master = [L.a_pages.float().clone(), L.b_pages.float().clone()]
    mom = [torch.zeros_like(m) for m in master]
    ads = torch.arange(w.n_adapters, dtype=torch.int32, device="cuda")
    R = L.max_rank
    ws = torch.empty(B.lora_orthogonal_step_workspace_bytes(w.n_adapters, R, w.d_in, w.d_out), dtype=torch.uint8,
                     device="cuda")
    for _ in range(2):
        L.forward()
        dA, dB, dX = L.backward()
        torch.cuda.synchronize()
        y, ty, x, tx = expected(w)
        check(L.Y, y, ty, "Y")
        check(dX, x, tx, "dX")
        grad = [dA.nan_to_num(0.0), dB.nan_to_num(0.0)]   # pages of unused adapters
        w0 = [m.double().cpu().numpy() for m in master]
        f = [B.FactorUpdate(p, g, mo, ma, 0.05, 0.01)
             for p, g, mo, ma in zip((L.a_pages, L.b_pages), grad, mom, master)]
        B.lora_orthogonal_step(L.pool, ads, w.n_adapters, R, f[0], f[1], 0.0, False, 5, B.NS_COEF, 1e-7, ws)
        torch.cuda.synchronize()
        lr, keep = float(np.float32(0.05)), float(np.float32(1) - np.float32(0.05) * np.float32(0.01))
        for i in (0, 1):
            g = grad[i].double().cpu().numpy()
            got = master[i].double().cpu().numpy()
            for a in range(w.n_adapters):
                r = w.page_ids[w.page_start[a]:w.page_start[a + 1]]
                O, tol = NS.newton_schulz(g[r], 5, B.NS_COEF, 1e-7), NS.tolerance(g[r], 5, B.NS_COEF, 1e-7)
                want = w0[i][r] * keep - lr * O
                t = lr * tol + 2.0 ** -24 * (3 * np.abs(w0[i][r]) + lr * np.abs(O) + np.abs(want))
                assert np.all(np.abs(got[r] - want) <= t)
        assert torch.equal(L.a_pages[w.page_ids], master[0][w.page_ids].to(L.a_pages.dtype))
        # the oracle's copy of the layer follows
        w.a_pages, w.b_pages = D.to_host(L.a_pages), D.to_host(L.b_pages)


def test_captured_loop_beside_an_eager_one():
    """A whole step captured while another layer's eager buffers live; replays
    equal eager steps from the same state."""
    def make():
        w = workload(40, 1, 256, 192, "bf16", N=4, mask=True, seed=33)
        L = Layer(w)
        L.dA, L.dB, L.gws = L.grad_buffers()
        L.dA.zero_(), L.dB.zero_()
        L.dX = torch.zeros(w.T, w.d_in, dtype=torch.bfloat16, device="cuda")
        L.xws = torch.empty(B.lora_grad_x_quantised_workspace_bytes(w.T, w.d_in, w.d_out, dt_of(w)),
                            dtype=torch.uint8, device="cuda")
        L.ad = torch.arange(4, dtype=torch.int32, device="cuda")
        L.sws = torch.empty(B.lora_orthogonal_step_workspace_bytes(4, L.max_rank, w.d_in, w.d_out),
                            dtype=torch.uint8, device="cuda")
        L.mom = [torch.zeros_like(L.dA), torch.zeros_like(L.dB)]
        L.f = [B.FactorUpdate(p, g, m, None, 0.05) for p, g, m in
               zip((L.a_pages, L.b_pages), (L.dA, L.dB), L.mom)]
        return L

    def step(L):
        w = L.w
        L.forward()
        L.run_grad(L.dA, L.dB, L.gws)
        B.lora_grad_x_quantised(L.dY, L.W8, L.keep_mask, w.T, w.K, L.pool, L.plan, L.gws, L.max_rank, L.dX, L.xws)
        B.lora_orthogonal_step(L.pool, L.ad, 4, L.max_rank, L.f[0], L.f[1], 0.9, True, 5, B.NS_COEF, 1e-7, L.sws)

    eager, cap = make(), make()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cap)
    for i in range(4):
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        for a, b in ((eager.Y, cap.Y), (eager.dX, cap.dX), (eager.a_pages, cap.a_pages), (eager.b_pages, cap.b_pages)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_methods(dtype):
    """DeviceLayer's calls give what the binding's give."""
    w = workload(70, 2, 320, 192, dtype, N=4, hi=20, mask=True, seed=5)
    L, R = D.DeviceLayer(w), Layer(w)
    R.forward()
    W8, L.ws = L.quantise_weight(), L.quantised_workspace()
    L.run_forward_quantised(W8, L.ws)
    assert torch.equal(L.Y, R.Y)
    Y = torch.empty_like(L.Y)
    L.run_apply_quantised(L.quantise_weight(both=False), L.quantised_workspace(), Y=Y)
    assert torch.equal(Y, R.Y)
    dA, dB, dX = R.backward()
    ga, gb, gws = L.grad_buffers()
    L.run_grad(ga, gb, gws)
    gx, xws = L.grad_x_quantised_buffers()
    L.run_grad_x_quantised(W8, gws, gx, xws)
    for a, b in ((ga, dA), (gb, dB), (gx, dX)):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    ads = torch.arange(4, dtype=torch.int32, device="cuda")
    grads = [ga.nan_to_num(0.0), gb.nan_to_num(0.0)]
    for master in (True, False):
        mom, own, ws = L.orthogonal_buffers(master)
        assert all((o is not None) == (master and dtype == "bf16") for o in own)
        want = [p.clone() for p in (L.a_pages, L.b_pages)]
        wm, wo = [m.clone() for m in mom], [None if o is None else o.clone() for o in own]
        rank = torch.zeros(4, dtype=torch.int32, device="cuda")
        L.run_orthogonal_step(ads, grads, mom, own, ws, lr=0.05, decay=0.1, out_rank=rank)
        f = [B.FactorUpdate(p, g, m, o, 0.05, 0.1) for p, g, m, o in zip(want, grads, wm, wo)]
        B.lora_orthogonal_step(L.pool, ads, 4, L.max_rank, f[0], f[1], 0.95, True, 5, B.NS_COEF, 1e-7, ws)
        torch.cuda.synchronize()
        assert rank.cpu().numpy().tolist() == w.rank.tolist()
        for a, b in ((L.a_pages, want[0]), (L.b_pages, want[1]), (mom[0], wm[0]), (mom[1], wm[1])):
            assert torch.equal(a, b)


def test_factor_gradients_against_differences():
    """Y is linear in A and in B: <dY, Y(A + D) - Y(A)> = <dA, D>, up to the
    fp32 sums of the two Y: at most d_in + 8 additions in a row for the base
    product (the MFMA's counted one by one), and at most 40 for the adapters'
    term (a lane's 8 products and 6 steps over the wave for U, its coefficient,
    then up to 12 rank rows and the partials)."""
    w = workload(24, 2, 192, 128, "f32", N=3, hi=6, mask=True, seed=40)
    L = Layer(w)
    L.forward()
    dA, dB, _ = L.backward()
    Y0, dY = L.Y.double(), L.dY.double()
    W8 = Q.weight_values(*Q.quantise_weight(D.as_f64(w.W_t)), w.d_in)
    X = np.abs(D.as_f64(w.X))
    base = np.abs(Q.row_values(*Q.quantise_rows(D.as_f64(w.X)), w.d_in)) @ np.abs(W8).T

    def lora(A, Bp):
        A, Bp = np.abs(A.double().cpu().numpy()), np.abs(Bp.double().cpu().numpy())
        m = np.zeros((w.T, w.d_out))
        for t, p, c in terms(w):
            m[t] += abs(c) * ((A[p] @ (X[t] * w.keep_mask[t])) @ Bp[p])
        return m

    rng = torch.Generator(device="cuda").manual_seed(1)
    for pages, grad in ((L.a_pages, dA), (L.b_pages, dB)):
        keep = pages.clone()
        step = torch.randn(pages.shape, generator=rng, device="cuda")
        pages += step
        moved = pages.double() - keep.double()
        L.forward()
        torch.cuda.synchronize()
        got = ((L.Y.double() - Y0) * dY).sum().item()
        pages.copy_(keep)
        used = ~torch.isnan(grad[:, 0])
        want = (grad.double()[used] * moved[used]).sum().item()
        lim = 2.0 ** -24 * float(np.sum(np.abs(D.as_f64(w.dY)) * (2 * (w.d_in + 8) * base + 40 * (
            lora(keep if pages is L.a_pages else L.a_pages, keep if pages is L.b_pages else L.b_pages) +
            lora(keep + step if pages is L.a_pages else L.a_pages, keep + step if pages is L.b_pages else L.b_pages)))))
        assert abs(got - want) <= lim, (got, want, lim)
        # a gradient wrong by a tenth (the keep scale, a gate, a scale) would fail
        assert 0.1 * abs(want) > lim, (want, lim)


def test_input_gradient_is_the_adjoint():
    """With rows that are e4m3 values already, X and dY are quantised without
    error: <dY, Y> = <dX, X> for the base product, each side fp32 sums."""
    w = workload(50, 1, 320, 192, "f32", N=3, seed=41)
    rng = np.random.default_rng(5)
    val = lambda *s: Q.round_e4m3(np.clip(rng.standard_normal(s) * 20, -448, 448)).astype(np.float32)
    w.X, w.dY = val(50, 320), val(50, 192)
    w.gates[:] = 0                                   # the base product alone
    L = Layer(w)
    L.forward()
    _, _, dX = L.backward()
    torch.cuda.synchronize()
    Y, X, dY = D.as_f64(L.Y_host()), D.as_f64(w.X), D.as_f64(w.dY)
    W8 = Q.weight_values(*Q.quantise_weight(D.as_f64(w.W_t)), w.d_in)
    mag = float(np.sum(np.abs(dY) * (np.abs(X) @ np.abs(W8).T)))
    assert abs(float(np.sum(dY * Y)) - float(np.sum(D.as_f64(D.to_host(dX)) * X))) <= (320 + 192) * 2.0 ** -24 * mag
