"""The 8-bit layer's product split over its workgroups at any K tile (the
stream form: more than 128 tokens, fewer tiles than fill the GPU, long K), and
rows whose last block is short.  Tolerances as in test_gpu_quantised."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import quantised as Q
from tests.test_gpu_quantised import Layer, check, expected, workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


# forward: ceil(T / 256) x ceil(d_out / 128) tiles of ceil(d_in / 128) blocks of
# K, at least 1020 in all (255 workgroups, four blocks each); dX the other way
# round.  Widths are odd multiples of 64, so that tiles begin inside a
# workgroup's run and the last block of K is short.
STREAM = [  # T, K, d_in, d_out, extra
    (300, 1, 4288, 1984, {}),                       # 2 x 16 tiles of 34
    (300, 1, 1984, 4288, {"mask": True}),
    (300, 2, 4288, 1984, {"mask": True, "hi": 40}),
    (300, 2, 1984, 4288, {"hi": 40}),
    (129, 1, 2112, 8000, {"mask": True}),           # 1 x 63 tiles of 17
    (700, 1, 8000, 704, {"runs": True, "hi": 80}),  # 3 x 6 tiles of 63
    (700, 1, 704, 8000, {"runs": True, "mask": True}),
]


@pytest.mark.parametrize("T,K,d_in,d_out,extra", STREAM)
def test_stream_form(T, K, d_in, d_out, extra):
    tiles = lambda d_k, d_n: -(-T // 256) * -(-d_n // 128) * -(-d_k // 128)
    assert max(tiles(d_in, d_out), tiles(d_out, d_in)) >= 1020
    w = workload(T, K, d_in, d_out, **extra)
    L = Layer(w)
    L.forward()
    _, _, dX = L.backward()
    torch.cuda.synchronize()
    y, ty, x, tx = expected(w)
    check(L.Y, y, ty, "Y")
    check(dX, x, tx, "dX")
    # the plan apart from the product, and the same again
    Y, U = L.Y.clone(), L.U()
    L.Y.fill_(float("nan"))
    L.ws.fill_(0x11)
    L.run_plan()
    B.lora_apply_quantised(L.X, L.W8, L.Y, L.T, L.K, L.gates, L.keep_mask, L.keep_scale, L.pool, L.plan, L.ws)
    torch.cuda.synchronize()
    assert torch.equal(L.Y, Y) and np.array_equal(L.U(), U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 192, 576])
def test_codes_past_the_end_are_zero(d, dtype):
    """.. in a block without a scale too."""
    rng = np.random.default_rng(d)
    x = torch.from_numpy(rng.standard_normal((4, d)).astype(np.float32)).cuda()
    x[1, d - 3], x[2, d - 64] = float("nan"), float("-inf")
    x = x.bfloat16() if dtype == "bf16" else x
    c = torch.full((4, B.lora_quantised_row_bytes(d)), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((4, B.lora_quantised_scale_bytes(d)), 0x55, dtype=torch.uint8, device="cuda")
    B.lora_quantise_rows(x, B.LORA_BF16 if dtype == "bf16" else B.LORA_F32, 4, d, c, s)
    torch.cuda.synchronize()
    v, sb = Q.quantise_rows(x.double().cpu().numpy())
    assert np.array_equal(c.view(torch.float8_e4m3fn).float().cpu().numpy(), v, equal_nan=True)
    assert np.array_equal(s.cpu().numpy()[:, :sb.shape[1]], sb) and not c[:, d:].any()


FORMS = [
    (40, 1, 576, 704, {}),
    (130, 2, 1344, 320, {"dtype": "f32", "mask": True}),
    (300, 2, 640, 1344, {"mask": True}),
    (300, 1, 4288, 1984, {}),
    (1030, 1, 256, 1536, {"runs": True, "hi": 70}),
    (4096, 1, 192, 4096, {"mask": True}),
]


@pytest.mark.parametrize("T,K,d_in,d_out,extra", FORMS)
def test_workspace_of_the_asked_size_and_of_more(T, K, d_in, d_out, extra):
    """Canaries around a workspace of the size the query gives, a longer one,
    and gradients over both."""
    w = workload(T, K, d_in, d_out, **extra)
    got = []
    for more in (0, 100 * 256 + 64):
        L = Layer(w)
        n, pad = L.ws.numel() + more, 4096
        buf = torch.full((n + 2 * pad,), 0x3c, dtype=torch.uint8, device="cuda")
        L.ws = buf[pad:pad + n]
        L.forward()
        dA, dB, dX = L.backward()
        torch.cuda.synchronize()
        assert (buf[:pad] == 0x3c).all() and (buf[pad + n:] == 0x3c).all()
        got.append((L.Y, dA.nan_to_num(7.0), dB.nan_to_num(7.0), dX, torch.from_numpy(L.U())))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    y, ty, x, tx = expected(w)
    check(got[0][0], y, ty, "Y")
    check(got[0][3], x, tx, "dX")


@pytest.mark.parametrize("T,K,d_in,d_out,extra", FORMS + [(2500, 1, 512, 768, {"mask": True, "hi": 40})])
def test_captured_and_beside_another_stream(T, K, d_in, d_out, extra):
    """Forward, gradients and dX of every form captured and replayed, and two
    layers at once on two streams, against eager calls."""
    w = workload(T, K, d_in, d_out, **extra)

    class Whole(Layer):
        def __init__(self, w):
            super().__init__(w)
            self.dA, self.dB, self.gws = self.grad_buffers()
            self.dX, self.xws = self.grad_x_quantised_buffers()
            self.out = (self.Y, self.dA, self.dB, self.dX)

        def step(self):
            self.forward()
            self.run_grad(self.dA, self.dB, self.gws)
            self.run_grad_x_quantised(self.W8, self.gws, self.dX, self.xws)

        def clear(self):
            for t in self.out:
                t.fill_(7.0)

    def equal(a, b):
        return all(torch.equal(x, y) for x, y in zip(a.out, b))

    L, M = Whole(w), Whole(w)
    L.clear()
    L.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in L.out]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (L, M):
        x.clear()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            L.step()
        with torch.cuda.stream(s2):
            M.step()
    torch.cuda.synchronize()
    assert equal(L, want) and equal(M, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.step()
    for i in range(3):
        L.clear()
        M.step()                                     # eager work between the replays
        g.replay()
        torch.cuda.synchronize()
        assert equal(L, want), i
