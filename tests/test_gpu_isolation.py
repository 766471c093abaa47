"""A non-finite adapter stays its own: a row's output sums its own pairs, an
adapter's gradient its own tokens, whatever form of the product runs.

Each case runs a layer twice, the second time with an infinity and a NaN put
into the pages of one adapter.  What does not depend on that adapter has to be
the same bit for bit; what does has to be non-finite just there.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from lora_adapter_amd import device as D
from tests.test_gpu_quantised import Layer, workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


class Base(D.DeviceLayer):
    """The layer over its own weight, with the calls of the 8-bit one."""

    def forward(self):
        B.lora_forward(self.ids, self.gates, self.T, self.K, self.X, self.W_t, self.Y, self.keep_mask,
                       self.keep_scale, self.pool, self.plan, self.ws)

    def backward(self):
        dA, dB, gws = self.grad_buffers()
        self.run_grad(dA, dB, gws)
        dX, xws = self.grad_x_buffers()
        self.run_grad_x(self.weight_transposed(), gws, dX, xws)
        return dA, dB, dX


def run(L):
    L.forward()
    dA, dB, dX = L.backward()
    torch.cuda.synchronize()
    return L.Y.clone(), dA, dB, dX


def same(a, b):
    return torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))


CASES = [  # kind, T, K, d_in, d_out, extra
    (Layer, 20, 1, 256, 256, {}),
    (Layer, 200, 2, 576, 704, {"mask": True, "hi": 40}),
    (Layer, 130, 2, 1344, 320, {"dtype": "f32", "mask": True, "hi": 40}),
    (Layer, 4096, 1, 192, 4096, {}),                              # tiles with the expand inside: rank <= 16
    (Layer, 4096, 1, 4096, 192, {"mask": True}),                  # .. dX with its mask
    (Layer, 4096, 1, 4096, 192, {}),
    (Layer, 4000, 2, 192, 4160, {"hi": 40}),                      # .. several slots, ranks over 16
    (Layer, 4000, 2, 4160, 192, {"hi": 40, "mask": True}),
    (Layer, 1030, 1, 256, 1536, {"hi": 70, "runs": True}),
    (Base, 20, 1, 256, 256, {}),
    (Base, 200, 2, 576, 704, {"mask": True, "hi": 40}),
    (Base, 4096, 1, 192, 4096, {}),
    (Base, 4096, 1, 4096, 192, {"mask": True}),
    (Base, 4000, 2, 192, 4160, {"hi": 40}),
    (Base, 130, 2, 1344, 320, {"dtype": "f32", "mask": True}),
    (Base, 2500, 1, 512, 768, {"mask": True, "hi": 40}),          # gradients as MFMA products
    (Layer, 1300, 2, 256, 512, {"hi": 20}),
]


class Poisoned:
    """A layer before, and with an infinity and a NaN in two columns of a page
    of B (`b`), then of A (`a`), of adapter 5."""

    def __init__(self, kind, T, K, d_in, d_out, extra):
        w = self.w = workload(T, K, d_in, d_out, **extra)
        p = 5
        pages = w.page_ids[w.page_start[p]:w.page_start[p + 1]]
        self.mine = torch.from_numpy(((w.ids == p) & (w.gates != 0)).any(axis=1)).cuda()
        assert self.mine.any() and not self.mine.all()
        # dropped elements of dX: 0 . inf is NaN in some forms and 0 in none, so they are left out
        self.kept = torch.ones(T, d_in, dtype=torch.bool, device="cuda") if w.keep_mask is None else \
            torch.from_numpy(w.keep_mask != 0).cuda()
        L = kind(w)
        self.clean = run(L)
        assert all(torch.isfinite(t).all() for t in (self.clean[0], self.clean[3]))
        before = L.b_pages.clone()
        self.b_page, self.a_page = int(pages[0]), int(pages[-1])
        self.b_cols, self.a_cols = [3, d_out - 1], [2, d_in - 2]
        L.b_pages[self.b_page, 3], L.b_pages[self.b_page, d_out - 1] = float("inf"), float("nan")
        self.b = run(L)
        L.b_pages.copy_(before)
        L.a_pages[self.a_page, 2], L.a_pages[self.a_page, d_in - 2] = float("nan"), float("inf")
        self.a = run(L)

    def rows(self, clean, got, cols):
        """Own rows differ in `cols` alone, other rows nowhere; the own rows there."""
        assert same(got[~self.mine], clean[~self.mine])
        rest = torch.ones(got.shape[1], dtype=torch.bool, device="cuda")
        rest[cols] = False
        assert same(got[self.mine][:, rest], clean[self.mine][:, rest])
        return got[self.mine][:, cols]


@pytest.mark.parametrize("kind,T,K,d_in,d_out,extra", CASES)
def test_rows_of_other_adapters(kind, T, K, d_in, d_out, extra):
    P = Poisoned(kind, T, K, d_in, d_out, extra)
    Y, _, _, dX = P.clean
    keep, every = P.kept[P.mine], lambda d: list(range(d))
    assert not torch.isfinite(P.rows(Y, P.b[0], P.b_cols)).any()
    assert not torch.isfinite(P.rows(dX, P.b[3], every(d_in))[keep]).any()     # through G
    assert not torch.isfinite(P.rows(Y, P.a[0], every(d_out))).any()           # through U
    assert not torch.isfinite(P.rows(dX, P.a[3], P.a_cols)[keep[:, P.a_cols]]).any()


@pytest.mark.parametrize("kind,T,K,d_in,d_out,extra", CASES)
def test_gradients_of_other_adapters(kind, T, K, d_in, d_out, extra):
    P = Poisoned(kind, T, K, d_in, d_out, extra)
    _, dA, dB, _ = P.clean
    for clean, got, page in ((dA, P.b[1], P.b_page), (dB, P.a[2], P.a_page)):
        rest = torch.ones(got.shape[0], dtype=torch.bool, device="cuda")
        rest[page] = False
        assert same(got[rest], clean[rest])
        assert not torch.isfinite(got[page]).any()
    assert same(P.b[2], dB) and same(P.a[1], dA)


@pytest.mark.parametrize("kind,T,K,d_in,d_out,extra", CASES)
def test_a_non_finite_token_stays_its_own(kind, T, K, d_in, d_out, extra):
    """A NaN in a row of X, then an infinity in a row of dY: the row's own
    outputs, and the pages of the adapters that the row uses."""
    w = workload(T, K, d_in, d_out, **extra)
    t = int(np.flatnonzero(((w.ids >= 0) & (w.gates != 0)).all(axis=1))[T // 3])
    L = kind(w)
    clean = run(L)
    pages = np.concatenate([w.page_ids[w.page_start[a]:w.page_start[a + 1]] for a in set(w.ids[t].tolist())])
    row = torch.arange(T, device="cuda") != t
    page = torch.ones(w.n_pages, dtype=torch.bool, device="cuda")
    page[torch.from_numpy(pages).long().cuda()] = False

    def others(got):
        for i, rest in ((0, row), (1, page), (2, page), (3, row)):
            assert same(got[i][rest], clean[i][rest]), i

    keep = L.X.clone()
    L.X[t, d_in - 1] = float("nan")
    got = run(L)
    others(got)
    assert torch.isnan(got[0][t]).all() and same(got[3], clean[3])     # dX does not read X
    L.X.copy_(keep)
    L.dY[t, 1] = float("inf")
    got = run(L)
    others(got)
    assert same(got[0], clean[0]) and not torch.isfinite(got[3][t]).any()


@pytest.mark.parametrize("kind,T,K,d_in,d_out,extra", [c for c in CASES if c[5].get("mask")])
def test_dropped_elements_do_not_enter_the_branch(kind, T, K, d_in, d_out, extra):
    """Infinities and NaNs of X where the keep mask is 0: U and the gradients
    of the factors are those of any other value there."""
    w = workload(T, K, d_in, d_out, **extra)
    L = kind(w)
    clean = run(L)
    U = L.U()
    off = torch.from_numpy(w.keep_mask == 0).cuda()
    bad = torch.where(torch.arange(d_in, device="cuda") % 3 == 0, float("inf"), float("nan")).to(L.X.dtype)
    L.X.copy_(torch.where(off, bad, L.X))
    got = run(L)
    assert np.array_equal(L.U(), U)
    assert all(same(got[i], clean[i]) for i in (1, 2, 3))
