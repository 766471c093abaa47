"""Gradient norms and clipping on the GPU against 64 bits.

Norms are float64 sums rounded once: half a step, and 2^-40 for the sums'
order.  A clipped value has two roundings, of the factor and of the product.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import training as R
from tests.gpu_training_cases import Guarded, f64, near, tables, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


class Layers:
    def __init__(self, n, N, lo, hi, widths, seed=0, in_place=False, size=1.0):
        rng = np.random.default_rng(seed)
        self.host, self.entries, self.outs = [], [], []
        for i in range(n):
            d, F = widths[i % len(widths)]
            rank, start, ids, P = tables(rng, N, lo, hi)
            a, b = ((rng.standard_normal((P, w)) * size / w ** 0.5).astype(np.float32) for w in (d, F))
            self.host.append(dict(rank=rank, page_start=start, page_ids=ids, n_pages=P, A=a.astype(np.float64),
                                  B=b.astype(np.float64)))
            dev = lambda x: torch.from_numpy(x).cuda()
            ga, gb = Guarded(P, d), Guarded(P, F)
            ga.t.copy_(dev(a))
            gb.t.copy_(dev(b))
            oa, ob = (ga, gb) if in_place else (Guarded(P, d), Guarded(P, F))
            pool = B.Pool(B.LORA_F32, d, F, ga.t, gb.t, dev(rank), dev(start), dev(ids), dev(np.ones(N, np.float32)))
            self.entries.append((pool, ga.t, gb.t, oa.t, ob.t))
            self.outs.append((oa, ob, ga, gb))
        self.layers = B.GradLayers(self.entries)

    def run(self, adapters, R_, top, together):
        M = len(adapters)
        norm = Guarded(M + 1)
        ads = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        ws = workspace(B.lora_clip_grad_workspace_bytes(self.layers, M, R_))
        B.lora_clip_grad(self.layers, ads, M, R_, top, together, norm.t, ws)
        torch.cuda.synchronize()
        norm.check("norm")
        for o in self.outs:
            for g in o:
                g.check("pages")
        return norm.t

    def check(self, adapters, R_, top, together):
        top = float(np.float32(top))                       # the entry point takes a float
        before = [(f64(e[3]), f64(e[4])) for e in self.entries]
        ref, out, taken = R.clip(self.host, adapters, R_, top, together)
        norm = self.run(adapters, R_, top, together)
        near(norm, ref, np.abs(ref) * (2.0 ** -24 + 2.0 ** -40) + 1e-45, "norm")
        for e, o, here, was in zip(self.entries, out, taken, before):
            pages = np.concatenate(list(here.values())) if here else np.zeros(0, int)
            for got, f, w in ((e[3], "A", was[0]), (e[4], "B", was[1])):
                want = w.copy()
                want[pages] = o[f][pages]
                tol = np.zeros_like(want)
                tol[pages] = np.abs(want[pages]) * (2.0 ** -23 + 2.0 ** -40) + 2.0 ** -149
                near(got, want, tol, f)


@pytest.mark.parametrize("n,N,lo,hi,widths", [(1, 1, 1, 1, [(64, 64)]), (1, 4, 16, 16, [(128, 320)]),
                                              (3, 5, 0, 7, [(64, 1088), (576, 64)]), (7, 6, 1, 40, [(4096, 192)]),
                                              (40, 3, 1, 5, [(64, 128), (192, 64), (64, 64)])])
@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_against_64_bits(n, N, lo, hi, widths, together, in_place):
    rng = np.random.default_rng(n)
    L = Layers(n, N, lo, hi, widths, seed=n, in_place=in_place)
    ads = [int(a) for a in rng.permutation(N)[: max(1, N - 1)]]
    ref = R.clip(L.host, ads, 64, 1.0, together)[0]
    top = float(np.float32(np.median(ref[:-1]) * (0.7 if together else 1.0)))   # some clipped, some not
    L.check(ads, 64, top, together)


@pytest.mark.parametrize("in_place", [False, True])
def test_nothing_clipped_and_norms_alone(in_place):
    L = Layers(3, 4, 1, 9, [(128, 64)], in_place=in_place)
    L.check([2, 0], 16, 1e6, False)
    L.check([2, 0, 1], 16, float("inf"), True)


def test_listed_twice_out_of_range_and_bad_tables():
    L = Layers(3, 6, 1, 9, [(64, 192)], seed=3)
    h = L.host
    h[0]["rank"][1] += 1                                   # a rank that is not its pages' number
    L.entries[0][0].tensors[2].copy_(torch.from_numpy(h[0]["rank"]))
    h[1]["page_ids"][h[1]["page_start"][2]] = h[1]["n_pages"]           # a page out of range
    L.entries[1][0].tensors[4].copy_(torch.from_numpy(h[1]["page_ids"]))
    h[2]["page_ids"][h[2]["page_start"][4]] = -1
    L.entries[2][0].tensors[4].copy_(torch.from_numpy(h[2]["page_ids"]))
    L.check([1, 2, 4, 2, -1, 6, 2 ** 31 - 1, 0, 0], 16, 0.05, False)
    L.check([1, 2, 4, 2, -1, 6, 5], 4, 0.05, True)         # ranks over 4 are left out


def test_sizes_that_float32_squares_do_not_hold():
    for size in (1e30, 1e-30, 3e37):
        L = Layers(2, 3, 2, 5, [(64, 64)], size=size)
        L.check([0, 1, 2], 8, size * 0.5, False)
        L.check([0, 1, 2], 8, size * 0.5, True)


def test_norms_past_float32():
    """A norm that float32 does not hold is reported as infinite and clips nothing."""
    L = Layers(2, 6, 1, 7, [(64, 64)], size=6.8e37, seed=4)
    ads = [0, 1, 2, 3, 4, 5]
    norm = R.clip(L.host, ads, 8, 5e37, False)[0]
    assert np.isinf(norm[:-1]).any() and np.isfinite(norm[:-1]).any() and np.isinf(norm[-1])
    L.check(ads, 8, 5e37, False)
    L.check(ads, 8, 5e37, True)


@pytest.mark.parametrize("in_place", [False, True])
def test_factors_that_float32_does_not_hold(in_place):
    """max_norm / n below float32's normal numbers: the product is rounded once all the same."""
    for size, top in ((1e30, 1e-11), (1e37, 1e-3), (1e30, 1e-20)):
        L = Layers(2, 3, 2, 5, [(64, 64)], size=size, in_place=in_place)
        L.check([0, 1, 2], 8, top, in_place)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_finite(value):
    """That adapter's gradients go through as they are; the others are clipped."""
    L = Layers(2, 3, 2, 4, [(64, 128)], seed=8)
    p = int(L.host[1]["page_ids"][L.host[1]["page_start"][1]])
    L.entries[1][2][p, 5] = value
    L.host[1]["B"][p, 5] = value
    L.check([0, 1, 2], 8, 0.5, False)
    L.check([0, 1, 2], 8, 0.5, True)


@pytest.mark.parametrize("n,M,together", [(7, 9, False), (7, 10, False), (7, 9, True), (7, 10, True), (7, 40, False),
                                          (40, 60, False), (40, 60, True)])
def test_partials_of_few_and_of_many(n, M, together):
    """2016 and 2240 partials, on both sides of where the second pass's workgroups add
    them; 8960 and 28800."""
    L = Layers(n, M + 2, 1, 16, [(64, 128), (192, 64)], seed=M)
    ads = [int(a) for a in np.random.default_rng(M).permutation(M + 2)[:M]]
    ref = R.clip(L.host, ads, 16, 1.0, together)[0]
    L.check(ads, 16, float(np.median(ref[:-1]) * (0.7 if together else 1.0)), together)


def test_no_layers_and_no_adapters():
    L = Layers(1, 2, 1, 3, [(64, 64)])
    assert L.run([], 4, 1.0, True).tolist() == [0.0]
    L.entries, L.outs = [], []
    L.layers = B.GradLayers([])
    assert L.run([0, 1], 4, 1.0, False).tolist() == [0.0, 0.0, 0.0]


def test_captured_and_deterministic():
    L = Layers(5, 4, 3, 9, [(128, 192)], seed=5)
    ads = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    norm = torch.zeros(4, device="cuda")
    ws = workspace(B.lora_clip_grad_workspace_bytes(L.layers, 3, 16))
    call = lambda: B.lora_clip_grad(L.layers, ads, 3, 16, 0.4, False, norm, ws)
    call()
    torch.cuda.synchronize()
    ref = [norm.clone()] + [e[k].clone() for e in L.entries for k in (3, 4)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for e in L.entries:
            e[3].view(torch.uint8).fill_(0x6b)
            e[4].view(torch.uint8).fill_(0x6b)
        graph.replay()
        torch.cuda.synchronize()
        got = [norm] + [e[k] for e in L.entries for k in (3, 4)]
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))
