"""The 64-bit oracles of the gated block, the cross entropy and the clipping,
pinned by differences, closed forms and worked values; and the refusals of
their entry points, which need no GPU."""
import ctypes
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import training as R


@pytest.fixture(scope="module")
def B():
    from lora_adapter_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from lora_adapter_amd import build
        build.build()
    return binding


# ---------------------------------------------------------------- oracles

@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_slopes_are_differences(act):
    x = np.linspace(-6, 6, 97)
    h = 1e-5
    d = (R.activation(act, x + h)[0] - R.activation(act, x - h)[0]) / (2 * h)
    assert np.max(np.abs(d - R.activation(act, x)[1])) < 1e-8


def test_activation_values():
    one = np.array([1.0])
    assert abs(R.activation("silu", one)[0][0] - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(R.activation("gelu", one)[0][0] - 0.8413447460685429) < 1e-15
    assert abs(R.activation("gelu_tanh", one)[0][0] - 0.8411919906082768) < 1e-12


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradient_is_the_differences(act):
    rng = np.random.default_rng(1)
    X, Wg, Wu, dH = (rng.standard_normal(s) for s in ((3, 8), (5, 8), (5, 8), (3, 5)))
    g, u, _ = R.gated(X, Wg, Wu, act)
    dg, du = R.gated_grad(dH, g, u, act)
    dX = dg @ Wg + du @ Wu
    h = 1e-6
    for t, i in ((0, 0), (1, 3), (2, 7)):
        Xp, Xm = X.copy(), X.copy()
        Xp[t, i] += h
        Xm[t, i] -= h
        d = ((R.gated(Xp, Wg, Wu, act)[2] - R.gated(Xm, Wg, Wu, act)[2]) * dH).sum() / (2 * h)
        assert abs(d - dX[t, i]) < 1e-7


def test_cross_entropy_against_torch_and_differences():
    rng = np.random.default_rng(2)
    X, W = rng.standard_normal((6, 4)), rng.standard_normal((9, 4))
    y, w = np.array([0, 8, -1, 3, 9, 5]), np.array([1, 0.5, 2, 0, 1, 3.0])
    loss, dX, _ = R.cross_entropy(X, W, y, w, 0.7)
    assert math.isnan(loss[4]) and loss[2] == loss[3] == 0 and not dX[2:5].any()
    live = [0, 1, 5]
    x = torch.tensor(X, requires_grad=True)
    l = torch.nn.functional.cross_entropy(0.7 * x @ torch.tensor(W).T, torch.tensor(np.maximum(y, 0) % 9),
                                          reduction="none")
    (l[live] * torch.tensor(w[live])).sum().backward()
    assert np.allclose(loss[live], (l[live] * torch.tensor(w[live])).detach().numpy(), rtol=1e-13, atol=0)
    assert np.allclose(dX[live], x.grad.numpy()[live], rtol=1e-12, atol=1e-14)
    h = 1e-6
    for t, i in ((0, 1), (5, 3)):
        Xp, Xm = X.copy(), X.copy()
        Xp[t, i] += h
        Xm[t, i] -= h
        d = (R.cross_entropy(Xp, W, y, w, 0.7)[0][t] - R.cross_entropy(Xm, W, y, w, 0.7)[0][t]) / (2 * h)
        assert abs(d - dX[t, i]) < 1e-8


def test_clip_worked_example():
    l = {"rank": [1, 2], "page_start": [0, 1, 3], "page_ids": [2, 0, 1], "n_pages": 4,
         "A": np.array([[3.0, 0], [0, 0], [1, 0], [7, 7]]), "B": np.array([[0, 4.0], [0, 0], [0, 1], [7, 7]])}
    norm, out, _ = R.clip([l, l], [1, 0, 1, 5], 4, 1.0, False)
    assert np.allclose(norm, [math.sqrt(50), 2, 0, 0, math.sqrt(54)])
    assert np.allclose(out[0]["A"], [[3 / math.sqrt(50), 0], [0, 0], [0.5, 0], [7, 7]])
    norm, out, _ = R.clip([l], [1, 0], 1, 10.0, True)              # rank 2 is over max_rank
    assert np.allclose(norm, [0, math.sqrt(2), math.sqrt(2)]) and np.array_equal(out[0]["A"], l["A"])


# ---------------------------------------------------------------- refusals

BIG = 1 << 40


def _pool(B, **kw):
    f = dict(dtype=B.LORA_BF16, d_in=128, d_out=192, n_adapters=2, n_pages=4, n_page_ids=3, a_pages=1 << 20,
             b_pages=1 << 21, rank=1 << 22, page_start=1 << 23, page_ids=1 << 24, scale=1 << 25)
    f.update(kw)
    return B.PoolDesc(*(f[n] for n, _ in B.PoolDesc._fields_))


def test_gated_refusals(B):
    L, r = B.lib(), ctypes.byref
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY

    def call(**kw):
        a = dict(X=1 << 12, Wg=2 << 12, Wu=3 << 12, act=0, H=4 << 12, pg=5 << 12, pu=6 << 12, T=4, K=1, gates=7 << 12,
                 mask=None, gate=_pool(B), up=_pool(B), plan=8 << 12, wg=9 << 12, ng=BIG, wu=10 << 12, nu=BIG)
        a.update(kw)
        f = L.lora_gated_apply(a["X"], a["Wg"], a["Wu"], a["act"], a["H"], a["pg"], a["pu"], a["T"], a["K"],
                               a["gates"], a["mask"], 1.0, r(a["gate"]), r(a["up"]), a["plan"], a["wg"], a["ng"],
                               a["wu"], a["nu"], None)
        g = L.lora_gated_forward(1 << 13, a["gates"], a["T"], a["K"], a["X"], a["Wg"], a["Wu"], a["act"], a["H"],
                                 a["pg"], a["pu"], a["mask"], 1.0, r(a["gate"]), r(a["up"]), a["plan"], BIG, a["wg"],
                                 a["ng"], a["wu"], a["nu"], None)
        assert f == g
        return f

    for name in ("X", "Wg", "Wu", "H", "gates", "plan", "wg", "wu"):
        assert call(**{name: None}) == INV, name
    assert call(pg=None) == INV and call(pu=None) == INV            # both or neither
    assert call(act=3) == INV and call(act=-1) == INV
    assert call(K=0) == INV and call(K=9) == INV and call(T=-1) == INV
    assert call(T=1 << 20, K=2) == UNS
    for name in ("H", "pg", "pu", "wg", "wu"):                      # outputs are no inputs and no other output
        for other in (1 << 12, 2 << 12, 3 << 12, 8 << 12):
            assert call(**{name: other}) == INV, (name, other)
    assert call(pg=4 << 12) == INV and call(pu=5 << 12) == INV and call(wu=9 << 12) == INV
    for kw in (dict(rank=1), dict(page_start=1), dict(page_ids=1), dict(n_pages=5), dict(n_page_ids=2),
               dict(n_adapters=3), dict(d_in=64), dict(d_out=64), dict(dtype=B.LORA_F32)):
        assert call(up=_pool(B, **kw)) == INV, kw                   # one plan serves both
    assert call(gate=_pool(B, d_in=100), up=_pool(B, d_in=100)) == UNS
    assert call(ng=0) == CAP and call(nu=0) == CAP


def test_gated_grad_refusals(B):
    L, r = B.lib(), ctypes.byref
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY

    def call(**kw):
        a = dict(dH=1 << 12, pg=2 << 12, pu=3 << 12, act=1, Wg=4 << 12, Wu=5 << 12, mask=None, T=4, K=1,
                 gates=6 << 12, gate=_pool(B), up=_pool(B), plan=7 << 12, R=16, dg=8 << 12, du=9 << 12, dX=10 << 12,
                 ws=11 << 12, n=BIG)
        a.update(kw)
        return L.lora_gated_grad(a["dH"], a["pg"], a["pu"], a["act"], a["Wg"], a["Wu"], a["mask"], 1.0, a["T"],
                                 a["K"], a["gates"], r(a["gate"]), r(a["up"]), a["plan"], a["R"], a["dg"], a["du"],
                                 a["dX"], a["ws"], a["n"], None)

    for name in ("dH", "pg", "pu", "Wg", "Wu", "gates", "plan", "dg", "du", "ws"):
        assert call(**{name: None}) == INV, name
    assert call(act=5) == INV and call(R=0) == INV and call(R=1025) == INV
    for name in ("dg", "du", "dX", "ws"):
        for other in (1 << 12, 4 << 12, 5 << 12, 7 << 12):
            assert call(**{name: other}) == INV, (name, other)
    assert call(dg=3 << 12) == INV and call(du=2 << 12) == INV      # in place each its own
    assert call(dX=2 << 12) == INV and call(dX=3 << 12) == INV and call(dg=9 << 12) == INV
    assert call(up=_pool(B, rank=1)) == INV
    assert call(gate=_pool(B, d_out=100), up=_pool(B, d_out=100)) == UNS
    n = B.lora_gated_grad_workspace_bytes(4, 1, 128, 192, 16, B.LORA_BF16)
    assert n > 0 and call(n=n - 1) == CAP
    assert B.lora_gated_grad_workspace_bytes(4, 1, 100, 192, 16, B.LORA_BF16) == 0
    assert B.lora_gated_grad_workspace_bytes(4, 1, 128, 192, 0, B.LORA_BF16) == 0
    assert call(T=0) == B.LORA_OK


def test_cross_entropy_refusals(B):
    L = B.lib()
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY

    def call(**kw):
        a = dict(X=1 << 12, W=2 << 12, dt=B.LORA_BF16, T=4, V=100, d=128, y=3 << 12, w=4 << 12, s=1.0, loss=5 << 12,
                 dX=6 << 12, ws=7 << 12, n=BIG)
        a.update(kw)
        return L.lora_cross_entropy(a["X"], a["W"], a["dt"], a["T"], a["V"], a["d"], a["y"], a["w"], a["s"],
                                    a["loss"], a["dX"], a["ws"], a["n"], None)

    for name in ("X", "W", "y", "loss", "ws"):
        assert call(**{name: None}) == INV, name
    assert call(dt=2) == INV and call(T=-1) == INV and call(V=0) == INV
    assert call(d=100) == UNS and call(d=0) == UNS and call(V=(1 << 22) + 1) == UNS and call(T=(1 << 20) + 1) == UNS
    for s in (0.0, math.nan, math.inf):
        assert call(s=s) == INV
    for name, at in (("X", 8), ("W", 4), ("dX", 2), ("ws", 1)):
        assert call(**{name: (9 << 12) + at}) == INV, name           # alignment
    for name in ("loss", "dX", "ws"):
        for other in (1 << 12, 2 << 12, 3 << 12, 4 << 12):
            assert call(**{name: other}) == INV, (name, other)
    assert call(dX=5 << 12) == INV and call(ws=6 << 12) == INV
    for grad in (True, False):
        n = B.lora_cross_entropy_workspace_bytes(4, 100, 128, B.LORA_BF16, grad)
        assert n > 0 and call(dX=(6 << 12) if grad else None, n=n - 1) == CAP
    assert B.lora_cross_entropy_workspace_bytes(4, 0, 128, B.LORA_BF16) == 0
    assert B.lora_cross_entropy_workspace_bytes(4, 100, 100, B.LORA_BF16) == 0
    assert call(T=0) == B.LORA_OK
    # the exponentials of a block of tokens are bounded, whatever the batch
    most = B.lora_cross_entropy_workspace_bytes(1 << 20, 128256, 4096, B.LORA_BF16)
    assert most < 3 * (512 << 20)


def test_clip_refusals(B):
    L = B.lib()
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY
    page = 4 * 128 * 4, 4 * 192 * 4                                   # bytes of A's and of B's pages

    def layer(**kw):
        f = dict(pool=_pool(B), a=1 << 16, b=2 << 16, oa=3 << 16, ob=4 << 16)
        f.update(kw)
        return B.GradDesc(f["pool"], f["a"], f["b"], f["oa"], f["ob"])

    def call(layers=None, n=None, ads=1 << 12, M=2, R=16, top=1.0, norm=2 << 12, ws=3 << 12, nb=BIG):
        ls = [layer()] if layers is None else layers
        arr = (B.GradDesc * max(1, len(ls)))(*ls)
        return L.lora_clip_grad(arr, len(ls) if n is None else n, ads, M, R, top, 0, norm, ws, nb, None)

    assert call(ads=None) == INV and call(norm=None) == INV and call(ws=None) == INV
    assert call(M=-1) == INV and call(n=-1) == INV and call(R=0) == INV and call(R=1025) == INV
    for top in (0.0, -1.0, math.nan):
        assert call(top=top) == INV
    assert call(M=16385) == UNS and call(n=1025, layers=[layer()] * 1025) == UNS
    for name in ("a", "b", "oa", "ob"):
        assert call([layer(**{name: None})]) == INV, name
        assert call([layer(**{name: (9 << 16) + 4})]) == INV, name    # alignment
    assert call([layer(pool=_pool(B, rank=None))]) == INV
    assert call([layer(pool=_pool(B, d_in=100))]) == UNS
    # overlaps: two outputs, an output and another gradient, its own gradient but not in place
    assert call([layer(ob=3 << 16)]) == INV
    assert call([layer(ob=(3 << 16) + page[0] - 16)]) == INV
    assert call([layer(oa=2 << 16)]) == INV and call([layer(ob=1 << 16)]) == INV
    assert call([layer(oa=(1 << 16) + 512)]) == INV and call([layer(oa=(1 << 16) - 512)]) == INV
    assert call([layer(), layer(a=5 << 16, b=6 << 16, oa=7 << 16)]) == INV          # ob of both
    assert call([layer(), layer(a=5 << 16, b=6 << 16, oa=7 << 16, ob=1 << 16)]) == INV
    assert call([layer(oa=1 << 16), layer(a=1 << 16, b=6 << 16, oa=7 << 16, ob=8 << 16)]) == INV
    n = L.lora_clip_grad_workspace_bytes(1, 2, 16)
    # what is allowed gets to the workspace's size: in place, side by side, one gradient of two layers
    for ls in ([layer(oa=1 << 16, ob=2 << 16)], [layer(ob=(3 << 16) + page[0])],
               [layer(), layer(oa=7 << 16, ob=8 << 16)]):
        assert call(ls, nb=n - 1) == CAP
    assert L.lora_clip_grad_workspace_bytes(-1, 2, 16) == 0 and L.lora_clip_grad_workspace_bytes(1, 2, 0) == 0


def test_binding_checks_shapes(B):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = torch.zeros(2, dtype=torch.int32)
    pool = B.Pool(B.LORA_BF16, 128, 192, t(4, 128), t(4, 192), i, torch.zeros(3, dtype=torch.int32), i, t(2, dt=torch.float32))
    ws = torch.zeros(64, dtype=torch.uint8)
    ok = dict(X=t(3, 128), W=t(192, 128), H=t(3, 192))
    for bad in (dict(X=t(3, 64)), dict(W=t(128, 192)), dict(H=t(3, 192, dt=torch.float32)), dict(H=t(192, 3).T)):
        a = {**ok, **bad}
        with pytest.raises(ValueError):
            B.lora_gated_forward(i, i, 3, 1, a["X"], a["W"], a["W"], 0, a["H"], None, None, None, 1.0, pool, pool, ws,
                                 ws, ws, 0)
        with pytest.raises(ValueError):
            B.lora_gated_apply(a["X"], a["W"], a["W"], 0, a["H"], None, None, 3, 1, i, None, 1.0, pool, pool, ws, ws,
                               ws, 0)
    with pytest.raises(ValueError):
        B.lora_gated_grad(t(3, 192), t(3, 192), t(3, 192), 0, t(192, 128), t(128, 192), None, 1.0, 3, 1, i, pool, pool,
                          ws, 16, t(3, 192), t(3, 192), t(3, 128), ws, 0)
    with pytest.raises(ValueError):
        B.lora_cross_entropy(t(3, 128), t(9, 128), B.LORA_BF16, 3, 9, 128, i, None, 1.0, t(3, dt=torch.float32), None,
                             ws, 0)
    f = lambda *s: torch.zeros(*s)
    with pytest.raises(ValueError):
        B.GradLayers([(pool, f(4, 128), f(4, 128))])
    with pytest.raises(ValueError):
        B.GradLayers([(pool, f(4, 128).bfloat16(), f(4, 192))])
    layers = B.GradLayers([(pool, f(4, 128), f(4, 192))])
    with pytest.raises(ValueError):
        B.lora_clip_grad(layers, i, 2, 16, 1.0, False, f(2), ws, 0)


def test_gated_alignment_and_widths(B):
    """16 bytes for what is read and written by vectors, 8 for the mask; offsets of a
    weight tile's rows fit 32 bits."""
    L, r = B.lib(), ctypes.byref
    INV, UNS = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED
    names = ("X", "Wg", "Wu", "H", "pg", "pu", "wg", "wu")

    def forward(pool=None, **off):
        a = {n: (i + 1 << 16) + off.get(n, 0) for i, n in enumerate(names)}
        p = pool or _pool(B)
        return L.lora_gated_apply(a["X"], a["Wg"], a["Wu"], 0, a["H"], a["pg"], a["pu"], 4, 1, 1 << 12, None, 1.0, r(p),
                                  r(p), 1 << 13, a["wg"], 0, a["wu"], 0, None)

    for n in names:
        for by in (2, 4, 8):
            assert forward(**{n: by}) == INV, (n, by)
    assert forward() == B.LORA_ERR_CAPACITY                          # all else in order
    names2 = ("dH", "pg", "pu", "Wg", "Wu", "dg", "du", "dX", "ws", "mask")

    def grad(pool=None, **off):
        a = {n: (i + 1 << 16) + off.get(n, 0) for i, n in enumerate(names2)}
        p = pool or _pool(B)
        return L.lora_gated_grad(a["dH"], a["pg"], a["pu"], 0, a["Wg"], a["Wu"], a["mask"], 1.0, 4, 1, 1 << 12, r(p),
                                 r(p), 1 << 13, 16, a["dg"], a["du"], a["dX"], a["ws"], 0, None)

    for n in names2:
        for by in (2, 4) if n == "mask" else (2, 4, 8):
            assert grad(**{n: by}) == INV, (n, by)
    assert grad() == B.LORA_ERR_CAPACITY
    for kw in (dict(d_in=(1 << 22) + 64), dict(d_out=(1 << 22) + 64)):
        assert forward(_pool(B, **kw)) == UNS and grad(_pool(B, **kw)) == UNS
        w = dict(d_in=128, d_out=192)
        w.update(kw)
        assert B.lora_gated_grad_workspace_bytes(4, 1, w["d_in"], w["d_out"], 16, B.LORA_BF16) == 0
    assert B.lora_cross_entropy_workspace_bytes(4, 100, (1 << 22) + 64, B.LORA_BF16) == 0


def test_clip_of_a_norm_that_float32_does_not_hold():
    l = {"rank": [1, 1], "page_start": [0, 1, 2], "page_ids": [0, 1], "n_pages": 2,
         "A": np.array([[3e38, 0], [3e38, 0]]), "B": np.array([[0, 3e38], [0, 1.0]])}
    norm, out, _ = R.clip([l], [0, 1], 4, 1e38, False)
    assert np.isinf(norm[0]) and norm[1] == 3e38 and np.isinf(norm[2])
    assert np.array_equal(out[0]["A"][0], l["A"][0]) and np.allclose(out[0]["A"][1], [1e38, 0])


SPOT = 1 << 26                 # buffers this far apart: none below reaches the next


def _overlaps(call, outs, ins, extra=()):
    """call(**{name: address}) at which two buffers overlap: INVALID_ARG, whichever way."""
    names = list(outs) + list(ins)
    at = {n: (i + 1) * SPOT for i, n in enumerate(names)}
    for o, size in outs.items():
        for n in names:
            if n == o or (o, n) in extra or (n, o) in extra:
                continue
            other = outs.get(n) or ins[n]
            # an output that begins inside the other, ends inside it, and its last 16 bytes
            for where in (at[n] + (other - 1) // 16 * 16, at[n] + 16 - (size + 15) // 16 * 16, at[n]):
                yield o, n, call(**{**at, o: where})


def test_gated_buffers_that_overlap(B):
    """Ranges, not starts alone; the mask, the gates, the ids and the pools among them."""
    L, r, INV = B.lib(), ctypes.byref, B.LORA_ERR_INVALID_ARG
    T, K, d, F, e, N, P = 160, 2, 128, 192, 2, 2, 4
    n = B.lora_apply_workspace_bytes(T, K, d, F, 16, B.LORA_BF16)
    tables = dict(rank=N * 4, page_start=N * 4 + 4, page_ids=12)
    ins = dict(X=T * d * e, Wg=F * d * e, Wu=F * d * e, gates=T * K * 4, mask=T * d, **tables, ga=P * d * e, gb=P * F * e,
               gs=N * 4, ua=P * d * e, ub=P * F * e, us=N * 4)
    rows = T * F * e
    pool = lambda a, p: _pool(B, a_pages=a[p + "a"], b_pages=a[p + "b"], scale=a[p + "s"], **{t: a[t] for t in tables})

    def forward(kind, **a):
        g, u = pool(a, "g"), pool(a, "u")
        tail = (a["gates"], T, K, a["X"], a["Wg"], a["Wu"], 0, a["H"], a["pg"], a["pu"], a["mask"], 1.0, r(g), r(u),
                a["plan"], BIG, a["wg"], n, a["wu"], n, None)
        if kind == "forward":
            return L.lora_gated_forward(a["ids"], *tail)
        return L.lora_gated_apply(a["X"], a["Wg"], a["Wu"], 0, a["H"], a["pg"], a["pu"], T, K, a["gates"], a["mask"], 1.0,
                                  r(g), r(u), a["plan"], a["wg"], n, a["wu"], n, None)

    outs = dict(H=rows, pg=rows, pu=rows, wg=n, wu=n, plan=B.lora_plan_bytes(T, K, N))
    for o, i, got in _overlaps(lambda **a: forward("forward", **a), outs, {**ins, "ids": T * K * 4}):
        assert got == INV, (o, i)
    for o, i, got in _overlaps(lambda **a: forward("apply", **a), outs, ins):
        assert got == INV, (o, i)
    at = {x: (i + 1) * SPOT for i, x in enumerate([*outs, *ins, "ids"])}
    for by in (1, 2, 4):
        assert forward("forward", **{**at, "mask": at["mask"] + by}) == INV
        assert forward("apply", **{**at, "mask": at["mask"] + by}) == INV

    nb = B.lora_gated_grad_workspace_bytes(T, K, d, F, 16, B.LORA_BF16)

    def grad(**a):
        g, u = pool(a, "g"), pool(a, "u")
        return L.lora_gated_grad(a["dH"], a["pg"], a["pu"], 0, a["Wg"], a["Wu"], a["mask"], 1.0, T, K, a["gates"], r(g),
                                 r(u), a["plan"], 16, a["dg"], a["du"], a["dX"], a["ws"], nb, None)

    ins = dict(dH=rows, pg=rows, pu=rows, **{k: ins[k] for k in ins if k != "X"})
    outs = dict(dg=rows, du=rows, dX=T * d * e, ws=nb, plan=outs["plan"])
    for o, i, got in _overlaps(grad, outs, ins, extra=(("dg", "pg"), ("du", "pu"))):
        assert got == INV, (o, i)
    at = {x: (i + 1) * SPOT for i, x in enumerate([*outs, *ins])}
    for o, i in (("dg", "pg"), ("du", "pu")):                        # in place, or apart
        for by in (16, -16, rows - 16, 16 - rows):
            assert grad(**{**at, o: at[i] + by}) == INV, (o, i, by)


def test_cross_entropy_buffers_that_overlap(B):
    T, V, d = 300, 500, 128
    for grad in (True, False):
        n = B.lora_cross_entropy_workspace_bytes(T, V, d, B.LORA_BF16, grad)
        outs, ins = dict(loss=T * 4, dX=T * d * 2, ws=n), dict(X=T * d * 2, W=V * d * 2, y=T * 4, w=T * 4)
        if not grad:
            del outs["dX"]

        def call(**a):
            return B.lib().lora_cross_entropy(a["X"], a["W"], B.LORA_BF16, T, V, d, a["y"], a["w"], 1.0, a["loss"],
                                              a.get("dX"), a["ws"], n, None)

        for o, i, got in _overlaps(call, outs, ins):
            assert got == B.LORA_ERR_INVALID_ARG, (o, i)


def test_clip_buffers_that_overlap(B):
    """Outputs, norm and workspace with gradients, the list and the page tables."""
    L, M, R, N, P = B.lib(), 3, 16, 2, 4
    n = L.lora_clip_grad_workspace_bytes(2, M, R)
    a_, b_ = P * 128 * 4, P * 192 * 4
    tables = {f"{t}{i}": s for i in (0, 1) for t, s in (("rank", N * 4), ("page_start", N * 4 + 4), ("page_ids", 12))}
    outs = dict(oa0=a_, ob0=b_, oa1=a_, ob1=b_, norm=4 * M + 4, ws=n)
    ins = dict(a0=a_, b0=b_, a1=a_, b1=b_, ads=4 * M, **tables)

    def call(**a):
        layers = [B.GradDesc(_pool(B, **{t: a[f"{t}{i}"] for t in ("rank", "page_start", "page_ids")}), a[f"a{i}"],
                             a[f"b{i}"], a[f"oa{i}"], a[f"ob{i}"]) for i in (0, 1)]
        return L.lora_clip_grad((B.GradDesc * 2)(*layers), 2, a["ads"], M, R, 1.0, 0, a["norm"], a["ws"],
                                a.get("n", n), None)

    place = [(o, f"{f}{i}") for i in (0, 1) for f in "ab" for o in (f"o{f}{i}",)]
    for o, i, got in _overlaps(call, outs, ins, extra=place):
        assert got == B.LORA_ERR_INVALID_ARG, (o, i)
    at = {x: (i + 1) * SPOT for i, x in enumerate([*outs, *ins])}
    for o, i in place:                                               # in place, or apart
        for by in (16, -16, ins[i] - 16):
            assert call(**{**at, o: at[i] + by}) == B.LORA_ERR_INVALID_ARG, (o, i, by)
    assert call(**at, n=n - 1) == B.LORA_ERR_CAPACITY
    assert call(**{**at, **{o: at[i] for o, i in place}}, n=n - 1) == B.LORA_ERR_CAPACITY
    for name, by in (("norm", 1), ("norm", 2), ("ws", 1), ("ws", 4)):
        assert call(**{**at, name: at[name] + by}, n=n - 1) == B.LORA_ERR_INVALID_ARG, (name, by)


def test_binding_checks_routing_and_lists(B):
    """ids, gates, the mask and the list of adapters: their sizes and elements."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f32, u8 = lambda *s: torch.zeros(*s), lambda *s: torch.zeros(*s, dtype=torch.uint8)
    T, K, d, F = 3, 2, 128, 192
    pool = B.Pool(B.LORA_BF16, d, F, bf(4, d), bf(4, F), i32(2), i32(3), i32(2), f32(2))
    ws = u8(64)
    bad = [("ids", i32(T, 1)), ("ids", i32(T, K).long()), ("ids", i32(K, T).T), ("gates", f32(T)), ("gates", f32(T, K).double()),
           ("gates", f32(T, K).half()), ("keep_mask", u8(T, d - 1)), ("keep_mask", f32(T, d)), ("keep_mask", u8(d, T).T)]
    for name, t in bad:
        a = {"ids": i32(T, K), "gates": f32(T, K), "keep_mask": u8(T, d), name: t}
        with pytest.raises(ValueError, match=name):
            B.lora_gated_forward(a["ids"], a["gates"], T, K, bf(T, d), bf(F, d), bf(F, d), 0, bf(T, F), None, None,
                                 a["keep_mask"], 1.0, pool, pool, ws, ws, ws, 0)
        if name == "ids":
            continue
        with pytest.raises(ValueError, match=name):
            B.lora_gated_apply(bf(T, d), bf(F, d), bf(F, d), 0, bf(T, F), None, None, T, K, a["gates"], a["keep_mask"],
                               1.0, pool, pool, ws, ws, ws, 0)
        with pytest.raises(ValueError, match=name):
            B.lora_gated_grad(bf(T, F), bf(T, F), bf(T, F), 0, bf(d, F), bf(d, F), a["keep_mask"], 1.0, T, K, a["gates"],
                              pool, pool, ws, 16, bf(T, F), bf(T, F), bf(T, d), ws, 0)
    layers = B.GradLayers([(pool, f32(4, d), f32(4, F))])
    for ads in (i32(1), i32(2).long(), i32(4)[::2]):
        with pytest.raises(ValueError, match="adapters"):
            B.lora_clip_grad(layers, ads, 2, 16, 1.0, False, f32(3), ws, 0)


def test_cross_entropy_workspace_is_bounded(B):
    """Exponentials and sums of a block of tokens, whichever are larger, and 20 bytes a token."""
    for dtype in (B.LORA_BF16, B.LORA_F32):
        for V, d in ((64, 4096), (1, 8192), (8192, 1024), (128256, 4096), (2000, 1024)):
            n = B.lora_cross_entropy_workspace_bytes(1 << 20, V, d, dtype)
            # e, sums, a sixteenth of e for the pieces' sums, 64 MiB of splits, lists
            assert n < (512 << 20) * 2.07 + (64 << 20) + 24 * (1 << 20), (dtype, V, d, n)
            assert B.lora_cross_entropy_workspace_bytes(1 << 20, V, d, dtype, False) < 80 << 20
