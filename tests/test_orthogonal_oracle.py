"""The orthogonalisation oracle pinned against singular values, and the
refusals of its entry points (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import orthogonal as NS

COEF = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def B():
    from lora_adapter_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from lora_adapter_amd import build
        build.build()
    return binding


@pytest.mark.parametrize("r,d", [(1, 64), (4, 64), (16, 128), (40, 64)])
def test_moves_singular_values_and_keeps_vectors(r, d):
    rng = np.random.default_rng(r * d)
    N = rng.standard_normal((r, d)) * 10.0 ** rng.uniform(-2, 0, (r, 1))
    u, s, vt = np.linalg.svd(N, full_matrices=False)
    x = s / (np.sqrt(np.sum(s * s)) + 1e-7)
    for _ in range(5):
        x = COEF[0] * x + COEF[1] * x ** 3 + COEF[2] * x ** 5
    np.testing.assert_allclose(NS.newton_schulz(N, 5, COEF, 1e-7), (u * x) @ vt, atol=1e-9)
    X = N / (np.linalg.norm(N) + 1e-7)
    np.testing.assert_allclose(NS.left_factor(N, 5, COEF, 1e-7) @ X, (u * x) @ vt, atol=1e-9)


def test_cubic_coefficients_converge_to_orthonormal_rows():
    rng = np.random.default_rng(1)
    O = NS.newton_schulz(rng.standard_normal((6, 64)), 32, (1.5, -0.5, 0.0), 1e-7)
    np.testing.assert_allclose(O @ O.T, np.eye(6), atol=1e-12)


def _pool(B, **kw):
    d = dict(dtype=B.LORA_BF16, d_in=128, d_out=192, n_adapters=2, n_pages=4, n_page_ids=4,
             a_pages=16, b_pages=16, rank=16, page_start=16, page_ids=16, scale=16)
    d.update(kw)
    return B.PoolDesc(*[d[f] for f, _ in B.PoolDesc._fields_])


def test_refusals_before_any_hip_call(B):
    L, r = B.lib(), ctypes.byref
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY
    co, big, pool = (ctypes.c_float * 3)(*COEF), 1 << 40, _pool(B)
    o = L.lora_orthogonalise
    ok = dict(pool=r(pool), ad=8, M=2, mr=4, src=16, out=32, d=128, steps=5, coef=co, eps=1e-7, ork=None,
              ws=48, n=big, s=None)
    call = lambda **kw: o(*{**ok, **kw}.values())
    assert call(pool=None) == INV and call(ad=None) == INV and call(M=-1) == INV
    assert call(mr=0) == INV and call(mr=1025) == INV
    assert call(steps=0) == INV and call(steps=33) == INV and call(coef=None) == INV
    assert call(eps=0.0) == INV and call(eps=float("nan")) == INV and call(eps=-1.0) == INV
    assert call(src=None) == INV and call(out=None) == INV and call(out=16) == INV and call(ws=None) == INV
    assert call(d=100) == UNS and call(M=20000) == UNS
    assert call(n=64) == CAP
    assert call(M=0, ad=None, src=None, out=None, ws=None, n=0) == 0
    F = B.FactorUpdateDesc
    fa, fb = F(16, 32, 48, 64, 0.1, 0.0), F(80, 96, 112, 128, 0.1, 0.0)
    st = L.lora_orthogonal_step
    ok2 = dict(pool=r(pool), ad=8, M=2, mr=4, a=r(fa), b=r(fb), mu=0.9, nes=1, steps=5, coef=co, eps=1e-7,
               ork=None, ws=48, n=big, s=None)
    call = lambda **kw: st(*{**ok2, **kw}.values())
    assert call(a=None) == INV and call(b=None) == INV
    assert call(a=r(F(None, 32, 48, 64, 0.1, 0))) == INV and call(a=r(F(16, 32, None, 64, 0.1, 0))) == INV
    assert call(a=r(F(16, 32, 48, None, 0.1, 0))) == INV
    assert call(a=r(F(16, 32, 48, 48, 0.1, 0))) == INV                      # gradient is the momentum
    assert call(b=r(F(16, 96, 112, 128, 0.1, 0))) == INV                    # the other factor's pages
    assert call(a=r(F(16, 16, 48, 64, 0.1, 0))) == INV                      # bf16 pages as their own master
    assert call(pool=r(_pool(B, dtype=B.LORA_F32)), a=r(F(16, 16, 48, 64, 0.1, 0)), n=64) == CAP   # fp32: allowed
    assert call(pool=r(_pool(B, d_in=100))) == UNS
    assert call(n=64) == CAP and call(ws=None) == INV
    assert call(M=0, a=None, b=None, ws=None) == 0
    assert B.lora_orthogonalise_workspace_bytes(0, 4, 128) == 0
    assert B.lora_orthogonalise_workspace_bytes(4, 2000, 128) == 0
    assert B.lora_orthogonal_step_workspace_bytes(4, 16, 100, 128) == 0
    assert B.lora_orthogonal_step_workspace_bytes(4, 16, 128, 192) > 0


def test_a_buffer_of_both_factors_is_refused(B):
    r, st = ctypes.byref, B.lib().lora_orthogonal_step
    names = ("pages", "master", "momentum", "grad")
    fa, fb = dict(zip(names, (16, 32, 48, 64))), dict(zip(names, (80, 96, 112, 128)))
    co = (ctypes.c_float * 3)(*COEF)

    def call(a, b):
        F = lambda u: r(B.FactorUpdateDesc(*(u[n] for n in names), 0.1, 0.0))
        return st(r(_pool(B)), 8, 2, 4, F(a), F(b), 0.9, 1, 5, co, 1e-7, None, 48, 64, None)

    for x in names:
        for y in names:
            # ws of 64 bytes: what is not refused for its buffers is too small
            want = B.LORA_ERR_CAPACITY if x == y == "grad" else B.LORA_ERR_INVALID_ARG
            assert call(fa, {**fb, y: fa[x]}) == want, (x, y)
    assert call({**fa, "master": None}, {**fb, "master": None}) == B.LORA_ERR_CAPACITY
