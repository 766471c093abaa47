"""The 8-bit oracle pinned against torch's own e4m3 conversion and the scale
rule's definition, and the refusals of the 8-bit entry points (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import quantised as Q


@pytest.fixture(scope="module")
def B():
    from lora_adapter_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from lora_adapter_amd import build
        build.build()
    return binding


def test_rounding_is_torchs():
    x = np.concatenate([np.linspace(-448, 448, 20001), np.ldexp(1.0 + np.arange(64) / 64, -9),
                        np.ldexp(np.arange(64) / 16, -9), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    got = Q.round_e4m3(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("amax", [0.0, 1e-45, 2.0 ** -126, 448.0, 448.0000305, 1.0, 0.875, 0.8750001, 3e38])
def test_scale_rule(amax):
    e = Q.exponent(float(np.float32(amax)))
    a = float(np.float32(amax))
    assert a <= 448 * 2.0 ** e and (e == -126 or a > 448 * 2.0 ** (e - 1))


def test_row_and_scale_bytes(B):
    assert [B.lora_quantised_row_bytes(d) for d in (64, 128, 192, 4096, 0, -64)] == [128, 128, 256, 4096, 0, 0]
    assert [B.lora_quantised_scale_bytes(d) for d in (64, 512, 576, 4096, 0)] == [4, 4, 8, 32, 0]


def _pool(B, **kw):
    d = dict(dtype=B.LORA_BF16, d_in=128, d_out=192, n_adapters=2, n_pages=4, n_page_ids=4,
             a_pages=16, b_pages=16, rank=16, page_start=16, page_ids=16, scale=16)
    d.update(kw)
    return B.PoolDesc(*[d[f] for f, _ in B.PoolDesc._fields_])


def _weight(B, **kw):
    d = dict(d_in=128, d_out=192, q_t=32, scale=48, q=64, scale_t=80)
    d.update(kw)
    return B.QuantisedWeightDesc(*[d[f] for f, _ in B.QuantisedWeightDesc._fields_])


def test_refusals_before_any_hip_call(B):
    L, r = B.lib(), ctypes.byref
    INV, UNS, CAP = B.LORA_ERR_INVALID_ARG, B.LORA_ERR_UNSUPPORTED, B.LORA_ERR_CAPACITY
    pool, w = _pool(B), _weight(B)
    # quantise
    assert L.lora_quantise_rows(8, 5, 4, 128, 16, 24, None) == INV
    assert L.lora_quantise_rows(8, B.LORA_F32, -1, 128, 16, 24, None) == INV
    assert L.lora_quantise_rows(8, B.LORA_F32, 4, 100, 16, 24, None) == UNS
    assert L.lora_quantise_rows(None, B.LORA_F32, 4, 128, 16, 24, None) == INV
    assert L.lora_quantise_rows(8, B.LORA_F32, 4, 128, 8, 24, None) == INV
    assert L.lora_quantise_rows(None, B.LORA_F32, 0, 128, None, None, None) == 0
    assert L.lora_quantise_weight(8, 5, r(w), None) == INV
    assert L.lora_quantise_weight(None, B.LORA_BF16, r(w), None) == INV
    assert L.lora_quantise_weight(8, B.LORA_BF16, None, None) == INV
    assert L.lora_quantise_weight(8, B.LORA_BF16, r(_weight(B, q_t=None)), None) == INV
    assert L.lora_quantise_weight(8, B.LORA_BF16, r(_weight(B, scale_t=None)), None) == INV   # q without its scales
    assert L.lora_quantise_weight(8, B.LORA_BF16, r(_weight(B, d_in=100)), None) == UNS
    assert L.lora_quantise_weight(32, B.LORA_BF16, r(w), None) == INV                         # aliases q_t
    # apply
    big = 1 << 30
    ap = L.lora_apply_quantised
    assert ap(8, r(w), 16, -1, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV
    assert ap(8, r(w), 16, 4, 1, 8, None, 1.0, None, 8, 8, big, None) == INV
    assert ap(8, None, 16, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV
    assert ap(8, r(_weight(B, d_in=192)), 16, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV
    assert ap(8, r(_weight(B, q_t=None)), 16, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV
    assert ap(8, r(w), 8, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV               # Y aliases X
    assert ap(8, r(w), 32, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == INV              # Y aliases the codes
    assert ap(8, r(w), 16, 4, 1, None, None, 1.0, r(pool), 8, 8, big, None) == INV
    assert ap(8, r(w), 16, 4, 1, 8, None, 1.0, r(pool), 8, None, big, None) == INV
    assert ap(8, r(w), 16, 4, 1, 8, None, 1.0, r(pool), 8, 8, 64, None) == CAP
    assert ap(8, r(w), 16, 4, 1, 8, None, 1.0, r(_pool(B, d_in=100)), 8, 8, big, None) == UNS
    assert ap(None, r(w), None, 0, 1, None, None, 1.0, r(pool), 8, None, 0, None) == 0
    # forward
    fw = L.lora_forward_quantised
    assert fw(8, 8, 4, 1, 8, r(w), 16, None, 1.0, r(pool), 8, 16, 8, big, None) == CAP       # plan too small
    assert fw(8, 8, 4, 9, 8, r(w), 16, None, 1.0, r(pool), 8, big, 8, big, None) == INV
    # a refusal of the apply half comes before the plan is launched
    assert fw(8, 8, 4, 1, None, r(w), 16, None, 1.0, r(pool), 8, big, 8, big, None) == INV
    assert fw(8, 8, 4, 1, 8, r(w), 16, None, 1.0, r(pool), 8, big, 8, 64, None) == CAP
    # grad_x
    gx = L.lora_grad_x_quantised
    assert gx(8, r(w), None, 4, 1, r(pool), 8, 8, big, 0, 16, 24, big, None) == INV
    assert gx(8, r(_weight(B, q=None, scale_t=None)), None, 4, 1, r(pool), 8, 8, big, 16, 16, 24, big, None) == INV
    assert gx(8, r(w), None, 4, 1, r(pool), 8, 8, 64, 16, 16, 24, big, None) == CAP
    assert gx(8, r(w), None, 4, 1, r(pool), 8, 8, big, 16, 16, 24, 16, None) == CAP
    assert gx(8, r(w), None, 4, 1, r(pool), 8, 8, big, 16, 8, 24, big, None) == INV
    assert gx(8, r(w), None, 4, 1, r(pool), None, 8, big, 16, 16, 24, big, None) == INV
    # sizes
    assert B.lora_apply_quantised_workspace_bytes(4, 1, 100, 128, 16, B.LORA_BF16) == 0
    assert B.lora_apply_quantised_workspace_bytes(4, 1, 128, 128, 16, 7) == 0
    assert B.lora_grad_x_quantised_workspace_bytes(-1, 128, 128, B.LORA_BF16) == 0
    n = B.lora_apply_quantised_workspace_bytes(300, 1, 512, 640, 16, B.LORA_BF16)
    assert n > B.lora_apply_workspace_bytes(300, 1, 512, 640, 16, B.LORA_BF16)


def test_a_buffer_twice_is_refused(B):
    f, r = B.lib().lora_quantise_weight, ctypes.byref
    one = dict(q_t=16, scale=32, q=48, scale_t=64)
    for a in one:
        assert f(one[a], B.LORA_BF16, r(_weight(B, **one)), None) == B.LORA_ERR_INVALID_ARG
        for b in one:
            if a != b:
                w = _weight(B, **{**one, a: one[b]})
                assert f(8, B.LORA_BF16, r(w), None) == B.LORA_ERR_INVALID_ARG, (a, b)


def test_weight_buffers_are_checked(B):
    e = lambda *s: torch.empty(s, dtype=torch.uint8)
    w = B.QuantisedWeight.empty(192, 128, "cpu")
    assert tuple(w.q_t.shape) == (192, 128) and tuple(w.q.shape) == (128, 256)
    assert tuple(w.scale.shape) == (2, 4) and tuple(w.scale_t.shape) == (1, 4)
    with pytest.raises(ValueError):
        B.QuantisedWeight(192, 128, e(192, 64), w.scale)
    with pytest.raises(ValueError):
        B.QuantisedWeight(192, 128, w.q_t, e(2, 1))
    with pytest.raises(ValueError):
        B.QuantisedWeight(192, 128, torch.empty(192, 128), w.scale)
