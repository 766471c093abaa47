"""Refusals of the 8-bit layer that need no GPU: every buffer a call writes is
none of those it reads."""
import ctypes
import os

import pytest

from tests.test_quantised_oracle import _pool, _weight


@pytest.fixture(scope="module")
def B():
    from lora_adapter_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from lora_adapter_amd import build
        build.build()
    return binding


def test_outputs_are_no_inputs(B):
    L, r, big = B.lib(), ctypes.byref, 1 << 30
    pool = _pool(B)
    w = _weight(B)                                     # q_t 32, scale 48, q 64, scale_t 80
    for Y in (8, 32, 48):                              # X, the codes, their scales
        assert L.lora_apply_quantised(8, r(w), Y, 4, 1, 8, None, 1.0, r(pool), 8, 8, big, None) == \
            B.LORA_ERR_INVALID_ARG, Y
        assert L.lora_forward_quantised(8, 8, 4, 1, 8, r(w), Y, None, 1.0, r(pool), 8, big, 8, big, None) == \
            B.LORA_ERR_INVALID_ARG, Y
    for dX in (8, 64, 80):                             # dY, the codes of W, their scales
        assert L.lora_grad_x_quantised(8, r(w), None, 4, 1, r(pool), 8, 8, big, 16, dX, 24, big, None) == \
            B.LORA_ERR_INVALID_ARG, dX


def test_workspace_holds_one_set_of_partials(B):
    """The room of the unquantised product's partials takes those of the
    quantised one, and the rows' codes where they fit behind them."""
    up = lambda n: -(-n // 256) * 256
    q, ap = B.lora_apply_quantised_workspace_bytes, B.lora_apply_workspace_bytes
    # fp32: split over K by eight there, whole here
    assert q(3000, 1, 4096, 4096, 16, B.LORA_F32) == up(ap(3000, 1, 4096, 4096, 16, B.LORA_F32))
    # stream form, one set of pieces each: the codes and scales of 256 rows
    n = q(256, 1, 4096, 11008, 128, B.LORA_BF16) - up(ap(256, 1, 4096, 11008, 128, B.LORA_BF16))
    assert n == up(256 * 4096) + up(256 * 32)
    # tiles with the expand inside: no partials there, so codes and scales behind U
    n = q(8192, 1, 4096, 11008, 16, B.LORA_BF16) - up(ap(8192, 1, 4096, 11008, 16, B.LORA_BF16))
    assert n == up(8192 * 4096) + up(8192 * 32)
