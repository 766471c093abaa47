"""Rows of the 8-bit layer whose last block is short."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lora_adapter_amd import binding as B
from oracle import quantised as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()


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
