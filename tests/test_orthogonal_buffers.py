"""The binding refuses pages that are not laid out as the in-place update and
the orthogonalisation take them, before any call of the library."""
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    from lora_adapter_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from lora_adapter_amd import build
        build.build()
    return binding


def _pool(B, dtype):
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    t = torch.bfloat16 if dtype == B.LORA_BF16 else torch.float32
    return B.Pool(dtype, 64, 128, torch.zeros(4, 64, dtype=t), torch.zeros(4, 128, dtype=t), i(1, 2), i(0, 1, 3),
                  i(0, 1, 2), torch.ones(2))


def test_factor_updates(B):
    z = lambda *s: torch.zeros(*s)
    with pytest.raises(ValueError):                                # every second page of a larger buffer
        B.FactorUpdate(z(8, 64)[::2], z(4, 64), z(4, 64), None, 0.1)
    ws, ad = torch.zeros(64, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)

    def step(dtype, pa, pb):
        f = [B.FactorUpdate(p, z(*p.shape), z(*p.shape), None, 0.1) for p in (pa, pb)]
        B.lora_orthogonal_step(_pool(B, dtype), ad, 1, 2, f[0], f[1], 0.9, True, 5, B.NS_COEF, 1e-7, ws, stream=0)

    for dtype, pa, pb in ((B.LORA_F32, z(4, 64).bfloat16(), z(4, 128)),      # an fp32 pool writes 4 bytes
                          (B.LORA_F32, z(4, 64), z(3, 128)),
                          (B.LORA_BF16, z(4, 64).bfloat16(), z(4, 64).bfloat16())):
        with pytest.raises(ValueError):
            step(dtype, pa, pb)


def test_orthogonalised_pages(B):
    z = lambda *s: torch.zeros(*s)
    ws, ad = torch.zeros(64, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    pool = _pool(B, B.LORA_BF16)
    for src, out in ((z(4, 64).bfloat16(), z(4, 64)), (z(4, 64), z(3, 64)), (z(4, 64), z(4, 128)[:, ::2])):
        with pytest.raises(ValueError):
            B.lora_orthogonalise(pool, ad, 1, 2, src, out, 64, 5, B.NS_COEF, 1e-7, ws, stream=0)
