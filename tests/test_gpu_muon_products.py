"""GPU checks of the orthogonalised updates where they go through the large products."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gradients(seed, E, r, c, dtype):
    """A few strong directions over noise."""
    rng = torch.Generator(DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=rng, device=DEV)
    g = normal(E, r, c) + 3.0 * normal(E, r, 4) @ normal(E, 4, c)
    return (1e-3 * g).to(DTYPES[dtype]), rng


@pytest.mark.parametrize("E,r,c", [(2, 90, 200), (1, 2048, 128), (2, 300, 700), (2, 700, 300), (2, 600, 5000),
                                   (2, 5000, 600)])
@pytest.mark.parametrize("steps", [2, 5])
def test_results_of_either_type_are_the_fp32_ones_rounded(cuda_lib, E, r, c, steps):
    """Weights of zeros take the steps' result in FP32: rounded, it is what 16-bit results hold, bit for bit. The last
    product has all of its operands' bits whatever it is rounded to."""
    moe = cuda_lib
    g, _ = gradients(c, E, r, c, "f32")
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    moe.moe_muon_step(w, g, m, lr=-1.0, momentum_decay=0.0, update_scale=1.0, steps=steps)
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(moe.moe_orthogonalize(g, dtype=dtype, steps=steps), w.to(dtype))
