"""GPU checks of the MXFP4 experts at the ends of their ranges: handles dropped while their work is queued, and buffers
of another type."""
import pytest
import torch

from tests.test_gpu_mxfp4 import DEV, _layer, activations

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ lifetimes

@pytest.mark.parametrize("how", ["argument", "current"])
def test_a_handle_dropped_while_its_work_is_queued(cuda_lib, how):
    """The last reference goes while the products still wait on another stream than the handle was made on: the memory
    that the handle held is not handed out before they are done."""
    moe = cuda_lib
    T, E, k, H, I = 64, 4, 2, 1024, 2048
    ex, _ = _layer(moe, E, H, I, torch.bfloat16, 11)
    x = activations(T, H, torch.bfloat16, 1).to(DEV)
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(DEV)
    ref = moe.moe_forward_mxfp4(ex, x, lg, k, True)
    sizes = [E * I * H // 2, E * I * H // 2, E * H * I // 2, ex._storage.numel()]
    s = torch.cuda.Stream()
    torch.full((8,), 0x77, dtype=torch.uint8, device=DEV)   # nothing below loads a module or maps memory: that would wait
    moe.moe_forward_mxfp4(ex, x, lg, k, True, stream=s)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)           # some 0.2 s
    if how == "argument":
        out = moe.moe_forward_mxfp4(ex, x, lg, k, True, stream=s)
    else:
        with torch.cuda.stream(s):
            out = moe.moe_forward_mxfp4(ex, x, lg, k, True)
    del ex
    junk = [torch.full((n,), 0x77, dtype=torch.uint8, device=DEV) for n in sizes * 2]
    torch.cuda.synchronize()
    assert moe.moe_device_status() == 0
    assert torch.equal(out, ref) and len(junk) == 8


def test_forward_refuses_buffers_of_another_type(cuda_lib):
    """The routing weights come in the logits' type and the indices as 32-bit integers: a buffer of the same size but
    another type would be read as something else."""
    moe = cuda_lib
    ex, _ = _layer(moe, 3, 64, 96, torch.bfloat16, 1)
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    lg = torch.zeros(8, 3, dtype=torch.bfloat16, device=DEV)
    e = lambda dtype: torch.empty(8, 2, dtype=dtype, device=DEV)
    for kw in (dict(weights=e(torch.float16)), dict(weights=e(torch.int16)), dict(indices=e(torch.float32)),
               dict(weights=e(torch.bfloat16), indices=e(torch.float32))):
        with pytest.raises(moe.MoeError):
            moe.moe_forward_mxfp4(ex, x, lg, 2, True, **kw)
    w, i = e(torch.bfloat16), e(torch.int32)
    moe.moe_forward_mxfp4(ex, x, lg, 2, True, weights=w, indices=i)
    assert torch.equal(w, torch.full_like(w, 0.5)) and i.tolist() == [[0, 1]] * 8
