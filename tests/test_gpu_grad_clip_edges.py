"""GPU checks of the gradient clip's bits and of the norm's small magnitudes.

Tolerance of tests/test_gpu_grad_clip.py, from a thread's 16 or 32 squares in FP32. A thread carries its units' sums as a
pair of FP32 whose additions are compensated: each rounding error goes to the second word, whose own rounding is 2^-48 of
the sum, so that n units are off by n 2^-48; where FP32 does not hold the squares, and above threads, sums are FP64. Both
are far below the 2^-24 that the bound counts, and neither depends on the size of the gradients."""
import pytest
import torch

from tests.test_gpu_grad_clip import DEV, DTYPES, check_norm, grads

pytestmark = pytest.mark.gpu
BITS = {torch.float32: torch.int32, torch.float16: torch.int16, torch.bfloat16: torch.int16}
INF_BITS = {torch.float32: 0x7F800000, torch.float16: 0x7C00, torch.bfloat16: 0x7F80}
SIGN = {torch.float32: -1 << 31, torch.float16: -1 << 15, torch.bfloat16: -1 << 15}


def with_nans(n, dtype, seed):
    """Random gradients with infinities, zeros and NaNs of both signs and many payloads in the head (before a 16-byte
    boundary), the vectors and the tail."""
    t = grads([(n, dtype)], seed)[0]
    b = t.view(BITS[dtype])
    at = torch.cat((torch.arange(0, n, 13), torch.arange(max(0, n - 9), n))).to(DEV)
    payload = (torch.arange(len(at), device=DEV) * 37 % (1 << 6)).to(BITS[dtype])   # 0: an infinity
    b[at] = payload + INF_BITS[dtype]
    b[at[::2]] |= SIGN[dtype]
    b[at[1::7]] = SIGN[dtype]                                                      # -0
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 3), (0, 1), (5, 2)])
def test_a_factor_of_one_copies_every_bit(cuda_lib, dtype, a, b):
    """With a norm that is not finite (and with one that is not larger than max_norm) dst gets src's bits, NaN signs
    and payloads among them, at equal and at different alignments."""
    moe = cuda_lib
    n = 70001
    src = with_nans(n + 8, dtype, a)
    dst = torch.full((n + 8,), 9.0, dtype=dtype, device=DEV)
    s, d = src[a:a + n], dst[b:b + n]
    norm = moe.moe_grad_norm([s])
    assert not torch.isfinite(norm)
    for v in (norm, torch.tensor(float("inf"), device=DEV), torch.tensor(0.5, device=DEV)):
        d.fill_(9.0)
        moe.moe_grad_clip([s], v, 0.5, out=[d])
        assert torch.equal(d.view(BITS[dtype]), s.view(BITS[dtype]))
        assert (dst[:b] == 9.0).all() and (dst[b + n:] == 9.0).all()
    keep = src.clone()
    moe.moe_grad_clip([s], norm, 0.5)
    assert torch.equal(src.view(BITS[dtype]), keep.view(BITS[dtype]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [2.0 ** -30, 1e-10, 1e-12, 1e-14, 2.0 ** -50, 2.0 ** -52, 1e-17])
def test_norm_of_small_gradients(cuda_lib, dtype, scale):
    """Across the magnitudes at which a thread's sum of squares passes 2^-60 and 2^-100, with units of both kinds in
    one sum, and zeros of both signs."""
    ts = grads([(300_000, dtype), (5, dtype), (70_001, dtype)], 9, scale)
    ts[0][:30_000] = 0
    ts[0][30_000:60_000] = -0.0
    ts[2][:20_000] *= 2.0 ** 12
    check_norm(cuda_lib.moe_grad_norm(ts), ts)
    tiny = [t * 2.0 ** -40 for t in ts]
    check_norm(cuda_lib.moe_grad_norm(tiny + ts), tiny + ts)


def test_negative_zeros(cuda_lib):
    for dtype in DTYPES:
        assert float(cuda_lib.moe_grad_norm([torch.full((50_001,), -0.0, dtype=dtype, device=DEV)])) == 0.0
