"""GPU checks of the MXFP4 experts at the ends of their ranges: gates whose exponential leaves FP32, handles dropped
while their work is queued, and buffers of another type.

Tolerance of SiLU for gates that are exact in FP32 (a sum of a few multiples of 1/4), relative to it. 16-bit outputs: the
exponent |g| log2(e) + 8 carries two roundings (|g| 2^-23 of the power), the hardware's exponential and reciprocal are
off by 2^-22 and 2^-23, four more roundings by 2^-24 each: below 2^-16 for |g| <= 110. FP32: expf within 2 ulp (2^-22),
twice, the reciprocal and two roundings: below 2^-20. A SiLU below 2^-126 (g < -92) may count as 0. u multiplies both;
then comes the output type's own rounding."""
import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.test_gpu_mxfp4 import DEV, DTYPES, _layer, activations, check

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ SiLU

def _gates():
    """Multiples of 1/4: where e^-g leaves FP32's normal range and then FP32, and ordinary gates of both signs."""
    far = np.arange(-110.0, -79.75, 0.25)
    near = np.concatenate((np.arange(-79.0, -1.0, 3.25), np.arange(-1.0, 1.25, 0.25), np.arange(2.0, 110.0, 6.75)))
    return np.concatenate((far, near))


def _weights(values):
    """MXFP4 rows [n, 64] whose elements sum to the values: multiples of 8 in the first block, of 1/4 in the second."""
    n = len(values)
    codes = np.zeros((n, 64), dtype=np.uint8)
    scales = np.zeros((n, 4), dtype=np.uint8)
    scales[:, 0], scales[:, 1] = 127 + 4, 127 - 1
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for r, v in enumerate(values):
        left, sign = abs(v), 8 if v < 0 else 0
        for start, unit in ((0, 16.0), (32, 0.5)):
            i = start
            for c in range(7, 0, -1):
                while left >= grid[c] * unit:
                    codes[r, i] = c | sign
                    left -= grid[c] * unit
                    i += 1
            assert i < start + 32
        assert left == 0
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def _silu_layer(moe, g, ue):
    """(experts, x of three rows of ones, offsets) whose gates are g [I] and whose u is 2^ue [I], both exactly."""
    I = len(g)
    gate = _weights(g)
    assert np.array_equal(mxfp4.values(*gate).sum(1), g)
    up = np.zeros((I, 32), dtype=np.uint8), np.zeros((I, 4), dtype=np.uint8)
    up[0][:, 0] = 2                                                                 # 1
    up[1][:, 0] = 127 + ue
    x = np.full((3, 32), 0x22, dtype=np.uint8), np.zeros((3, 4), dtype=np.uint8)    # ones
    x[1][:, :2] = 127
    mx = lambda p, *lead: moe.Mxfp4(*(torch.from_numpy(a).to(DEV).view(*lead, a.shape[-1]) for a in p))
    ex = moe.ExpertsMxfp4(mx(gate, 1, I), mx(up, 1, I), mx(mxfp4.quantize(np.ones((64, I))), 1, 64))
    return ex, mx(x, 3), torch.tensor([0, 3], dtype=torch.int32, device=DEV)


def _padded_gates():
    g = _gates()
    return np.concatenate((g, np.zeros(-len(g) % 32)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_silu_of_large_negative_gates(cuda_lib, dtype):
    """h = SiLU(g) u is a normal number of the type once u is large, where e^-g has left FP32."""
    moe = cuda_lib
    g = _padded_gates()
    ue = np.where(g < -79.5, 112, 0)
    ex, x, offs = _silu_layer(moe, g, ue)
    h = moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype)
    u = 2.0 ** ue
    ref = np.where(g < 0, g * np.exp(-np.abs(g)), g) / (1.0 + np.exp(-np.abs(g))) * u
    assert np.abs(ref).max() < 60000
    err = 2.0 ** (-20 if dtype == torch.float32 else -16) * np.abs(ref)
    err += np.where(np.abs(ref / u) < 2.0 ** -126, 2.0 ** -126, 2.0 ** -150) * u
    check(h, np.tile(ref, (3, 1)), np.tile(err, (3, 1)), dtype, "h")
    hq = moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype, quantized=True)
    q = moe.moe_mxfp4_quantize(h)
    assert torch.equal(hq.codes, q.codes) and torch.equal(hq.scales, q.scales)


@pytest.mark.parametrize("dtype", DTYPES)
def test_silu_does_not_depend_on_its_neighbours(cuda_lib, dtype):
    """The bits of an ordinary gate's h are the same with and without large negative gates around it."""
    moe = cuda_lib
    rng = np.random.default_rng(5)
    g = np.round(rng.uniform(-79.0, 79.0, 256) * 4) / 4
    among = g.copy()
    far = rng.random(256) < 0.25
    among[far] = -95.0
    zero = np.zeros(256, dtype=np.int64)
    h = [moe.moe_experts_mxfp4_gate_up(*_silu_layer(moe, v, zero), dtype=dtype) for v in (g, among)]
    keep = torch.from_numpy(~far).to(DEV)
    assert torch.equal(h[0][:, keep], h[1][:, keep]) and not torch.equal(h[0], h[1])


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
