"""GPU checks of the MXFP4 experts at the ends of their ranges: gates whose exponential leaves FP32, handles dropped
while their work is queued, buffers of another type, buffers past 2^31 elements, the longest rows, every expert chosen,
and the grouped sigmoid routing in front of the 4-bit stages.

Tolerance of SiLU for gates that are exact in FP32 (a sum of a few multiples of 1/4), relative to it. 16-bit outputs: the
exponent |g| log2(e) + 8 carries two roundings (|g| 2^-23 of the power), the hardware's exponential and reciprocal are
off by 2^-22 and 2^-23, four more roundings by 2^-24 each: below 2^-16 for |g| <= 110. FP32: expf within 2 ulp (2^-22),
twice, the reciprocal and two roundings: below 2^-20. A SiLU below 2^-126 (g < -92) may count as 0. u multiplies both;
then comes the output type's own rounding."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle, mxfp4
from tests.parity import f64
from tests.test_gpu_mxfp4 import ACC, DEV, DTYPES, _layer, activations, check, u8

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


# ------------------------------------------------------------------ sizes

def test_buffers_past_2_to_the_31_elements(cuda_lib):
    """Quantise, dequantise and the down product whose last rows lie past 2^31 elements (and past 2^32 bytes)."""
    moe = cuda_lib
    K, rows = 8192, (1 << 31) // 8192 + 37
    tail = torch.randn(64, K, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x = torch.ones(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-64:] = tail.to(DEV)
    q = moe.moe_mxfp4_quantize(x)
    codes, scales = mxfp4.quantize(f64(tail))
    assert np.array_equal(u8(q.codes[-64:]), codes) and np.array_equal(u8(q.scales[-64:]), scales)
    assert bool((q.codes[:-64] == 0x66).all()) and bool((q.scales[:-64] == 125).all())   # 1 = 4 * 2^-2
    v = moe.moe_mxfp4_dequantize(q, out=x)
    assert np.array_equal(f64(v[-64:]), mxfp4.values(codes, scales)) and bool((v[:-64] == 1.0).all())
    # y [rows, 8192] from 32 elements of K: two experts, the second with the last 50 rows
    w = mxfp4.quantize(np.random.default_rng(4).standard_normal((2 * K, 32)))
    mx = lambda p, *lead: moe.Mxfp4(*(torch.from_numpy(a).to(DEV).view(*lead, a.shape[-1]) for a in p))
    gate = mxfp4.quantize(np.ones((64, K)))
    ex = moe.ExpertsMxfp4(mx(gate, 2, 32), mx(gate, 2, 32), mx(w, 2, K))
    h = moe.Mxfp4(q.codes[:, -16:].contiguous(), torch.zeros(rows, 4, dtype=torch.uint8, device=DEV))
    h.scales[:, 0] = q.scales[:, -1]
    hv = mxfp4.values(*(u8(t[-60:]) for t in h))
    del q
    offs = torch.tensor([0, rows - 50, rows], dtype=torch.int32, device=DEV)
    y = moe.moe_experts_mxfp4_down(ex, h, offs, out=x)
    wv = mxfp4.values(*w).reshape(2, K, 32)
    ref = mxfp4.down(hv, wv, np.array([0, 10, 60]))
    check(y[-60:], ref, ACC * 32 * mxfp4.down(np.abs(hv), np.abs(wv), np.array([0, 10, 60])), torch.bfloat16, "y")
    assert moe.moe_device_status() == 0
    # the rows of ones, all alike
    assert torch.equal(y[:-64], y[:1].expand(rows - 64, K))


@pytest.mark.parametrize("quantized", [False, True])
def test_a_first_stage_past_2_to_the_31_elements(cuda_lib, quantized):
    """h [rows, I] with rows * I above 2^31, in BF16 and as codes (one byte for two): every row is the one row that a
    small call gives, two experts share the rows."""
    moe = cuda_lib
    H, I, n, split = 64, 16384, (1 << 31) // 16384 + 301, 90_000
    rng = np.random.default_rng(6)
    mx = lambda p, *lead: moe.Mxfp4(*(torch.from_numpy(a).to(DEV).view(*lead, a.shape[-1]) for a in p))
    gate, up = (mx(mxfp4.quantize(rng.standard_normal((2 * I, H)) * H ** -0.5), 2, I) for _ in range(2))
    ex = moe.ExpertsMxfp4(gate, up, mx(mxfp4.quantize(np.ones((2 * H, I))), 2, H))
    one = moe.moe_mxfp4_quantize(torch.from_numpy(rng.standard_normal((1, H))).to(torch.bfloat16).to(DEV))
    rep = lambda r: moe.Mxfp4(*(t.expand(r, t.shape[1]).contiguous() for t in one))
    offs = lambda *o: torch.tensor(o, dtype=torch.int32, device=DEV)
    call = lambda x, o: moe.moe_experts_mxfp4_gate_up(ex, x, o, quantized=quantized)
    few, many = call(rep(2), offs(0, 1, 2)), call(rep(n), offs(0, split, n))
    for f, m in zip(*((few, many) if quantized else ((few,), (many,)))):
        assert torch.equal(m[:split], f[:1].expand(split, f.shape[1]))
        assert torch.equal(m[split:], f[1:].expand(n - split, f.shape[1]))
        assert not torch.equal(f[0], f[1])
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("H,I", [(262144, 32), (32, 262144)])
def test_the_longest_rows(cuda_lib, H, I):
    """K = 262144 in either stage (1024 stages a tile, rows of 128 KB of codes) and as many output columns."""
    moe = cuda_lib
    rows, g = 5, torch.Generator().manual_seed(7)
    x = torch.randn(rows, H, generator=g).to(torch.bfloat16)
    w = [(torch.randn(1, n, K, generator=g) * K ** -0.5).to(torch.bfloat16) for n, K in ((I, H), (I, H), (H, I))]
    ex = moe.ExpertsMxfp4.from_float(*(t.to(DEV) for t in w))
    offs = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    q = moe.moe_mxfp4_quantize(x.to(DEV))
    codes, scales = mxfp4.quantize(f64(x))
    assert np.array_equal(u8(q.codes), codes) and np.array_equal(u8(q.scales), scales)
    hq = moe.moe_experts_mxfp4_gate_up(ex, q, offs, dtype=torch.float32, quantized=True)
    h = moe.moe_experts_mxfp4_gate_up(ex, q, offs, dtype=torch.float32)
    qh = moe.moe_mxfp4_quantize(h)
    assert torch.equal(hq.codes, qh.codes) and torch.equal(hq.scales, qh.scales)
    y = moe.moe_experts_mxfp4_down(ex, hq, offs, dtype=torch.float32)
    wv = [mxfp4.values(*mxfp4.quantize(f64(t)[0]))[None] for t in w]
    xv, hv, o = mxfp4.values(codes, scales), mxfp4.values(u8(hq.codes), u8(hq.scales)), np.array([0, rows])
    href, gv, uv = mxfp4.gate_up(xv, wv[0], wv[1], o)
    _, ag, au = mxfp4.gate_up(np.abs(xv), np.abs(wv[0]), np.abs(wv[1]), o)
    eg, eu = ACC * H * ag, ACC * H * au
    silu = np.abs(gv / (1.0 + np.exp(-gv)))
    check(h, href, 1.1 * eg * np.abs(uv) + (silu + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(href), torch.float32, "h")
    check(y, mxfp4.down(hv, wv[2], o), ACC * I * mxfp4.down(np.abs(hv), np.abs(wv[2]), o), torch.float32, "y")


@pytest.mark.parametrize("E,k", [(128, 128), (1024, 1024)])
def test_forward_with_every_expert_chosen(cuda_lib, E, k):
    """top_k = E: the whole forward gives the bits of its split calls."""
    moe = cuda_lib
    T, H, I = 7, 64, 32
    ex, _ = _layer(moe, E, H, I, torch.bfloat16, 31)
    x = activations(T, H, torch.bfloat16, 32).to(DEV)
    lg = torch.randn(T, E, generator=torch.Generator().manual_seed(33)).to(DEV)
    out = moe.moe_forward_mxfp4(ex, x, lg, k, True)
    idx, wt = moe.moe_route(lg, k, True)
    disp = moe.moe_dispatch(idx, E)
    xq = moe.moe_mxfp4_quantize(x, inv=disp.inv, top_k=k)
    y = moe.moe_experts_mxfp4_forward_dispatched(ex, xq, disp.offsets)
    assert torch.equal(out, moe.moe_combine(y, disp.inv, wt)) and bool(torch.isfinite(out).all())
    assert moe.moe_device_status() == 0


# ------------------------------------------------------------------ the other routing

def test_grouped_sigmoid_routing_in_front_of_the_4_bit_stages(cuda_lib):
    """The split calls together: grouped routing with its dispatch, quantise, both products, combine."""
    moe = cuda_lib
    T, E, k, H, I = 200, 16, 4, 512, 384
    ex, w = _layer(moe, E, H, I, torch.bfloat16, 21)
    x = activations(T, H, torch.bfloat16, 22)
    g = torch.Generator().manual_seed(23)
    logits, bias = torch.randn(T, E, generator=g), torch.randn(E, generator=g) * 0.1
    opt = moe.GroupRoutingOptions(k, 4, 2, group_top_two=True, renormalize=True, scale=2.5)
    idx, wt, disp = moe.moe_route_sigmoid_grouped_dispatch(logits.to(DEV), bias.to(DEV), opt)
    xq = moe.moe_mxfp4_quantize(x.to(DEV), inv=disp.inv, top_k=k)
    hq = moe.moe_experts_mxfp4_gate_up(ex, xq, disp.offsets, quantized=True)
    y = moe.moe_experts_mxfp4_forward_dispatched(ex, xq, disp.offsets)
    out = moe.moe_combine(y, disp.inv, wt)
    assert torch.equal(y, moe.moe_experts_mxfp4_down(ex, hq, disp.offsets))
    dp = moe_oracle.dispatch(idx.cpu().numpy().view(np.uint32), E)
    codes, scales = mxfp4.quantize(f64(x))
    src = dp.row_src.astype(np.int64) // k
    assert np.array_equal(u8(xq.codes), codes[src]) and np.array_equal(u8(xq.scales), scales[src])
    offs = dp.offsets.astype(np.int64)
    wv = [mxfp4.values(*mxfp4.quantize(f64(t).reshape(-1, t.shape[-1]))).reshape(t.shape) for t in w]
    hv = mxfp4.values(u8(hq.codes), u8(hq.scales))
    check(y, mxfp4.down(hv, wv[2], offs), ACC * I * mxfp4.down(np.abs(hv), np.abs(wv[2]), offs), torch.bfloat16, "y")
    rows = dp.inv.astype(np.int64).reshape(T, k)
    yv, wf = f64(y), f64(wt)
    check(out, np.einsum("tj,tjh->th", wf, yv[rows]),
          k * ACC * np.einsum("tj,tjh->th", np.abs(wf), np.abs(yv[rows])), torch.bfloat16, "out")
