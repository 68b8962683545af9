"""GPU checks of MXFP4 quantisation and of the experts on MXFP4 operands
against the f64 oracle.

Tolerances, from the arithmetic. Quantised bytes and dequantised values are
exact. A product of n terms accumulates in FP32: at most n * 2^-23 of the sum
of |terms| (one rounding or truncation per addition; the products are exact:
two-bit significands and powers of two). SiLU adds a few FP32 ulps (2^-20 is
allowed), and its slope is at most 1.1. The result is rounded once to the
output type: half an ulp, or half the subnormal step.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle, mxfp4
from tests.parity import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACC = 2.0 ** -23


def u8(t):
    return t.detach().cpu().numpy()


def activations(rows, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    x[:, torch.randint(0, K, (max(1, K // 64),), generator=g)] *= 20.0
    return x.to(dtype)


def special_rows(dtype):
    """Blocks at the edges of the format: zeros, subnormals, the largest values, ties, infinities, NaNs."""
    big = torch.finfo(dtype).max
    tiny = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}[dtype]
    grid = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], dtype=torch.float64)
    both = torch.cat((grid, -grid))
    rows = [torch.zeros(32), -torch.zeros(32), both, both * 2.0 ** -10, both * 3.0, torch.full((32,), big),
            torch.full((32,), tiny), both * tiny * 8, torch.linspace(-7.999, 7.999, 32),
            torch.linspace(-1, 1, 32) * big]
    x = torch.stack([r.double() for r in rows])
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, 32).double()
        r[17] = bad
        x = torch.cat((x, r[None]))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 160), (17, 2048), (130, 1184), (2, 14336)])
def test_quantize_matches_the_oracle(cuda_lib, dtype, rows, K):
    x = activations(rows, K, dtype, rows + K)
    q = cuda_lib.moe_mxfp4_quantize(x.to(DEV))
    codes, scales = mxfp4.quantize(f64(x))
    assert np.array_equal(u8(q.scales), scales)
    assert np.array_equal(u8(q.codes), codes)
    assert np.array_equal(f64(cuda_lib.moe_mxfp4_dequantize(q, torch.float32)), mxfp4.values(codes, scales))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_special_blocks(cuda_lib, dtype):
    x = special_rows(dtype)
    q = cuda_lib.moe_mxfp4_quantize(x.to(DEV))
    codes, scales = mxfp4.quantize(f64(x))
    assert np.array_equal(u8(q.scales), scales)
    assert np.array_equal(u8(q.codes), codes)
    assert (u8(q.scales)[-3:, 0] == 255).all() and not u8(q.codes)[-3:].any()


def test_quantize_leading_dimensions_and_no_rows(cuda_lib):
    moe = cuda_lib
    x = activations(24, 64, torch.bfloat16, 3).to(DEV)
    q = moe.moe_mxfp4_quantize(x.view(2, 3, 4, 64))
    flat = moe.moe_mxfp4_quantize(x)
    assert q.codes.shape == (2, 3, 4, 32) and q.scales.shape == (2, 3, 4, 4)
    assert torch.equal(q.codes.view(24, 32), flat.codes) and torch.equal(q.scales.view(24, 4), flat.scales)
    e = moe.moe_mxfp4_quantize(x[:0])
    assert e.codes.shape == (0, 32) and moe.moe_mxfp4_dequantize(e).shape == (0, 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(cuda_lib, dtype):
    """All 256 scales against all 16 codes; the rounding to the type is torch's from the exact f64 value."""
    codes = np.tile((np.arange(16, dtype=np.uint8) * 17), (256, 1))           # both halves of every byte
    codes[:, 1::2] = codes[:, 1::2] ^ 0x35
    scales = np.zeros((256, 4), dtype=np.uint8)
    scales[:, 0] = np.arange(256)
    v = torch.from_numpy(mxfp4.values(codes, scales)).to(dtype)
    q = cuda_lib.Mxfp4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    got = cuda_lib.moe_mxfp4_dequantize(q, dtype).cpu()
    assert torch.equal(torch.nan_to_num(got, nan=123.0), torch.nan_to_num(v, nan=123.0))


@pytest.mark.parametrize("T,k,K", [(1, 1, 32), (16, 8, 2048), (37, 3, 416)])
def test_quantize_into_dispatched_order(cuda_lib, T, k, K):
    """Rows land where inv says; slots that were not dispatched are skipped
    and their rows keep what was there."""
    moe = cuda_lib
    x = activations(T, K, torch.bfloat16, T)
    g = torch.Generator().manual_seed(5)
    inv = torch.randperm(T * k, generator=g).to(torch.int32)
    skipped = inv[::7].clone()
    inv[::7] = -1
    n = T * k
    out = moe.Mxfp4(torch.full((n, K // 2), 0xA5, dtype=torch.uint8, device=DEV),
                    torch.full((n, mxfp4.scale_pitch(K)), 0x5A, dtype=torch.uint8, device=DEV))
    moe.moe_mxfp4_quantize(x.to(DEV), inv=inv.to(DEV), top_k=k, out=out)
    codes, scales = mxfp4.quantize(f64(x))
    want_c = np.full((n, K // 2), 0xA5, dtype=np.uint8)
    want_s = np.full((n, mxfp4.scale_pitch(K)), 0x5A, dtype=np.uint8)
    for slot, r in enumerate(inv.tolist()):
        if r >= 0:
            want_c[r], want_s[r] = codes[slot // k], scales[slot // k]
    assert skipped.numel() > 0
    assert np.array_equal(u8(out.codes), want_c) and np.array_equal(u8(out.scales), want_s)


# ------------------------------------------------------------------ experts

class Case:
    def __init__(self, E, H, I, counts, seed=0, spread=False):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I = E, H, I
        self.offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int64)
        self.rows = int(self.offsets[-1])

        def draw(rows, K, std):
            v = rng.standard_normal((rows, K)) * std
            if spread:   # blocks of very different sizes: a misplaced scale cannot hide
                v *= np.repeat(2.0 ** rng.integers(-6, 7, (rows, K // 32)), 32, axis=1)
            return mxfp4.quantize(v)

        self.x = draw(self.rows, H, 1.0)
        self.h = draw(self.rows, I, 1.0)
        self.w = [draw(E * n, K, K ** -0.5) for n, K in ((I, H), (I, H), (H, I))]

    def mx(self, moe, pair, lead=None):
        c, s = (torch.from_numpy(a).to(DEV) for a in pair)
        return moe.Mxfp4(*(t.view(lead + (t.shape[-1],)) if lead else t for t in (c, s)))

    def on(self, moe):
        shapes = ((self.E, self.I), (self.E, self.I), (self.E, self.H))
        ex = moe.ExpertsMxfp4(*(self.mx(moe, p, s) for p, s in zip(self.w, shapes)))
        offs = torch.from_numpy(self.offsets).to(torch.int32).to(DEV)
        return ex, offs

    def values(self):
        v = [mxfp4.values(*p) for p in self.w]
        return [v[0].reshape(self.E, self.I, self.H), v[1].reshape(self.E, self.I, self.H),
                v[2].reshape(self.E, self.H, self.I)]


def check(got, ref, err, dtype, what):
    got = f64(got)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    tol = err + HALF_ULP[dtype] * (np.abs(ref) + err) + TINY[dtype]
    bad = np.abs(got - ref) > tol
    bad &= ~np.isnan(ref)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(np.abs(got - ref) / tol)))


def gate_up_bound(c, xv, gate, up):
    """(h, first-order error of h before its rounding)."""
    h, g, u = mxfp4.gate_up(xv, gate, up, c.offsets)
    _, ag, au = mxfp4.gate_up(np.abs(xv), np.abs(gate), np.abs(up), c.offsets)
    eg, eu = ACC * c.H * ag, ACC * c.H * au
    silu = np.abs(g / (1.0 + np.exp(-g)))
    return h, 1.1 * eg * np.abs(u) + (silu + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(h)


SHAPES = [
    (1, 32, 32, [1]),
    (1, 64, 128, [16]),
    (2, 256, 128, [17, 40]),
    (3, 96, 160, [5, 0, 33]),
    (2, 544, 288, [31, 64]),
    (4, 1184, 736, [1, 100, 0, 57]),
    (1, 256, 256, [224]),
    (1, 320, 384, [225]),
    (2, 512, 640, [500, 129]),
    (1, 2048, 256, [130]),
    (40, 288, 160, [3, 0, 1, 2] * 10),           # decode-sized: at most 8 rows an expert
    (64, 512, 384, [75, 1] + [0] * 60 + [2, 2]),  # decode-sized with one long expert
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{s[0]}_H{s[1]}_I{s[2]}_rows{sum(s[3])}")
@pytest.mark.parametrize("spread", [False, True])
def test_down_matches_the_oracle(cuda_lib, shape, dtype, spread):
    moe = cuda_lib
    c = Case(*shape, seed=1, spread=spread)
    ex, offs = c.on(moe)
    y = moe.moe_experts_mxfp4_down(ex, c.mx(moe, c.h), offs, dtype=dtype)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == 0
    hv, w = mxfp4.values(*c.h), c.values()[2]
    ref = mxfp4.down(hv, w, c.offsets)
    err = ACC * c.I * mxfp4.down(np.abs(hv), np.abs(w), c.offsets)
    if dtype == torch.float16:
        assert np.abs(ref).max() < 60000
    check(y, ref, err, dtype, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{s[0]}_H{s[1]}_I{s[2]}_rows{sum(s[3])}")
def test_gate_up_matches_the_oracle(cuda_lib, shape, dtype):
    moe = cuda_lib
    c = Case(*shape, seed=2)
    ex, offs = c.on(moe)
    x = c.mx(moe, c.x)
    h = moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype)
    hq = moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype, quantized=True)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == 0
    gate, up, _ = c.values()
    ref, err = gate_up_bound(c, mxfp4.values(*c.x), gate, up)
    check(h, ref, err, dtype, "h")
    # The quantised output is the quantisation of h, byte for byte (pad bytes too).
    q = moe.moe_mxfp4_quantize(h)
    assert torch.equal(hq.scales, q.scales)
    assert torch.equal(hq.codes, q.codes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("op", ["gate_up", "down"])
@pytest.mark.parametrize("E,H,I,counts", [
    (8, 512, 2048, [700, 300, 900, 1, 0, 450, 1000, 208]),
    (48, 1024, 736, [200 + 3 * i for i in range(48)]),
    (128, 1536, 768, [i % 4 for i in range(128)])])
def test_many_tiles_on_every_sm(cuda_lib, op, dtype, E, H, I, counts):
    """Far more tiles than SMs, so that every ring, accumulator and scale buffer is used over and over: against FP64
    products on the GPU, and the same bits on every one of twelve runs."""
    moe = cuda_lib
    g = torch.Generator(device=DEV).manual_seed(E)
    K, N = (H, I) if op == "gate_up" else (I, H)

    def mx(*lead, K):
        return moe.Mxfp4(torch.randint(0, 256, lead + (K // 2,), dtype=torch.uint8, device=DEV, generator=g),
                         torch.randint(122, 126, lead + (mxfp4.scale_pitch(K),), dtype=torch.uint8, device=DEV,
                                       generator=g))

    w = [mx(E, I, K=H), mx(E, I, K=H), mx(E, H, K=I)]
    ex = moe.ExpertsMxfp4(*w)
    offs = np.concatenate(([0], np.cumsum(counts)))
    a = mx(int(offs[-1]), K=K)
    call = moe.moe_experts_mxfp4_gate_up if op == "gate_up" else moe.moe_experts_mxfp4_down
    o32 = torch.from_numpy(offs).to(torch.int32).to(DEV)
    got = call(ex, a, o32, dtype=dtype)
    for _ in range(11):
        assert torch.equal(got, call(ex, a, o32, dtype=dtype))
    if op == "gate_up":
        hq = call(ex, a, o32, dtype=dtype, quantized=True)
        q = moe.moe_mxfp4_quantize(got)
        assert torch.equal(hq.codes, q.codes) and torch.equal(hq.scales, q.scales)
    f = lambda q: moe.moe_mxfp4_dequantize(q, torch.float32).double()
    av = f(a)
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        m = [f(moe.Mxfp4(t.codes[e], t.scales[e])) for t in w]
        if op == "down":
            ref = av[r] @ m[2].T
            err = ACC * K * (av[r].abs() @ m[2].abs().T)
        else:
            gv, uv = av[r] @ m[0].T, av[r] @ m[1].T
            eg, eu = (ACC * K * (av[r].abs() @ t.abs().T) for t in m[:2])
            s = torch.sigmoid(gv)
            ref = gv * s * uv
            err = 1.1 * eg * uv.abs() + ((gv * s).abs() + 1.1 * eg) * eu + 2.0 ** -20 * ref.abs()
        tol = err + HALF_ULP[dtype] * (ref.abs() + err) + TINY[dtype]
        diff = (got[r].double() - ref).abs()
        if dtype == torch.float16:   # beyond FP16's largest value: infinity
            diff = torch.where(ref.abs() < 65000, diff, 0.0)
        assert bool((diff <= tol).all()), (e, float((diff / tol).max()))
    assert moe.moe_device_status() == 0


def test_forward_dispatched_is_the_two_stages(cuda_lib):
    moe = cuda_lib
    c = Case(5, 416, 544, [70, 0, 3, 230, 16], seed=3)
    ex, offs = c.on(moe)
    x = c.mx(moe, c.x)
    for dtype in DTYPES:
        y = moe.moe_experts_mxfp4_forward_dispatched(ex, x, offs, dtype=dtype)
        hq = moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype, quantized=True)
        assert torch.equal(y, moe.moe_experts_mxfp4_down(ex, hq, offs, dtype=dtype))


def test_rows_behind_the_last_expert_keep_their_contents(cuda_lib):
    """offsets[E] below rows: the rows past it are read by no tile and written by none."""
    moe = cuda_lib
    c = Case(3, 96, 160, [20, 1, 40], seed=4)
    ex, offs = c.on(moe)
    short = offs.clone()
    short[3] = 45
    out = torch.full((c.rows, c.I), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_experts_mxfp4_gate_up(ex, c.mx(moe, c.x), short, dtype=torch.bfloat16, out=out)
    full = moe.moe_experts_mxfp4_gate_up(ex, c.mx(moe, c.x), offs, dtype=torch.bfloat16)
    assert torch.equal(out[:45], full[:45]) and (out[45:] == 7.0).all()


def test_a_nan_block_stays_with_its_token(cuda_lib):
    moe = cuda_lib
    c = Case(2, 288, 160, [30, 9], seed=6)
    ex, offs = c.on(moe)
    x = c.mx(moe, c.x)
    clean = moe.moe_experts_mxfp4_gate_up(ex, x, offs)
    x.scales[11, 4] = 255
    got = moe.moe_experts_mxfp4_gate_up(ex, x, offs)
    assert torch.isnan(got[11]).all()
    keep = [r for r in range(c.rows) if r != 11]
    assert torch.equal(got[keep], clean[keep])
    hq = moe.moe_experts_mxfp4_gate_up(ex, x, offs, quantized=True)
    assert (hq.scales[11, :5] == 255).all() and not hq.codes[11].any()


def test_pad_bytes_of_scales_are_not_read(cuda_lib):
    """K / 32 not a multiple of 4: NaN bytes in the pad of weights and tokens change nothing."""
    moe = cuda_lib
    c = Case(2, 160, 96, [30, 9], seed=7)
    ex, offs = c.on(moe)
    ref = moe.moe_experts_mxfp4_forward_dispatched(ex, c.mx(moe, c.x), offs)
    for p in c.w + [c.x]:
        nb = p[0].shape[1] // 16
        p[1][:, nb:] = 255
    ex2, _ = c.on(moe)
    assert torch.equal(ref, moe.moe_experts_mxfp4_forward_dispatched(ex2, c.mx(moe, c.x), offs))


def test_offsets_that_leave_the_buffers(cuda_lib):
    """offsets[E] past the rows of the buffers: the rows that exist are right, nothing else is touched."""
    moe = cuda_lib
    c = Case(3, 96, 160, [20, 1, 40], seed=8)
    ex, offs = c.on(moe)
    x = c.mx(moe, c.x)
    ref = moe.moe_experts_mxfp4_gate_up(ex, x, offs)
    far = offs.clone()
    far[3] += 300
    guard = torch.full((c.rows + 400, c.I), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_experts_mxfp4_gate_up(ex, x, far, out=guard[:c.rows])
    assert torch.equal(guard[:c.rows], ref) and (guard[c.rows:] == 7.0).all()


def test_both_outputs_of_the_first_stage_at_once(cuda_lib):
    """The C ABI gives h and its quantisation in one call."""
    import ctypes
    moe = cuda_lib
    lib = moe.load_library()
    c = Case(3, 160, 288, [230, 1, 40], seed=9)
    ex, offs = c.on(moe)
    x = c.mx(moe, c.x)
    for dtype, code in ((torch.float32, 0), (torch.float16, 1), (torch.bfloat16, 2)):
        h = torch.empty(c.rows, c.I, dtype=dtype, device=DEV)
        q = moe.Mxfp4(torch.empty(c.rows, c.I // 2, dtype=torch.uint8, device=DEV),
                      torch.empty(c.rows, mxfp4.scale_pitch(c.I), dtype=torch.uint8, device=DEV))
        args = [ctypes.c_void_p(t.data_ptr()) for t in (x.codes, x.scales, offs)]
        st = lib.moe_experts_mxfp4_gate_up(ex.handle, *args, c.rows, code, h.data_ptr(), q.codes.data_ptr(),
                                           q.scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(h, moe.moe_experts_mxfp4_gate_up(ex, x, offs, dtype=dtype))
        ref = moe.moe_mxfp4_quantize(h)
        assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
        # refusals that need a handle: one of the pair missing, no output, misaligned, too many rows
        hp = h.data_ptr()
        for rows, hh, qc, qs, want in ((c.rows, hp, q.codes.data_ptr(), None, 1), (c.rows, None, None, None, 1),
                                       (c.rows, hp + 2, None, None, 5), (1 << 31, hp, None, None, 2),
                                       (-1, hp, None, None, 2)):
            assert lib.moe_experts_mxfp4_gate_up(ex.handle, *args, rows, code, hh, qc, qs, None) == want


@pytest.mark.parametrize("dtype", DTYPES)
def test_buffers_on_16_byte_boundaries(cuda_lib, dtype):
    """Bases that are 16- but not 32-byte aligned (the wide loads and stores do not apply), and odd outputs."""
    moe = cuda_lib
    es = torch.finfo(dtype).bits // 8
    x = activations(7, 224, dtype, 4)
    buf = torch.empty(7 * 224 + 32, dtype=dtype, device=DEV)
    v = buf[16 // es:16 // es + 7 * 224].view(7, 224)
    assert v.data_ptr() % 32 == 16
    v.copy_(x)
    codes, scales = mxfp4.quantize(f64(x))
    q = moe.moe_mxfp4_quantize(v)
    assert np.array_equal(u8(q.codes), codes) and np.array_equal(u8(q.scales), scales)
    back = torch.empty(7 * 224 + 32, dtype=dtype, device=DEV)
    o = back[16 // es:16 // es + 7 * 224].view(7, 224)
    assert torch.equal(moe.moe_mxfp4_dequantize(q, dtype, out=o), moe.moe_mxfp4_dequantize(q, dtype))
    c = Case(2, 64, 96, [5, 30], seed=3)
    ex, offs = c.on(moe)
    out = torch.empty(35 * 96 + 32, dtype=dtype, device=DEV)
    o = out[16 // es:16 // es + 35 * 96].view(35, 96)
    h = moe.moe_experts_mxfp4_gate_up(ex, c.mx(moe, c.x), offs, dtype=dtype)
    assert torch.equal(moe.moe_experts_mxfp4_gate_up(ex, c.mx(moe, c.x), offs, dtype=dtype, out=o), h)


def test_the_largest_expert_count(cuda_lib):
    moe = cuda_lib
    counts = [(7 * e) % 3 for e in range(1024)]
    c = Case(1024, 32, 32, counts, seed=10)
    ex, offs = c.on(moe)
    y = moe.moe_experts_mxfp4_down(ex, c.mx(moe, c.h), offs, dtype=torch.float32)
    hv, w = mxfp4.values(*c.h), c.values()[2]
    check(y, mxfp4.down(hv, w, c.offsets), ACC * c.I * mxfp4.down(np.abs(hv), np.abs(w), c.offsets), torch.float32, "y")


# ------------------------------------------------------------------ the chain

def _layer(moe, E, H, I, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    w = [(torch.randn(E, n, K, generator=g) * K ** -0.5).to(dtype) for n, K in ((I, H), (I, H), (H, I))]
    return moe.ExpertsMxfp4.from_float(*(t.to(DEV) for t in w)), w


@pytest.mark.parametrize("T,E,k,H,I,dtype,renorm", [
    (1, 4, 1, 64, 96, torch.float32, True), (16, 32, 8, 512, 256, torch.bfloat16, True),
    (77, 5, 2, 160, 224, torch.float16, False), (600, 24, 5, 512, 384, torch.bfloat16, True)])
def test_forward_is_its_parts_and_matches_the_oracle(cuda_lib, T, E, k, H, I, dtype, renorm):
    """moe_forward_mxfp4 gives the bits of its split calls; each part matches the oracle (the products stage by
    stage, so that a rounding of h near a border cannot be taken for an error); the combine sums the parts."""
    moe = cuda_lib
    ex, w = _layer(moe, E, H, I, dtype, T)
    x = activations(T, H, dtype, T + 1)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(T + 2)).to(dtype)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    out = moe.moe_forward_mxfp4(ex, x.to(DEV), logits.to(DEV), k, renorm, indices=idx)
    i2, wt, disp = moe.moe_route_dispatch(logits.to(DEV), k, renorm)
    xq = moe.moe_mxfp4_quantize(x.to(DEV), inv=disp.inv, top_k=k)
    hq = moe.moe_experts_mxfp4_gate_up(ex, xq, disp.offsets, dtype=dtype, quantized=True)
    y = moe.moe_experts_mxfp4_forward_dispatched(ex, xq, disp.offsets, dtype=dtype)
    split = moe.moe_combine(y, disp.inv, wt)
    torch.cuda.synchronize()
    assert moe.moe_device_status() == 0
    assert torch.equal(idx, i2) and torch.equal(out, split)

    rt = moe_oracle.route(logits, k, renorm)
    assert (idx.cpu().numpy().view(np.uint32) == rt.indices).all()
    dp = moe_oracle.dispatch(rt.indices, E)
    codes, scales = mxfp4.quantize(f64(x))
    src = dp.row_src.astype(np.int64) // k
    assert np.array_equal(u8(xq.codes), codes[src]) and np.array_equal(u8(xq.scales), scales[src])
    wv = [mxfp4.values(*mxfp4.quantize(f64(t).reshape(-1, t.shape[-1]))).reshape(t.shape) for t in w]
    hv = mxfp4.values(u8(hq.codes), u8(hq.scales))
    offs = dp.offsets.astype(np.int64)
    ref = mxfp4.down(hv, wv[2], offs)
    check(y, ref, ACC * I * mxfp4.down(np.abs(hv), np.abs(wv[2]), offs), dtype, "y")
    rows = dp.inv.astype(np.int64).reshape(T, k)
    yv, wf = f64(y), f64(wt)
    ref = np.einsum("tj,tjh->th", wf, yv[rows])
    check(out, ref, k * ACC * np.einsum("tj,tjh->th", np.abs(wf), np.abs(yv[rows])), dtype, "out")


def test_forward_captured_replayed_and_on_another_stream(cuda_lib):
    moe = cuda_lib
    T, E, k, H, I = 40, 8, 2, 256, 160
    ex, _ = _layer(moe, E, H, I, torch.bfloat16, 9)
    x = [activations(T, H, torch.bfloat16, s).to(DEV) for s in (1, 2)]
    lg = [torch.randn(T, E, generator=torch.Generator().manual_seed(s)).to(DEV) for s in (3, 4)]
    ref = [moe.moe_forward_mxfp4(ex, a, l, k, True) for a, l in zip(x, lg)]
    sx, sl, so = x[0].clone(), lg[0].clone(), torch.empty_like(x[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_mxfp4(ex, sx, sl, k, True, out=so)
    for i in (0, 1, 0):
        sx.copy_(x[i])
        sl.copy_(lg[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(so, ref[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[moe.moe_forward_mxfp4(ex, x[i], lg[i], k, True, stream=s) for _ in range(5)]
            for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, ref[i]) for o in outs[i])


def test_no_tokens(cuda_lib):
    moe = cuda_lib
    ex, _ = _layer(moe, 3, 64, 96, torch.float16, 1)
    x = torch.empty(0, 64, dtype=torch.float16, device=DEV)
    assert moe.moe_forward_mxfp4(ex, x, torch.empty(0, 3, device=DEV), 2, True).shape == (0, 64)
    q = moe.moe_mxfp4_quantize(x)
    offs = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert moe.moe_experts_mxfp4_gate_up(ex, q, offs).shape == (0, 96)
    assert moe.moe_experts_mxfp4_forward_dispatched(ex, q, offs).shape == (0, 64)


def test_refusals_on_the_device(cuda_lib):
    moe = cuda_lib
    ex, _ = _layer(moe, 3, 64, 96, torch.float16, 1)
    q = moe.moe_mxfp4_quantize(torch.zeros(8, 64, device=DEV))
    offs = torch.tensor([0, 8, 8, 8], dtype=torch.int32, device=DEV)
    for bad in (
        lambda: moe.moe_experts_mxfp4_down(ex, q, offs),                                  # K is not I
        lambda: moe.moe_experts_mxfp4_gate_up(ex, q, offs[:3].contiguous()),
        lambda: moe.moe_experts_mxfp4_gate_up(ex, q, offs.long()),
        lambda: moe.moe_experts_mxfp4_gate_up(ex, q, offs, dtype=torch.float64),
        lambda: moe.moe_experts_mxfp4_gate_up(ex, moe.Mxfp4(q.codes, q.scales[:, :2].contiguous()), offs),
        lambda: moe.moe_experts_mxfp4_gate_up(ex, q, offs, out=torch.empty(8, 64, dtype=torch.bfloat16, device=DEV)),
        lambda: moe.moe_experts_mxfp4_forward_dispatched(ex, q, offs,
                                                         workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(8, 64, device=DEV, dtype=torch.float64)),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(8, 48, device=DEV)),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(8, 64, device=DEV), inv=offs, top_k=2),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(8 * 64 + 1, device=DEV)[1:].view(8, 64)),   # not 16-byte aligned
        lambda: moe.moe_forward_mxfp4(ex, torch.zeros(8, 96, device=DEV), torch.zeros(8, 3, device=DEV), 2, True),
        lambda: moe.moe_forward_mxfp4(ex, torch.zeros(8, 64, device=DEV), torch.zeros(8, 4, device=DEV), 2, True),
        lambda: moe.moe_forward_mxfp4(ex, torch.zeros(8, 64, device=DEV), torch.zeros(8, 3, device=DEV), 4, True),
        lambda: moe.ExpertsMxfp4(q, q, q),
    ):
        with pytest.raises(moe.MoeError):
            bad()
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize(torch.zeros(8, 128, device=DEV)[:, ::2])
