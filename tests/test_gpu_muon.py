"""GPU checks of the orthogonalised updates against the FP64 steps (oracle/block.py).

Tolerance: how far the FP64 result moves when every product of it is off by the full size of what its operands' 22 bits
and a truncating FP32 accumulator may lose, with drawn signs (oracle.block.newton_schulz_moved), as a 2-norm over the
matrix, times 2 for another draw of the signs. A BF16 result's last product has operands of 11 bits, each off by at
most half a step of FP16, 2^-11: each term by (1 + 2^-11)^2 - 1 < 2^-10 (1 + 2^-11), the product by that of the sum of
its terms' sizes. A result in 16 bits adds half a step of its type for each entry. FP32
weights add 3 roundings of 2^-24 (keep, rate, the sum)."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def gradients(rng, E, r, c, dtype, scale=1e-3):
    """A few strong directions over noise."""
    k = min(4, r, c)
    g = rng.normal(size=(E, r, c)) + 3.0 * rng.normal(size=(E, r, k)) @ rng.normal(size=(E, k, c))
    return torch.tensor(g * scale, dtype=DTYPES[dtype], device=DEV)


def last_product(m, dtype, steps=5, eps=1e-7):
    """What a BF16 result's last product may be off by."""
    if dtype != torch.bfloat16:
        return 0.0
    return 2.0 ** -10 * (1 + 2.0 ** -11) * block.newton_schulz_last_size(m, steps, eps)


def check_matrices(got, inputs, rng, u=None, steps=5, eps=1e-7):
    """got [E, r, c] against the FP64 steps on inputs (numpy [E, r, c])."""
    u = torch.finfo(got.dtype).eps / 2 if u is None else u
    g = f64(got)
    for e, m in enumerate(inputs):
        ref = block.newton_schulz(m, steps, eps)
        move = 2 * np.linalg.norm(block.newton_schulz_moved(m, rng, steps, eps) - ref)
        tol = u * np.abs(ref) + last_product(m, got.dtype, steps, eps) * (1 + u)
        off = np.abs(g[e] - ref)
        assert np.linalg.norm(off) <= move + np.linalg.norm(tol), (e, np.linalg.norm(off), move, np.linalg.norm(tol))
        assert (off <= move + tol).all()


# one entry; vectors; under one MMA; ends inside and at tile borders, wide, tall and square; K over many blocks
SHAPES = [(1, 1, 1), (2, 1, 5), (2, 5, 1), (3, 7, 9), (1, 16, 16), (2, 33, 130), (2, 130, 33), (2, 127, 128),
          (1, 128, 128), (2, 129, 257), (2, 257, 129), (1, 256, 256), (1, 260, 300), (3, 64, 1000), (3, 1000, 64),
          (1, 385, 520), (1, 640, 385), (1, 40, 5000), (1, 5000, 40), (37, 24, 40)]


@pytest.mark.parametrize("E,r,c", SHAPES)
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f16"), ("f16", "bf16")])
def test_orthogonalize(cuda_lib, E, r, c, dtype, out):
    moe = cuda_lib
    rng = np.random.default_rng(E * r * c)
    g = gradients(rng, E, r, c, dtype)
    o = moe.moe_orthogonalize(g, dtype=DTYPES[out])
    assert o.shape == g.shape and o.dtype == DTYPES[out]
    check_matrices(o, f64(g), rng)
    assert moe.moe_device_status() == 0


# short sides up to 128 take one launch: each size of cluster, its blocks' columns whole, ragged and none at all; sides
# that end inside 16; a long side past what a cluster holds; more clusters than run at once, and too many
SMALL = [(1, 128, 2048), (1, 2048, 128), (2, 100, 1537), (2, 1537, 100), (1, 128, 3000), (1, 3000, 97), (1, 17, 2999),
         (1, 17, 3100), (2, 113, 769), (2, 769, 113), (5, 90, 385), (5, 385, 90), (4, 128, 192), (4, 193, 128),
         (3, 1, 192), (3, 700, 1), (160, 31, 65), (160, 65, 31), (20, 20, 700), (30, 128, 2048), (1, 129, 2048)]


@pytest.mark.parametrize("E,r,c", SMALL)
@pytest.mark.parametrize("dtype,out", [("f32", "f16"), ("bf16", "bf16")])
def test_short_sides(cuda_lib, E, r, c, dtype, out):
    moe = cuda_lib
    rng = np.random.default_rng(E + r * c)
    g = gradients(rng, E, r, c, dtype)
    behind = torch.full((E * r * c + 64,), 7.0, dtype=DTYPES[out], device=DEV)
    o = moe.moe_orthogonalize(g, out=behind[:E * r * c].view(E, r, c))
    check_matrices(o[:3], f64(g[:3]), rng)
    check_matrices(o[-1:], f64(g[-1:]), rng)
    assert (behind[E * r * c:] == 7.0).all()
    assert torch.equal(o, moe.moe_orthogonalize(g, dtype=DTYPES[out]))
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("E,r,c", [(40, 64, 300), (40, 300, 64), (3, 128, 1000)])
@pytest.mark.parametrize("dtype,out,shift", [("bf16", "bf16", 0), ("f32", "bf16", 0), ("f32", "f16", 1), ("f16", "f16", 3)])
def test_short_sides_over_their_inputs(cuda_lib, E, r, c, dtype, out, shift):
    """The result over the matrices' own memory, of the same or another element size, at its start or `shift` in."""
    moe = cuda_lib
    rng = np.random.default_rng(r)
    n = E * r * c
    g = torch.empty(n + 8, dtype=DTYPES[dtype], device=DEV)
    g[:n] = gradients(rng, E, r, c, dtype).view(-1)
    inputs = f64(g[:n].view(E, r, c))
    o = g.view(DTYPES[out])[shift:shift + n].view(E, r, c)
    moe.moe_orthogonalize(g[:n].view(E, r, c), out=o)
    check_matrices(o[:2], inputs[:2], rng)
    check_matrices(o[E // 2:E // 2 + 2], inputs[E // 2:E // 2 + 2], rng)
    check_matrices(o[-1:], inputs[-1:], rng)
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("E,r,c", [(1, 128, 2048), (3, 515, 77), (50, 48, 130)])
@pytest.mark.parametrize("wdtype,gdtype", [("f32", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_short_sides_muon_step(cuda_lib, E, r, c, wdtype, gdtype):
    """As test_muon_step, at the sizes that take one launch; the matrices at the ends and in the middle."""
    moe = cuda_lib
    rng = np.random.default_rng(r + c)
    w = torch.tensor(rng.normal(size=(E, r, c)) / 8, dtype=DTYPES[wdtype], device=DEV)
    m = torch.tensor(rng.normal(size=(E, r, c)) * 1e-3, dtype=torch.float32, device=DEV)
    g = gradients(rng, E, r, c, gdtype)
    w0, m0, g0 = f64(w), f64(m), f64(g)
    lr, mu, wd, scale = (float(np.float32(v)) for v in (0.02, 0.9, 0.1, 1.5))
    moe.moe_muon_step(w, g, m, lr=lr, momentum_decay=mu, weight_decay=wd, update_scale=scale)
    got_m, got = f64(m), f64(w)
    assert (np.abs(got_m - (mu * m0 + g0)) <= 2.0 ** -24 * (np.abs(mu * m0 + g0) + 2.0 ** -100)).all()
    keep, rate = float(np.float32(1 - lr * wd)), float(np.float32(lr * scale))
    for e in {0, E // 2, E - 1}:
        u = g0[e] + mu * got_m[e]
        o = block.newton_schulz(u)
        move = 2 * np.linalg.norm(block.newton_schulz_moved(u, rng) - o) + last_product(u, w.dtype)
        eps = torch.finfo(w.dtype).eps / 2 + 3 * 2.0 ** -24
        tol = eps * (np.abs(keep * w0[e]) + np.abs(rate * o)) + rate * move
        assert (np.abs(got[e] - (keep * w0[e] - rate * o)) <= tol).all()
    assert moe.moe_device_status() == 0


def test_short_sides_of_the_most_matrices(cuda_lib):
    """65535 matrices, past 2^31 bytes: the first, one in the middle and the last."""
    moe = cuda_lib
    rng = np.random.default_rng(21)
    some = gradients(rng, 7, 128, 128, "bf16")
    g = some[torch.arange(65535, device=DEV) % 7]
    o = moe.moe_orthogonalize(g, out=g)
    for e in (0, 40000, 65534):
        check_matrices(o[e:e + 1], f64(some[e % 7:e % 7 + 1]), rng)
    assert torch.equal(o[7:14], o[:7]) and torch.equal(o[-7:], o[1:8])
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("steps", [1, 2, 8])
@pytest.mark.parametrize("r,c", [(60, 200), (200, 60)])
def test_steps(cuda_lib, steps, r, c):
    moe = cuda_lib
    rng = np.random.default_rng(steps)
    g = gradients(rng, 2, r, c, "f32")
    check_matrices(moe.moe_orthogonalize(g, dtype=torch.float16, steps=steps), f64(g), rng, steps=steps)


@pytest.mark.parametrize("scale", [1e-30, 1e-19, 1e-3, 1e15, 1e30])
def test_scales_that_fp32_squares_leave(cuda_lib, scale):
    """eps far below the smallest norm: the result does not depend on the gradients' scale."""
    moe = cuda_lib
    rng = np.random.default_rng(11)
    g = gradients(rng, 2, 48, 80, "f32", scale)
    check_matrices(moe.moe_orthogonalize(g, dtype=torch.float16, eps=1e-37), f64(g), rng, eps=1e-37)


def test_eps_counts_for_small_gradients(cuda_lib):
    moe = cuda_lib
    rng = np.random.default_rng(12)
    g = gradients(rng, 1, 32, 32, "f32", 1e-8)
    check_matrices(moe.moe_orthogonalize(g, eps=1e-5), f64(g), rng, eps=1e-5)


@pytest.mark.parametrize("r,c", [(40, 72), (72, 40), (300, 280)])
def test_zeros_and_bad_values_stay_in_their_matrix(cuda_lib, r, c):
    moe = cuda_lib
    rng = np.random.default_rng(13)
    g = gradients(rng, 5, r, c, "bf16")
    good = moe.moe_orthogonalize(g)
    g[1] = 0
    g[2, r // 2, 3] = float("nan")
    g[4, 0, 0] = float("-inf")
    o = moe.moe_orthogonalize(g)
    assert (o[1] == 0).all() and torch.isnan(o[2]).all() and torch.isnan(o[4]).all()
    assert torch.equal(o[[0, 3]], good[[0, 3]])


def test_out_in_the_inputs_memory_and_what_lies_behind(cuda_lib):
    moe = cuda_lib
    rng = np.random.default_rng(14)
    g = gradients(rng, 3, 70, 50, "bf16")
    ref = moe.moe_orthogonalize(g)
    big = torch.full((5, 70, 50), 7.0, dtype=torch.bfloat16, device=DEV)
    big[:3] = g
    assert moe.moe_orthogonalize(big[:3], out=big[:3]).data_ptr() == big.data_ptr()
    assert torch.equal(big[:3], ref) and (big[3:] == 7).all()
    # one element past a 16-byte boundary
    off = torch.empty(g.numel() + 1, dtype=g.dtype, device=DEV)[1:].view_as(g)
    off.copy_(g)
    assert torch.equal(moe.moe_orthogonalize(off), ref)
    assert torch.equal(moe.moe_orthogonalize(g.view(3, 1, 70, 50)), ref.view(3, 1, 70, 50))
    assert torch.equal(moe.moe_orthogonalize(g[0]), ref[0])


def test_nothing_to_do(cuda_lib):
    moe = cuda_lib
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        e = torch.empty(shape, device=DEV)
        assert moe.moe_orthogonalize(e).shape == shape
        assert moe.moe_muon_step(e, e.clone(), e.clone(), lr=0.1) is e


@pytest.mark.parametrize("E,r,c", [(2, 96, 64), (3, 45, 130), (1, 300, 260)])
@pytest.mark.parametrize("wdtype,gdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step(cuda_lib, E, r, c, wdtype, gdtype, nesterov):
    moe = cuda_lib
    rng = np.random.default_rng(r + c)
    w = torch.tensor(rng.normal(size=(E, r, c)) / 8, dtype=DTYPES[wdtype], device=DEV)
    m = torch.tensor(rng.normal(size=(E, r, c)) * 1e-3, dtype=torch.float32, device=DEV)
    lr, mu, wd = 0.02, 0.9, 0.1
    scale = max(1.0, r / c) ** 0.5
    for _ in range(2):
        g = gradients(rng, E, r, c, gdtype)
        w0, m0 = f64(w), f64(m)
        assert moe.moe_muon_step(w, g, m, lr=lr, momentum_decay=mu, nesterov=nesterov, weight_decay=wd) is w
        mu32 = float(np.float32(mu))
        ref_m = mu32 * m0 + f64(g)
        got_m = f64(m)
        assert (np.abs(got_m - ref_m) <= 2.0 ** -24 * (np.abs(ref_m) + 2.0 ** -100)).all()   # one fused rounding
        u = f64(g) + mu32 * got_m if nesterov else got_m
        keep, rate = (float(np.float32(v)) for v in (1 - float(np.float32(lr)) * float(np.float32(wd)),
                                                     float(np.float32(lr)) * float(np.float32(scale))))
        for e in range(E):
            o = block.newton_schulz(u[e])
            move = 2 * np.linalg.norm(block.newton_schulz_moved(u[e], rng) - o) + last_product(u[e], w.dtype)
            # u itself is rounded once, 2^-24 of it: less than the operands' 2^-22 that `move` has
            ref = keep * w0[e] - rate * o
            eps = torch.finfo(w.dtype).eps / 2 + 3 * 2.0 ** -24
            tol = eps * (np.abs(keep * w0[e]) + np.abs(rate * o)) + rate * move
            assert (np.abs(f64(w)[e] - ref) <= tol).all()


def test_muon_orthogonalizes_what_orthogonalize_does(cuda_lib):
    """momentum_decay 0 and weights of zeros: the FP32 weights rounded are moe_orthogonalize's bits."""
    moe = cuda_lib
    rng = np.random.default_rng(15)
    for r, c in ((90, 200), (200, 90)):
        g = gradients(rng, 2, r, c, "f32")
        w, m = torch.zeros_like(g), torch.ones_like(g)
        moe.moe_muon_step(w, g, m, lr=-1.0, momentum_decay=0.0, update_scale=1.0)
        assert torch.equal(m, g)
        assert torch.equal(w.to(torch.float16), moe.moe_orthogonalize(g, dtype=torch.float16))


def test_more_than_2_31_elements(cuda_lib):
    moe = cuda_lib
    E, r, c = 2100, 64, 16400
    g = torch.zeros(E, r, c, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(16)
    last = gradients(rng, 2, r, c, "bf16")
    g[0], g[-1] = last[0], last[1]
    o = moe.moe_orthogonalize(g, out=g)
    check_matrices(o[-1:], f64(last[1:]), rng)
    check_matrices(o[:1], f64(last[:1]), rng)
    assert (o[E // 2] == 0).all() and (o[-2] == 0).all()


def test_streams_graphs_and_repeats(cuda_lib):
    moe = cuda_lib
    rng = np.random.default_rng(17)
    a, b = gradients(rng, 6, 300, 200, "f32"), gradients(rng, 2, 100, 700, "bf16")
    ref = [moe.moe_orthogonalize(t) for t in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [moe.moe_orthogonalize(a, stream=side), moe.moe_orthogonalize(b)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    graphs, outs = [], []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(moe.moe_orthogonalize(t))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, outs))
    assert moe.moe_device_status() == 0


def test_refusals_of_the_binding(cuda_lib):
    moe = cuda_lib
    g = torch.zeros(2, 16, 24, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g.transpose(1, 2))
    with pytest.raises(ValueError):
        moe.moe_orthogonalize(g.cpu())
    bad = [
        lambda: moe.moe_orthogonalize(g[0, 0]),
        lambda: moe.moe_orthogonalize(g, dtype=torch.float32),
        lambda: moe.moe_orthogonalize(g, dtype=torch.float64),
        lambda: moe.moe_orthogonalize(g.double()),
        lambda: moe.moe_orthogonalize(g, out=torch.empty(2, 24, 16, dtype=torch.bfloat16, device=DEV)),
        lambda: moe.moe_orthogonalize(g, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
        lambda: moe.moe_orthogonalize(g, steps=0),
        lambda: moe.moe_muon_step(g, g, torch.zeros_like(g), lr=0.1),
        lambda: moe.moe_muon_step(g, g.clone(), torch.zeros_like(g).bfloat16(), lr=0.1),
        lambda: moe.moe_muon_step(g, g.clone()[:1], torch.zeros_like(g), lr=0.1),
        lambda: moe.moe_muon_step(g, g.clone(), torch.zeros_like(g), lr=float("nan")),
        lambda: moe.moe_muon_step(g, g.clone(), torch.zeros_like(g), lr=0.1, momentum_decay=1.0),
    ]
    for call in bad:
        with pytest.raises(moe.MoeError):
            call()
