"""GPU checks of the orthogonalised updates where they go through the large products: short sides of several tiles and
of several bands of tiles, steps one at a time and by two, wide and tall, into results and into weights. The FP64 steps
run on the GPU too (PyTorch), because these sizes are slow on the CPU.

Tolerance: how far the FP64 result moves when every product of the kernel's own sequence is off by the full size of what
its operands' 22 bits (2^-22 of each entry) and a truncating FP32 accumulator (2^-23 of the sum of the terms' sizes, for
each of the 3 K / 16 additions) may lose, with drawn signs, as a 2-norm over the matrix, times 2 for another draw of the
signs. A result in 16 bits adds half a step of its type for each entry; weights add 3 roundings of 2^-24 (keep, rate,
the sum)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NS = (3.4445, -4.7750, 2.0315)


def by_two(E, r, c):
    """Whether the steps go two at a time (from 2e9 multiplications saved)."""
    s, l = min(r, c), max(r, c)
    return E * s * s * (l - s) > 2e9


def steps_of(x, steps, two, product):
    """`steps` of X <- B X (X B) by `product`, two of them as (B1 B) X where `two`."""
    a, b, c = NS
    tall = x.shape[0] > x.shape[1]
    eye = torch.eye(min(x.shape), dtype=x.dtype, device=x.device)

    def poly(m):
        return a * eye + b * m + c * product(m, m)

    while steps > 0:
        now = 2 if two and steps >= 2 else 1
        steps -= now
        m = product(x.T, x) if tall else product(x, x.T)
        q = poly(m)
        if now == 2:
            q = product(poly(product(product(q, m), q)), q)
        x = product(x, q) if tall else product(q, x)
    return x


def reference(g, steps, two, rng, eps=1e-7):
    """The FP64 result, and how far rounding may move it."""
    def sign(v):
        return 2.0 * torch.randint(0, 2, v.shape, generator=rng, device=DEV, dtype=torch.float64) - 1.0

    def rounded(p, q):
        p, q = (v * (1 + 2.0 ** -22 * sign(v)) for v in (p, q))
        adds = -(-p.shape[1] // 16) * 3
        return p @ q + adds * 2.0 ** -23 * (p.abs() @ q.abs()) * sign(p[:, :1] @ q[:1])

    x = g / (g.square().sum().sqrt() + eps)
    ref = steps_of(x, steps, False, torch.matmul)   # by the definition, one at a time
    return ref, 2 * float((steps_of(x, steps, two, rounded) - ref).norm())


def gradients(seed, E, r, c, dtype):
    """A few strong directions over noise."""
    rng = torch.Generator(DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=rng, device=DEV)
    g = normal(E, r, c) + 3.0 * normal(E, r, 4) @ normal(E, 4, c)
    return (1e-3 * g).to(DTYPES[dtype]), rng


def check(got, g, steps, two, rng):
    u = torch.finfo(got.dtype).eps / 2
    for e in range(len(g)):
        ref, move = reference(g[e].double(), steps, two, rng)
        tol, off = u * ref.abs(), (got[e].double() - ref).abs()
        assert float(off.norm()) <= move + float(tol.norm()), (e, float(off.norm()), move, float(tol.norm()))
        assert bool((off <= move + tol).all())


# two and three row blocks that end inside a tile, by two; a few matrices, one step at a time
@pytest.mark.parametrize("E,r,c", [(2, 600, 5000), (2, 5000, 600), (1, 1000, 3111), (3, 700, 300), (2, 290, 610)])
@pytest.mark.parametrize("steps", [1, 2, 4, 5])
@pytest.mark.parametrize("dtype,out", [("f32", "f16"), ("bf16", "bf16")])
def test_products_of_several_tiles(cuda_lib, E, r, c, steps, dtype, out):
    moe = cuda_lib
    g, rng = gradients(r + steps, E, r, c, dtype)
    o = moe.moe_orthogonalize(g, dtype=DTYPES[out], steps=steps)
    check(o, g, steps, by_two(E, r, c), rng)
    assert moe.moe_device_status() == 0


# 9, 12 and 17 row blocks: past one band of 8, past two; square, and by two
@pytest.mark.parametrize("E,r,c", [(1, 2060, 2100), (1, 2100, 2060), (2, 2060, 4200), (2, 4200, 2060), (1, 2900, 2901),
                                   (1, 4100, 4110)])
def test_products_of_several_bands(cuda_lib, E, r, c):
    moe = cuda_lib
    g, rng = gradients(r, E, r, c, "f32")
    o = moe.moe_orthogonalize(g, dtype=torch.float16, steps=3)
    check(o, g, 3, by_two(E, r, c), rng)
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("E,r,c", [(2, 600, 5000), (2, 5000, 600), (2, 300, 700)])
@pytest.mark.parametrize("wdtype,gdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("steps", [4, 5])
def test_weights_by_products_of_several_tiles(cuda_lib, E, r, c, wdtype, gdtype, steps):
    moe = cuda_lib
    g, rng = gradients(c, E, r, c, gdtype)
    m = 1e-3 * torch.randn(E, r, c, generator=rng, device=DEV)
    w = (torch.randn(E, r, c, generator=rng, device=DEV) / 8).to(DTYPES[wdtype])
    w0, m0 = w.double(), m.double()
    lr, mu, wd, scale = (float(torch.tensor(v, dtype=torch.float32)) for v in (0.02, 0.9, 0.1, 1.5))
    moe.moe_muon_step(w, g, m, lr=lr, momentum_decay=mu, weight_decay=wd, update_scale=scale, steps=steps)
    want = mu * m0 + g.double()
    assert bool(((m.double() - want).abs() <= 2.0 ** -24 * (want.abs() + 2.0 ** -100)).all())   # one fused rounding
    u = g.double() + mu * m.double()
    eps = torch.finfo(w.dtype).eps / 2 + 3 * 2.0 ** -24
    for e in range(E):
        o, move = reference(u[e], steps, by_two(E, r, c), rng)
        ref = (1 - lr * wd) * w0[e] - lr * scale * o
        tol = eps * (((1 - lr * wd) * w0[e]).abs() + (lr * scale * o).abs())
        off = (w[e].double() - ref).abs()
        assert float(off.norm()) <= lr * scale * move + float(tol.norm())
        assert bool((off <= lr * scale * move + tol).all())
    assert moe.moe_device_status() == 0


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
