"""GPU checks of the gradient norm and clip against f64 sums.

Tolerances, from the arithmetic: a thread's group of 16 (32) squares is summed
in FP32 (each square's and addition's rounding: at most 33 * 2^-24 of a sum of
positive terms), everything above in FP64, the root is rounded once to FP32:
|norm - exact| <= (33 / 2 + 1) * 2^-24 of it. A clipped element has the
factor's error, half an ulp of the division and of the FP32 product, and half
an ulp of its type.
"""
import numpy as np
import pytest
import torch

from oracle import mxfp4
from tests.parity import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
NORM_TOL = 17.5 * 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def grads(sizes, seed, scale=0.02):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(d).to(DEV) for n, d in sizes]


def exact(ts):
    return mxfp4.grad_norm([f64(t) for t in ts])


def check_norm(got, ts):
    ref = exact(ts)
    assert abs(float(got) - ref) <= NORM_TOL * ref + 2.0 ** -150, (float(got), ref)


def check_clip(out, ts, norm, max_norm):
    f = max_norm / norm if norm > max_norm else 1.0
    for o, t in zip(out, ts):
        ref = f64(t) * f
        tol = (NORM_TOL + 3 * 2.0 ** -24 + HALF_ULP[t.dtype]) * np.abs(ref) + TINY[t.dtype]
        assert o.dtype == t.dtype and (np.abs(f64(o) - ref) <= tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 17, 511, 4097, 8192, 16385, 100003])
def test_norm_and_clip_of_one_tensor(cuda_lib, dtype, n):
    moe = cuda_lib
    ts = grads([(n, dtype)], n)
    norm = moe.moe_grad_norm(ts)
    check_norm(norm, ts)
    out = [torch.full_like(t, 5.0) for t in ts]
    got = moe.moe_clip_grad_norm(ts, float(norm) / 3, out=out)
    assert torch.equal(got, norm)
    check_clip(out, ts, exact(ts), float(norm) / 3)


@pytest.mark.parametrize("n_tensors", [0, 1, 5, 127, 128, 129, 300])
def test_many_tensors_of_mixed_types(cuda_lib, n_tensors):
    """More tensors than one launch's table, empty ones among them."""
    moe = cuda_lib
    rng = np.random.default_rng(n_tensors)
    sizes = [(int(rng.integers(0, 4000)) * int(rng.integers(0, 2)) + int(rng.integers(0, 3)), DTYPES[i % 3])
             for i in range(n_tensors)]
    ts = grads(sizes, 3)
    norm = moe.moe_grad_norm(ts)
    if n_tensors == 0:
        assert float(norm) == 0.0
        return
    check_norm(norm, ts)
    keep = [t.clone() for t in ts]
    got = moe.moe_grad_clip(ts, norm, float(norm) * 0.25)
    assert all(a is b for a, b in zip(got, ts))
    check_clip(ts, keep, exact(keep), float(norm) * 0.25)


def test_views_at_every_alignment(cuda_lib):
    """Views that start off a 16-byte boundary, source and destination differently; their neighbours keep their
    values."""
    moe = cuda_lib
    for dtype in DTYPES:
        for a in range(0, 9):
            for b in (0, 1, a):
                src = grads([(70000, dtype)], a)[0]
                dst = torch.full((70000,), 9.0, dtype=dtype, device=DEV)
                s, d = src[a:a + 65001], dst[b:b + 65001]
                norm = moe.moe_clip_grad_norm([s], 0.5, out=[d])
                check_norm(norm, [s])
                check_clip([d], [s], exact([s]), 0.5)
                assert (dst[:b] == 9.0).all() and (dst[b + 65001:] == 9.0).all()


@pytest.mark.parametrize("dtype,scale", [(torch.float32, 1e30), (torch.float32, 1e-30), (torch.float32, 1e-42),
                                         (torch.bfloat16, 1e30), (torch.bfloat16, 1e-35), (torch.float16, 1e-7),
                                         (torch.float16, 1e4)])
def test_magnitudes_whose_squares_leave_fp32(cuda_lib, dtype, scale):
    ts = grads([(5000, dtype), (3, dtype), (40000, dtype)], 4, scale)
    ts[2][:20000] = 0
    check_norm(cuda_lib.moe_grad_norm(ts), ts)


def test_zero_gradients(cuda_lib):
    moe = cuda_lib
    ts = [torch.zeros(100000, device=DEV), -torch.zeros(77, device=DEV, dtype=torch.bfloat16)]
    out = [torch.ones_like(t) for t in ts]
    assert float(moe.moe_clip_grad_norm(ts, 1.0, out=out)) == 0.0
    assert not any(o.any() for o in out)
    assert float(moe.moe_clip_grad_norm(ts, 0.0, out=out)) == 0.0


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(cuda_lib, bad):
    moe = cuda_lib
    ts = grads([(5000, torch.float32), (300, torch.bfloat16)], 5)
    ts[0][4321] = bad
    keep = [t.clone() for t in ts]
    norm = moe.moe_clip_grad_norm(ts, 1e-3)
    assert torch.equal(torch.isnan(norm), torch.isnan(torch.tensor(bad, device=DEV))) and not torch.isfinite(norm)
    for t, k in zip(ts, keep):
        assert torch.equal(torch.nan_to_num(t, nan=1.0), torch.nan_to_num(k, nan=1.0))
    out = [torch.zeros_like(t) for t in ts]
    moe.moe_grad_clip(ts, norm, 1e-3, out=out)
    assert torch.equal(out[1], keep[1])


def test_a_small_norm_changes_no_bit(cuda_lib):
    moe = cuda_lib
    ts = grads([(5000, torch.float32), (301, torch.float16)], 6)
    keep = [t.clone() for t in ts]
    norm = moe.moe_grad_norm(ts)
    moe.moe_grad_clip(ts, norm, float(norm))          # equal: not larger
    assert all(torch.equal(t, k) for t, k in zip(ts, keep))
    moe.moe_grad_clip(ts, norm, 0.0)
    assert not any(t.any() for t in ts)


def test_the_same_bits_on_every_run_and_in_a_graph(cuda_lib):
    moe = cuda_lib
    ts = grads([(3_000_001, torch.float32), (500_003, torch.bfloat16), (17, torch.float16)], 7)
    out = [torch.empty_like(t) for t in ts]
    ws = torch.empty(moe.load_library().moe_grad_norm_workspace_size(3), dtype=torch.uint8, device=DEV)
    first = moe.moe_clip_grad_norm(ts, 1.0, out=out, workspace=ws).clone()
    want = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    n1 = torch.empty((), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_grad_norm(ts, out=n1, workspace=ws)
        moe.moe_grad_clip(ts, n1, 1.0, out=out)
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        assert torch.equal(n1, first) and all(torch.equal(o, w) for o, w in zip(out, want))
        ws.fill_(0xFF)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_clip_grad_norm(ts, 1.0, out=out, stream=s)
    s.synchronize()
    assert torch.equal(got, first) and all(torch.equal(o, w) for o, w in zip(out, want))


def test_a_training_step_clips_the_experts_gradients(cuda_lib):
    """moe_experts_backward's three FP32 gradients (an expert without rows among them) and a router gradient."""
    moe = cuda_lib
    E, H, I, rows = 4, 64, 96, 50
    g = torch.Generator().manual_seed(8)
    w = [(torch.randn(E, n, K, generator=g) * K ** -0.5).to(torch.bfloat16).to(DEV)
         for n, K in ((I, H), (I, H), (H, I))]
    ex = moe.Experts(*w)
    x = torch.randn(rows, H, generator=g).to(torch.bfloat16).to(DEV)
    offs = torch.tensor([0, 20, 20, 37, 50], dtype=torch.int32, device=DEV)
    y, cache = moe.moe_experts_forward_training(ex, x, offs)
    gr = moe.moe_experts_backward(ex, cache, torch.randn(rows, H, generator=g).to(torch.bfloat16).to(DEV))
    ts = [gr.dgate, gr.dup, gr.ddown, torch.randn(E, H, generator=g).to(torch.bfloat16).to(DEV)]
    keep = [t.clone() for t in ts]
    norm = moe.moe_clip_grad_norm(ts, 1.0)
    check_norm(norm, keep)
    check_clip(ts, keep, exact(keep), 1.0)
    assert abs(exact(ts) - 1.0) < 1e-2 and not ts[0][1].any()


def test_refusals_on_the_device(cuda_lib):
    moe = cuda_lib
    t = torch.zeros(64, device=DEV)
    norm = torch.ones((), device=DEV)
    for bad in (
        lambda: moe.moe_grad_clip([t, t], norm, 1.0),
        lambda: moe.moe_grad_clip([t], norm, -1.0),
        lambda: moe.moe_grad_clip([t], norm.double(), 1.0),
        lambda: moe.moe_grad_clip([t], norm, 1.0, out=[t.half()]),
        lambda: moe.moe_grad_clip([t], norm, 1.0, out=[]),
        lambda: moe.moe_grad_clip([t[:32]], norm, 1.0, out=[t[16:48]]),
        lambda: moe.moe_grad_norm([t.double()]),
        lambda: moe.moe_grad_norm([t], workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
    ):
        with pytest.raises(moe.MoeError):
            bad()
    with pytest.raises(ValueError):
        moe.moe_grad_norm([torch.zeros(8, 8, device=DEV).t()])
    assert float(moe.moe_grad_norm([t, t])) == 0.0
