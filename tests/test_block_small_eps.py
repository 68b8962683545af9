"""The smallest eps of the norms' backward calls: refused below, right from there on, for rows of zeros and rows far
below sqrt(eps) too."""
import ctypes

import numpy as np
import pytest

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build
from oracle import block

A = [ctypes.c_void_p(0x1000000 * i) for i in range(1, 20)]   # far apart, never dereferenced
LEAST = 2.0 ** -80


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -128, 1e-30, LEAST * (1 - 2.0 ** -23)])
def test_smaller_ones_are_refused(eps):
    _build.build()
    lib = moe.load_library()
    assert lib.moe_block_norm_backward(A[0], A[1], 2, A[2], 0, None, eps, 4, 64, A[3], A[4], A[5], 1 << 20, None) == 2
    assert "2^-80" in lib.moe_last_error().decode()
    p = moe.BlockJoinParams(A[1].value, A[2].value, None, 0, 0, 1.0, 1.0, eps)
    assert lib.moe_block_join_backward(A[4], A[5], A[6], A[7], 2, p, 4, 64, A[8], A[9], A[10], None, A[12], A[13],
                                       1 << 20, None) == 2
    assert "2^-80" in lib.moe_last_error().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(6, 64), (6, 2048), (900, 2048), (900, 2047)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -60, 2.0 ** -45, 2.0 ** -40, 2.0 ** -30])
def test_rows_below_its_root(cuda_lib, T, H, scale):
    """FP32 rows; tolerance as in test_gpu_block_norm.py: 2^-18 of the terms' sizes, a column's sum (T + 16) 2^-24 more."""
    import torch

    rng = np.random.default_rng(T + H)
    x, f, dy, dout = (rng.normal(size=(T, H)) for _ in range(4))
    x, f = x * scale, f * scale
    w, w2 = (1 + 0.3 * rng.normal(size=H) for _ in range(2))
    x, f, dy, dout, w, w2 = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (x, f, dy, dout, w, w2))
    h = lambda t: t.double().cpu().numpy()

    def close(got, ref, size, cols=0.0):
        g = h(got)
        assert np.isfinite(g).all()
        assert (np.abs(g - ref) <= (2.0 ** -18 + cols) * size + 2.0 ** -24 * np.abs(ref) + 2.0 ** -149).all()

    cols = (T + 16) * 2.0 ** -24
    g = cuda_lib.moe_block_norm_backward(dy, x, w, eps=LEAST)
    (dx, dw), (sx, sw) = (fn(h(x), h(w), d, LEAST) for fn, d in
                          ((block.norm_backward, h(dy)), (block.norm_backward_size, np.abs(h(dy)))))
    close(g.dx, dx, sx)
    close(g.dweight, dw, sw, cols)
    got = cuda_lib.moe_block_join_backward(dout, f, dnormed=dy, joined=x, norm_weight=w, next_weight=w2, eps=LEAST)
    args = (h(dout), h(dy), h(f), h(x), h(w), np.ones((1, 1)), h(w2), 1.0, 1.0, LEAST)
    ref, size = block.join_backward(*args), block.join_backward_size(*args)
    close(got.dbranch, ref.dbranch, size.dbranch)
    close(got.dresidual, ref.dresidual, size.dresidual)
    close(got.dnorm_weight, ref.dnorm_weight, size.dnorm_weight, cols)
    close(got.dnext_weight, ref.dnext_weight, size.dnext_weight, cols)
