"""MXFP4 experts and gradient clipping without a GPU: the oracle against
hand-worked values, and the C ABI's and the binding's refusals (every check
runs on the host before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build
from oracle import mxfp4

P = ctypes.c_void_p
A = P(0x100000)   # aligned, never dereferenced: every case below fails a host check first
BAD16 = P(0x100008)
BAD4 = P(0x100002)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


# ------------------------------------------------------------------ the oracle

def test_oracle_rounds_by_the_nearest_value_and_even_ties():
    """Every grid value, every midpoint and the points beside it, against a search over all values."""
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    ys = sorted({g for g in grid} | {(a + b) / 2 + d for a, b in zip(grid, grid[1:]) for d in (-2 ** -20, 0, 2 ** -20)}
                | {7.0, 7.99})
    for y in ys:
        x = np.zeros((1, 32))
        x[0, 0], x[0, 1], x[0, 2] = 4.0, y, -float(y)          # a in [4, 8): the scale is 1
        codes, scales = mxfp4.quantize(x)
        assert scales[0, 0] == 127
        d = [abs(y - g) for g in grid]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert codes[0, 0] >> 4 == want and codes[0, 1] & 15 == want + 8, y


def test_oracle_scales():
    for a, byte in ((0.0, 0), (6.0, 127), (4.0, 127), (3.999, 126), (8.0, 128), (1.0, 125), (2.0 ** -127, 0),
                    (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (3.4e38, 252), (np.inf, 255), (np.nan, 255)):
        x = np.zeros((1, 64))
        x[0, 40] = -a
        codes, scales = mxfp4.quantize(x)
        assert scales[0].tolist() == [0, byte, 0, 0], a
        assert not codes[0, :16].any()


def test_oracle_values_invert_the_codes():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (4, 48), dtype=np.uint8)
    scales = rng.integers(3, 250, (4, 4), dtype=np.uint8)
    scales[:, 3] = 0
    v = mxfp4.values(codes, scales)
    for blk in range(3):
        v[:, 32 * blk] = 6.0 * 2.0 ** (scales[:, blk].astype(float) - 127)   # pins the scale
    q, s = mxfp4.quantize(v)
    assert np.array_equal(s, scales)
    assert np.array_equal(mxfp4.values(q, s), v)


def test_oracle_clip():
    g = [np.array([3.0, 0.0]), np.array([-4.0])]
    assert mxfp4.grad_norm(g) == 5.0
    assert [x.tolist() for x in mxfp4.grad_clip(g, 5.0, 2.5)] == [[1.5, 0.0], [-2.0]]
    assert [x.tolist() for x in mxfp4.grad_clip(g, 5.0, 5.0)] == [[3.0, 0.0], [-4.0]]
    assert [x.tolist() for x in mxfp4.grad_clip(g, np.inf, 2.5)] == [[3.0, 0.0], [-4.0]]


# ------------------------------------------------------------------ refusals, C ABI

def test_scale_pitch(lib):
    assert [lib.moe_mxfp4_scale_pitch(k) for k in (32, 96, 128, 160, 4096)] == [4, 4, 4, 8, 128]
    assert [lib.moe_mxfp4_scale_pitch(k) for k in (0, -32, 16, 33)] == [0, 0, 0, 0]


def _quantize(lib, x=A, dtype=2, rows=4, K=64, inv=None, top_k=1, codes=A, scales=A):
    return lib.moe_mxfp4_quantize(x, dtype, rows, K, inv, top_k, codes, scales, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(K=0), 2), (dict(K=48), 2), (dict(K=262144 + 32), 2),
    (dict(K=-32), 2),
    (dict(top_k=2), 4), (dict(top_k=0), 4), (dict(inv=A, top_k=0), 4), (dict(rows=-1), 2),
    (dict(rows=1 << 31, inv=A, top_k=2), 2), (dict(rows=(1 << 32) - 1), 2),
    (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(x=BAD16), 5), (dict(codes=BAD16), 5), (dict(scales=BAD4), 5), (dict(inv=BAD4, top_k=1), 5),
])
def test_quantize_rejects_bad_arguments(lib, kwargs, status):
    assert _quantize(lib, **kwargs) == status
    assert lib.moe_last_error().decode() != ""


def test_quantize_without_rows_is_a_no_op(lib):
    assert _quantize(lib, x=None, codes=None, scales=None, rows=0) == 0


def _dequantize(lib, codes=A, scales=A, rows=4, K=64, out=A, dtype=2):
    return lib.moe_mxfp4_dequantize(codes, scales, rows, K, out, dtype, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=9), 3), (dict(K=31), 2), (dict(rows=-2), 2), (dict(rows=(1 << 32) - 1), 2), (dict(codes=None), 1),
    (dict(scales=None), 1), (dict(out=None), 1), (dict(out=BAD16), 5), (dict(codes=BAD16), 5), (dict(scales=BAD4), 5),
])
def test_dequantize_rejects_bad_arguments(lib, kwargs, status):
    assert _dequantize(lib, **kwargs) == status


def _create(lib, E=4, H=64, I=96, ptrs=None, storage=A, nbytes=None, out=True):
    h = P()
    p = dict(gc=A, gs=A, uc=A, us=A, dc=A, ds=A)
    p.update(ptrs or {})
    n = lib.moe_experts_mxfp4_storage_size(E, H, I) if nbytes is None else nbytes
    return lib.moe_experts_mxfp4_create(p["gc"], p["gs"], p["uc"], p["us"], p["dc"], p["ds"], E, H, I, storage, n, None,
                                        ctypes.byref(h) if out else None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(out=False), 1), (dict(E=0), 2), (dict(E=1025), 2), (dict(H=40), 2), (dict(I=0), 2), (dict(I=262176), 2),
    (dict(ptrs=dict(gc=None)), 1), (dict(ptrs=dict(us=None)), 1), (dict(ptrs=dict(ds=None)), 1),
    (dict(ptrs=dict(dc=BAD16)), 5), (dict(ptrs=dict(gs=BAD4)), 5),
    (dict(storage=None), 6), (dict(nbytes=100), 6), (dict(storage=P(0x100010)), 5),
])
def test_create_rejects_bad_arguments(lib, kwargs, status):
    assert _create(lib, **kwargs) == status


def test_storage_size(lib):
    # gate and up: 1 row block of 128, 1 word of 128 K elements; down: 2 row blocks; 512 bytes each, 4 experts
    assert lib.moe_experts_mxfp4_storage_size(4, 64, 96) == 4 * (1 + 1 + 2) * 512
    # 768 channels are 6 row blocks of 16 words; 2048 down rows 16 row blocks of 6
    assert lib.moe_experts_mxfp4_storage_size(128, 2048, 768) == 128 * (2 * 6 * 16 + 16 * 6) * 512
    assert lib.moe_experts_mxfp4_storage_size(0, 64, 96) == 0
    assert lib.moe_experts_mxfp4_storage_size(4, 65, 96) == 0


def test_stage_calls_reject_a_null_handle(lib):
    assert lib.moe_experts_mxfp4_gate_up(None, A, A, A, 4, 2, A, None, None, None) == 1
    assert lib.moe_experts_mxfp4_down(None, A, A, A, 4, 2, A, None) == 1
    assert lib.moe_experts_mxfp4_forward_dispatched(None, A, A, A, 4, 2, A, A, 1 << 20, None) == 1
    assert lib.moe_forward_mxfp4(None, A, 2, A, 2, 4, 2, 1, A, None, None, A, 1 << 20, None) == 1
    assert lib.moe_experts_mxfp4_forward_dispatched_workspace_size(None, 4) == 0
    assert lib.moe_forward_mxfp4_workspace_size(None, 4, 2, 2) == 0
    lib.moe_experts_mxfp4_destroy(None)


def _grads(*entries):
    t = (moe.GradTensor * max(1, len(entries)))()
    for e, (src, dst, n, dt) in zip(t, entries):
        e.src, e.dst, e.numel, e.dtype = src, dst, n, dt
    return t


OK = (0x10000, 0x10000, 100, 0)


@pytest.mark.parametrize("entries,n,status", [
    ([OK], -1, 2), ([OK], (1 << 24) + 1, 2), ([(0x10000, 0, 100, 5)], 1, 3), ([(0x10000, 0, -1, 0)], 1, 2),
    ([(0, 0, 100, 0)], 1, 1), ([(0x10002, 0, 100, 0)], 1, 5), ([(0x10001, 0, 100, 2)], 1, 5),
])
def test_grad_norm_rejects_bad_tensors(lib, entries, n, status):
    assert lib.moe_grad_norm(_grads(*entries), n, A, A, 1 << 20, None) == status


def test_grad_norm_rejects_bad_buffers(lib):
    t = _grads(OK)
    need = lib.moe_grad_norm_workspace_size(1)
    assert need % 256 == 0 and lib.moe_grad_norm_workspace_size(-1) == 0
    assert lib.moe_grad_norm_workspace_size(1000) > need
    assert lib.moe_grad_norm(t, 1, None, A, need, None) == 1
    assert lib.moe_grad_norm(t, 1, BAD4, A, need, None) == 5
    assert lib.moe_grad_norm(t, 1, A, None, need, None) == 6
    assert lib.moe_grad_norm(t, 1, A, A, need - 1, None) == 6
    assert lib.moe_grad_norm(t, 1, A, P(0x100010), need, None) == 5
    assert lib.moe_grad_norm(None, 1, A, A, need, None) == 1


@pytest.mark.parametrize("entries,status", [
    ([(0x10000, 0, 100, 0)], 1),                                              # no dst
    ([OK, OK], 2),                                                            # the same tensor twice, in place
    ([(0x10000, 0x20000, 100, 0), (0x11000, 0x20100, 100, 0)], 2),            # dst ranges overlap
    ([(0x10000, 0x10004, 100, 0)], 2),                                        # dst shifted into its own src
    ([(0x10000, 0x20000, 100, 0), (0x20000, 0x30000, 100, 0)], 2),            # a dst is another one's src
    ([(0x10000, 0x10002, 1, 0)], 5),
])
def test_grad_clip_rejects_bad_tensors(lib, entries, status):
    assert lib.moe_grad_clip(_grads(*entries), len(entries), A, 1.0, None) == status


@pytest.mark.parametrize("max_norm,norm,status", [(-1.0, A, 2), (float("nan"), A, 2), (float("inf"), A, 2),
                                                  (1.0, None, 1), (1.0, BAD4, 5)])
def test_grad_clip_rejects_bad_norms(lib, max_norm, norm, status):
    assert lib.moe_grad_clip(_grads(OK), 1, norm, max_norm, None) == status


# ------------------------------------------------------------------ refusals, binding

def test_binding_refuses_host_tensors_and_bad_shapes(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize(x)
    with pytest.raises(moe.MoeError):
        moe.moe_mxfp4_scale_pitch(40)
    with pytest.raises(ValueError):
        moe.moe_grad_norm([x])
    q = moe.Mxfp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_mxfp4_dequantize(q)
    with pytest.raises(ValueError):
        moe.ExpertsMxfp4(q, q, q)
