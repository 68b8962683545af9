"""The norms around a block without a GPU: the oracle's gradients against central differences, and every refusal of
the C entry points, which come before any CUDA call."""
import ctypes

import numpy as np
import pytest

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build
from oracle import block

EPS = 1e-3
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


# ------------------------------------------------------------------ the oracle's gradients

@pytest.mark.parametrize("gate_shape", [None, (1, 5), (4, 1), (4, 5)])
@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
def test_oracle_gradients_against_differences(gate_shape, post, nxt):
    rng = np.random.default_rng(7)
    T, H = 4, 5
    p = dict(branch=rng.normal(size=(T, H)), residual=rng.normal(size=(T, H)))
    if post:
        p["norm_weight"] = 1 + 0.3 * rng.normal(size=H)
    if nxt:
        p["next_weight"] = 1 + 0.3 * rng.normal(size=H)
    if gate_shape:
        p["gate"] = rng.normal(size=gate_shape)
    dout, dy = rng.normal(size=(T, H)), rng.normal(size=(T, H))

    def loss(q):
        out = block.join(q["branch"], q["residual"], q.get("norm_weight"), q.get("gate", 1.0), 0.9, 0.6, EPS)
        total = (dout * out).sum()
        return total + (dy * block.norm(out, q["next_weight"], EPS)).sum() if nxt else total

    joined = block.join(p["branch"], p["residual"], p.get("norm_weight"), p.get("gate", 1.0), 0.9, 0.6, EPS)
    g = block.join_backward(dout, dy, p["branch"], joined, p.get("norm_weight"), p.get("gate", 1.0),
                            p.get("next_weight"), 0.9, 0.6, EPS)
    got = dict(branch=g.dbranch, residual=g.dresidual, norm_weight=g.dnorm_weight, next_weight=g.dnext_weight)
    if gate_shape:
        got["gate"] = g.dgate_full.sum(tuple(i for i in (0, 1) if gate_shape[i] == 1), keepdims=True)
    h = 1e-5
    for name, v in p.items():
        for i in np.ndindex(v.shape):
            lo, hi = (dict(p, **{name: v + s * h * (np.arange(v.size).reshape(v.shape) ==
                                                   np.ravel_multi_index(i, v.shape))}) for s in (-1, 1))
            # differences: h^2 times a third derivative of order 10, and 1e-16 / h of rounding
            assert abs((loss(hi) - loss(lo)) / (2 * h) - got[name][i]) < 1e-8


def test_oracle_sizes_bound_the_gradients():
    rng = np.random.default_rng(8)
    a = [rng.normal(size=(3, 6)) for _ in range(4)]
    args = (*a, rng.normal(size=6), rng.normal(size=(3, 1)), rng.normal(size=6), -0.5, 0.6, EPS)
    for g, s in zip(block.join_backward(*args), block.join_backward_size(*args)):
        assert (np.abs(g) <= s * (1 + 1e-12)).all()


# ------------------------------------------------------------------ refusals

A = [P(0x1000000 * i) for i in range(1, 20)]   # far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


def _norm(lib, x=A[0], dtype=2, w=A[1], wdt=2, eps=1e-6, T=4, H=64, y=A[2]):
    return lib.moe_block_norm(x, dtype, w, wdt, eps, T, H, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(dtype=5), 3), (dict(wdt=1), 3), (dict(wdt=9), 3),
    (dict(H=0), 2), (dict(H=32769), 2), (dict(T=-1), 2), (dict(T=1 << 31), 2), (dict(eps=0.0), 2), (dict(eps=-1.0), 2),
    (dict(eps=NAN), 2), (dict(eps=INF), 2),
    (dict(x=P(0x1000001)), 5), (dict(y=P(0x3000001)), 5), (dict(w=P(0x2000001)), 5), (dict(w=P(0x2000002), wdt=0), 5),
    (dict(y=P(0x1000002)), 2), (dict(y=A[1]), 2),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert lib.moe_last_error().decode() != ""


def test_no_rows_is_a_no_op(lib):
    assert _norm(lib, x=None, y=None, T=0) == 0
    p = moe.BlockJoinParams(A[1].value, A[3].value, None, 0, 2, 1.0, 1.0, 1e-6)
    assert lib.moe_block_join(None, None, 2, p, 0, 64, None, None, None) == 0
    assert lib.moe_combine_join(None, 2, None, None, 2, None, p, 0, 2, 64, None, None, None) == 0


def _norm_backward(lib, dy=A[0], x=A[1], dtype=2, w=A[2], wdt=0, dres=None, eps=1e-6, T=4, H=64, dx=A[3], dw=A[4],
                   ws=A[5], n=1 << 20):
    return lib.moe_block_norm_backward(dy, x, dtype, w, wdt, dres, eps, T, H, dx, dw, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(dx=None), 1), (dict(dw=None), 1),
    (dict(dtype=3), 3), (dict(wdt=1), 3), (dict(H=0), 2), (dict(T=-2), 2), (dict(eps=0.0), 2),
    (dict(ws=None), 6), (dict(n=255), 6), (dict(ws=P(0x6000010)), 5), (dict(dw=P(0x5000002)), 5),
    (dict(dres=P(0x7000001)), 5), (dict(dx=A[4]), 2), (dict(dw=A[1]), 2), (dict(dx=P(0x1000010)), 2),
    (dict(dx=A[5]), 2), (dict(ws=A[0]), 2),
])
def test_norm_backward_refusals(lib, kw, status):
    assert _norm_backward(lib, **kw) == status


def test_norm_backward_workspace_sizes(lib):
    assert lib.moe_block_norm_backward_workspace_size(4, 64) == 256     # one block, 64 floats
    assert lib.moe_block_norm_backward_workspace_size(0, 64) == 256
    for T, H in ((-1, 8), (1, 0), (1, 32769), (1 << 31, 8)):
        assert lib.moe_block_norm_backward_workspace_size(T, H) == 0
        assert lib.moe_block_join_backward_workspace_size(T, H) == 0


def _params(norm=A[1], nxt=A[2], gate=A[3], kind=1, vec=0, alpha=1.0, beta=1.0, eps=1e-6):
    v = lambda p: None if p is None else p.value
    return moe.BlockJoinParams(v(norm), v(nxt), v(gate), kind, vec, alpha, beta, eps)


BAD_PARAMS = [
    (dict(kind=4), 2), (dict(kind=-1), 2), (dict(gate=None), 1), (dict(alpha=NAN), 2), (dict(beta=INF), 2),
    (dict(eps=0.0), 2), (dict(vec=1), 3), (dict(norm=P(0x2000002)), 5), (dict(nxt=P(0x3000001)), 5),
    (dict(gate=P(0x4000002)), 5), (dict(gate=P(0x4000001), kind=3), 5),
]


def _join(lib, params=None, f=A[4], x=A[5], dtype=2, T=4, H=64, out=A[6], y=A[7]):
    return lib.moe_block_join(f, x, dtype, params, T, H, out, y, None)


@pytest.mark.parametrize("kw,status", BAD_PARAMS)
def test_join_refuses_bad_params(lib, kw, status):
    assert _join(lib, _params(**kw)) == status
    assert lib.moe_combine_join(A[4], 2, A[8], A[9], 2, A[5], _params(**kw), 4, 2, 64, A[6], A[7], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(f=None), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(y=None), 1), (dict(dtype=8), 3), (dict(H=0), 2),
    (dict(T=-1), 2), (dict(out=A[7]), 2), (dict(out=P(0x6000002)), 2), (dict(y=A[1]), 2), (dict(y=A[3]), 2),
    (dict(x=P(0x6000001)), 5),
])
def test_join_refusals(lib, kw, status):
    assert _join(lib, _params(), **kw) == status
    assert lib.moe_last_error().decode() != ""


def test_join_refuses_missing_params_and_an_unasked_norm(lib):
    assert _join(lib, None) == 1
    assert _join(lib, _params(nxt=None)) == 1      # normed without next_weight


@pytest.mark.parametrize("kw,status", [
    (dict(inv=None), 1), (dict(w=None), 1), (dict(wdt=4), 3), (dict(k=0), 4), (dict(T=1 << 30, k=4), 2),
    (dict(inv=P(0x9000002)), 5), (dict(w=P(0xA000001)), 5), (dict(out=A[4]), 2), (dict(out=A[8]), 2),
])
def test_combine_join_refusals(lib, kw, status):
    a = dict(inv=A[8], w=A[9], wdt=2, T=4, k=2, out=A[6])
    a.update(kw)
    assert lib.moe_combine_join(A[4], 2, a["inv"], a["w"], a["wdt"], A[5], _params(), a["T"], a["k"], 64, a["out"],
                                A[7], None) == status


def _join_backward(lib, params, dout=A[4], dn=A[5], f=A[6], joined=A[7], dtype=2, T=4, H=64, df=A[8], dx=A[9],
                   dw=A[10], dg=A[11], dw2=A[12], ws=A[13], n=1 << 20):
    return lib.moe_block_join_backward(dout, dn, f, joined, dtype, params, T, H, df, dx, dw, dg, dw2, ws, n, None)


@pytest.mark.parametrize("kw,status", BAD_PARAMS)
def test_join_backward_refuses_bad_params(lib, kw, status):
    assert _join_backward(lib, _params(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(f=None), 1), (dict(dn=None), 1), (dict(joined=None), 1), (dict(df=None), 1), (dict(dx=None), 1),
    (dict(dw=None), 1), (dict(dg=None), 1), (dict(dw2=None), 1), (dict(dtype=-1), 3), (dict(H=40000), 2),
    (dict(ws=None), 6), (dict(n=64 * 4 * 3 * 1 - 1), 6), (dict(ws=P(0xE000008)), 5), (dict(df=A[9]), 2),
    (dict(dg=A[10]), 2), (dict(dx=P(0x8000002)), 2), (dict(dw=A[2]), 2), (dict(dw2=P(0xD000002)), 5),
])
def test_join_backward_refusals(lib, kw, status):
    assert _join_backward(lib, _params(), **kw) == status


def test_join_backward_needs_a_gradient_without_the_next_norm(lib):
    p = _params(nxt=None)
    assert _join_backward(lib, p, dout=None, dw2=None) == 1
    assert _join_backward(lib, p) == 1             # dnext_weight without next_weight
    assert _join_backward(lib, _params(kind=0, gate=None)) == 1   # dgate without a gate
