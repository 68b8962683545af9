"""The orthogonalised updates without a GPU: the oracle against singular values, and every refusal of the C entry
points, which come before any CUDA call."""
import ctypes

import numpy as np
import pytest

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build
from oracle import block

P = ctypes.c_void_p
A = [P(0x10000000 * i) for i in range(1, 8)]   # far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


@pytest.mark.parametrize("r,c", [(5, 9), (9, 5), (6, 6), (1, 4), (4, 1), (1, 1)])
@pytest.mark.parametrize("steps", [1, 5])
def test_oracle_maps_singular_values(r, c, steps):
    """X = U f(S) V^T with the quintic f(s) = a s + b s^3 + c s^5, `steps` times."""
    g = np.random.default_rng(r * c).normal(size=(r, c))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(steps):
        s = block.NS[0] * s + block.NS[1] * s ** 3 + block.NS[2] * s ** 5
    assert np.abs(block.newton_schulz(g, steps) - (u * s) @ vt).max() < 1e-12


def test_bounds_that_the_stored_scales_rest_on():
    """The quintic keeps [0, 1.21] in itself; with s there, s, s^2 and a + b s^2 + c s^4 times their powers of two
    stay under FP16's largest value."""
    a, b, c = block.NS
    s = np.linspace(0, 1.21, 200001)
    assert (np.abs(a * s + b * s ** 3 + c * s ** 5) < 1.2035).all()
    for v, e in ((s, 14), (s * s, 14), (a + b * s ** 2 + c * s ** 4, 13)):
        assert np.abs(v).max() * 2.0 ** e * (1 + 1e-3) < 65504


def test_oracle_of_zeros_and_of_nan():
    assert (block.newton_schulz(np.zeros((3, 4))) == 0).all()
    g = np.ones((3, 4))
    g[1, 2] = NAN
    assert np.isnan(block.newton_schulz(g)).all()


WS = 1 << 26


def _orth(lib, g=A[0], dt=0, E=2, r=64, c=96, steps=5, eps=1e-7, out=A[1], odt=2, ws=A[2], n=WS):
    return lib.moe_orthogonalize(g, dt, E, r, c, steps, eps, out, odt, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(out=None), 1), (dict(dt=7), 3), (dict(odt=0), 3), (dict(odt=5), 3), (dict(E=-1), 2),
    (dict(E=65536), 2), (dict(r=-1), 2), (dict(r=65537), 2), (dict(c=65537), 2), (dict(E=60000, r=65536, c=8), 2),
    (dict(steps=0), 2), (dict(steps=101), 2), (dict(eps=0.0), 2), (dict(eps=NAN), 2), (dict(eps=INF), 2),
    (dict(eps=-1e-7), 2), (dict(ws=None), 6), (dict(n=1000), 6), (dict(ws=P(0x30000080)), 5),
    (dict(g=P(0x10000002)), 5), (dict(out=P(0x20000001)), 5), (dict(out=A[2]), 2), (dict(ws=A[0]), 2),
])
def test_orthogonalize_refusals(lib, kw, status):
    assert _orth(lib, **kw) == status
    assert lib.moe_last_error().decode() != ""


@pytest.mark.parametrize("kw", [dict(E=0), dict(r=0), dict(c=0)])
def test_nothing_to_do(lib, kw):
    assert _orth(lib, g=None, out=None, ws=None, n=0, **kw) == 0
    assert lib.moe_orthogonalize_workspace_size(kw.get("E", 1), kw.get("r", 1), kw.get("c", 1)) == 0


def test_workspace_size(lib):
    size = lib.moe_orthogonalize_workspace_size
    assert size(-1, 4, 4) == size(65536, 4, 4) == size(1, 65537, 4) == 0
    n = 4 * 512 * 1000
    assert n * 8 < size(4, 512, 1000) < n * 8 + 4 * 512 * 512 * 16 + 35_000_000
    n = 300 * 512 * 1000
    assert n * 8 < size(300, 512, 1000) < n * 8 + 300 * 512 * 512 * 16 + (1 << 20)
    assert size(4, 512, 1000) % 256 == 0


def _muon(lib, w=A[0], wdt=0, g=A[1], gdt=0, m=A[2], E=2, r=64, c=96, ws=A[3], n=WS, params=True, **kw):
    p = dict(lr=0.1, momentum_decay=0.9, weight_decay=0.1, update_scale=1.0, eps=1e-7, steps=5, nesterov=1)
    p.update(kw)
    return lib.moe_muon_step(w, wdt, g, gdt, m, E, r, c, moe.MuonParams(*p.values()) if params else None, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), 1), (dict(g=None), 1), (dict(m=None), 1), (dict(params=False), 1), (dict(wdt=3), 3),
    (dict(gdt=-1), 3), (dict(E=-1), 2), (dict(r=70000), 2), (dict(lr=NAN), 2), (dict(weight_decay=INF), 2),
    (dict(update_scale=NAN), 2), (dict(momentum_decay=1.0), 2), (dict(momentum_decay=-0.1), 2),
    (dict(momentum_decay=NAN), 2), (dict(steps=0), 2), (dict(eps=0.0), 2), (dict(ws=None), 6), (dict(n=0), 6),
    (dict(ws=P(0x40000008)), 5), (dict(w=P(0x10000002)), 5), (dict(m=P(0x30000001)), 5), (dict(g=A[0]), 2),
    (dict(m=A[1]), 2), (dict(m=A[0]), 2), (dict(ws=A[2]), 2),
])
def test_muon_refusals(lib, kw, status):
    assert _muon(lib, **kw) == status
    assert lib.moe_last_error().decode() != ""
