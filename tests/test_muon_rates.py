"""Rates of a Muon step that are finite one by one and not as the factors that the weights get."""
import ctypes

import pytest

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build

A = [ctypes.c_void_p(0x10000000 * i) for i in range(1, 5)]   # far apart, never dereferenced


@pytest.mark.parametrize("kw", [dict(lr=1e30, update_scale=1e30), dict(lr=-1e20, update_scale=1e20, weight_decay=0.0),
                                dict(lr=1e30, weight_decay=-1e30), dict(lr=3e38, weight_decay=2.0)])
def test_factors_out_of_range_are_refused(kw):
    _build.build()
    lib = moe.load_library()
    p = dict(lr=0.1, momentum_decay=0.9, weight_decay=0.1, update_scale=1.0, eps=1e-7, steps=5, nesterov=1)
    p.update(kw)
    # (a workspace of 0 bytes: the call ends at its checks either way)
    assert lib.moe_muon_step(A[0], 0, A[1], 0, A[2], 2, 64, 96, moe.MuonParams(*p.values()), A[3], 0, None) == 2
    assert "FP32's range" in lib.moe_last_error().decode()
