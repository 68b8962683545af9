"""Refusals of the gradient clip that need no GPU: every check runs on the host before anything is enqueued."""
import ctypes

import pytest

import moe_routing_swiglu_gb300 as moe
from moe_routing_swiglu_gb300 import _build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


@pytest.mark.parametrize("norm", [0x20000, 0x20000 + 4 * 50, 0x20000 + 4 * 99])
@pytest.mark.parametrize("src", [0x10000, 0x20000])
def test_a_norm_inside_a_written_gradient_is_refused(lib, src, norm):
    """Blocks that start late would read the norm after it was scaled."""
    t = (moe.GradTensor * 2)()
    t[0].src, t[0].dst, t[0].numel, t[0].dtype = src, 0x20000, 100, 0
    t[1].src, t[1].dst, t[1].numel, t[1].dtype = 0x40000, 0x40000, 7, 2
    assert lib.moe_grad_clip(t, 2, P(norm), 1.0, None) == 2
    assert "norm" in lib.moe_last_error().decode()
