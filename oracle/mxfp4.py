"""Plain CPU statement of MXFP4 and of the experts on it, and of the gradient
norm and clip, in f64. TEST INFRASTRUCTURE, apart from the CUDA library.

MXFP4 (OCP Microscaling Formats v1.0, sections 5.3.3 and 6.3): blocks of 32
E2M1 elements with one E8M0 scale; the scale's exponent is the exponent of the
block's largest magnitude minus 2 (the exponent of E2M1's largest element), the
elements are rounded to nearest even and saturated.
"""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# The halfway points between neighbours and the code an exact tie goes to (the even one of the two).
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
TIE_CODE = np.array([0, 2, 2, 4, 4, 6, 6])


def scale_pitch(K: int) -> int:
    return (K // 32 + 3) // 4 * 4


def quantize(x: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """x [rows, K] (f64 copies of the dtype's values) -> codes [rows, K/2], scales [rows, pitch], uint8."""
    rows, K = x.shape
    v = x.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    a = np.abs(v).max(-1)
    _, ex = np.frexp(a)                                   # a = m 2^ex, 1/2 <= m < 1
    byte = np.where(a > 0, np.clip(ex - 1 - 2 + 127, 0, 254), 0)
    y = np.abs(v) * np.ldexp(1.0, 127 - byte)[..., None]  # exact: a power of two in f64
    code = np.searchsorted(BORDERS, y, side="left")       # borders strictly below y
    tie = np.searchsorted(BORDERS, y, side="right") != code
    code = np.where(tie, TIE_CODE[np.minimum(code, 6)], code) + 8 * np.signbit(v)
    codes = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(rows, K)
    scales = np.zeros((rows, scale_pitch(K)), dtype=np.uint8)
    scales[:, :K // 32] = np.where(bad, 255, byte)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The f64 values of codes [.., K/2] with scales [.., pitch]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c >= 8, -1.0, 1.0) * VALUES[c & 7]
    K = c.shape[-1]
    s = scales[..., :K // 32].astype(np.float64)
    s = np.where(s == 255, np.nan, 2.0 ** (np.minimum(s, 254) - 127))
    return v * np.repeat(s, 32, axis=-1)


def gate_up(x: np.ndarray, gate: np.ndarray, up: np.ndarray, offsets) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """f64 h, g, u [rows, I] of values x [rows, H], gate/up [E, I, H]."""
    g = np.zeros((x.shape[0], gate.shape[1]))
    u = np.zeros_like(g)
    for e in range(gate.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        g[lo:hi] = x[lo:hi] @ gate[e].T
        u[lo:hi] = x[lo:hi] @ up[e].T
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    return h, g, u


def down(h: np.ndarray, w: np.ndarray, offsets) -> np.ndarray:
    """f64 y [rows, H] of values h [rows, I], w [E, H, I]."""
    y = np.zeros((h.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi] = h[lo:hi] @ w[e].T
    return y


def grad_norm(grads) -> float:
    return float(np.sqrt(sum(float(np.sum(np.square(g))) for g in grads)))


def grad_clip(grads, norm: float, max_norm: float):
    f = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return [g * f for g in grads]
