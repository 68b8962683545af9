"""The norms around a block in numpy FP64, and the Newton-Schulz steps of the
orthogonalised update: the formulas of include/moe.h, one step after another."""
from __future__ import annotations

from collections import namedtuple

import numpy as np

NS = (3.4445, -4.7750, 2.0315)


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def norm(v, w, eps):
    return v * rstd(v, eps) * w


def join(branch, residual, norm_weight, gate, alpha, beta, eps):
    """out before rounding; gate broadcasts against [T, H] (1.0 for none)."""
    b = branch if norm_weight is None else norm(branch, norm_weight, eps)
    return alpha * residual + beta * gate * b


def norm_backward(v, w, dy, eps):
    """(gradient of v, summed gradient of w)."""
    r = rstd(v, eps)
    n = v * r
    dn = dy * w
    return r * (dn - n * (dn * n).mean(-1, keepdims=True)), (dy * n).sum(0)


JoinGrads = namedtuple("JoinGrads", "dbranch dresidual dnorm_weight dgate_full dnext_weight")


def join_backward(dout, dnormed, branch, joined, norm_weight, gate, next_weight, alpha, beta, eps):
    """dgate_full is the gradient of every element's gate, to be summed over what a gate is shared by."""
    d, dw2 = dout, None
    if next_weight is not None:
        dj, dw2 = norm_backward(joined, next_weight, dnormed, eps)
        d = d + dj
    b = branch if norm_weight is None else norm(branch, norm_weight, eps)
    dgate = beta * d * b
    db, dw = beta * d * gate, None
    if norm_weight is not None:
        db, dw = norm_backward(branch, norm_weight, db, eps)
    return JoinGrads(db, alpha * d, dw, dgate, dw2)


def norm_backward_size(v, w, dy, eps):
    """The sizes of norm_backward's terms added up without their signs: what a relative rounding error multiplies.
    dy holds sizes too."""
    r = rstd(v, eps)
    n, dn = np.abs(v * r), dy * np.abs(w)
    return r * (dn + n * (dn * n).mean(-1, keepdims=True)), (dy * n).sum(0)


def join_backward_size(dout, dnormed, branch, joined, norm_weight, gate, next_weight, alpha, beta, eps):
    a = np.abs
    d, dw2 = a(dout), None
    if next_weight is not None:
        dj, dw2 = norm_backward_size(joined, next_weight, a(dnormed), eps)
        d = d + dj
    b = a(branch if norm_weight is None else norm(branch, norm_weight, eps))
    dgate = abs(beta) * d * b
    db, dw = abs(beta) * d * a(gate), None
    if norm_weight is not None:
        db, dw = norm_backward_size(branch, norm_weight, db, eps)
    return JoinGrads(db, abs(alpha) * d, dw, dgate, dw2)


def newton_schulz(g, steps=5, eps=1e-7):
    """The orthogonalised update of one matrix: X = G / (|G| + eps), then
    X <- a X + (b A + c A A) X with A = X X^T, `steps` times."""
    a, b, c = NS
    with np.errstate(invalid="ignore"):
        x = g / (np.sqrt((g * g).sum()) + eps)
        for _ in range(steps):
            if x.shape[0] <= x.shape[1]:
                m = x @ x.T
                x = a * x + (b * m + c * (m @ m)) @ x
            else:
                m = x.T @ x
                x = a * x + x @ (b * m + c * (m @ m))
    return x


def newton_schulz_moved(g, rng, steps=5, eps=1e-7):
    """newton_schulz with every product off by what FP16 pairs and a truncating FP32 accumulator may lose, at its full
    size and with signs drawn: an operand by 2^-22 of each entry; an entry of a product over K by 2^-23 of the sum of
    its terms' sizes for each of the 3 K / 16 additions. How far the result moves by it is what rounding may cost."""
    a, b, c = NS
    sign = lambda v: rng.choice((-1.0, 1.0), size=v.shape)

    def product(p, q):
        p, q = (v * (1 + 2.0 ** -22 * sign(v)) for v in (p, q))
        adds = -(-p.shape[1] // 16) * 3
        v = p @ q
        return v + adds * 2.0 ** -23 * (np.abs(p) @ np.abs(q)) * sign(v)

    x = g / (np.sqrt((g * g).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    for _ in range(steps):
        m = product(x.T, x) if tall else product(x, x.T)
        poly = a * np.eye(len(m)) + product(m, b * np.eye(len(m)) + c * m)
        x = product(x, poly) if tall else product(poly, x)
    return x


def newton_schulz_last_size(g, steps=5, eps=1e-7):
    """|B| |X| of the last product B X (X B): its terms' sizes added up."""
    a, b, c = NS
    x = newton_schulz(g, steps - 1, eps)
    tall = x.shape[0] > x.shape[1]
    m = x.T @ x if tall else x @ x.T
    poly = np.abs(a * np.eye(len(m)) + b * m + c * (m @ m))
    return np.abs(x) @ poly if tall else poly @ np.abs(x)
