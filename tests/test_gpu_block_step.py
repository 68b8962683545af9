"""The operators around the expert layer together, as a model uses them: a whole training step of a block (norm, router,
experts, join with the next norm, every gradient, clip, optimizer step) and a decoding step, eager and as a captured
graph.

Tolerance of the training step's gradients, 2-norm relative to each: FP32 throughout, sums of at most 257 terms, so every
stage adds at most 270 * 2^-24 of its result's size; 8 stages behind one another, and the norms and routing weights
magnify an error by their condition, below 16 here (sizes of terms over sizes of sums): 8 * 16 * 270 * 2^-24 < 2.1e-3."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu()


def _layer(T, E, H, I, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)
    p = dict(x=n(T, H), w0=1 + 0.2 * n(H), router=n(H, E, std=H ** -0.5 * 3), gate=n(E, I, H, std=H ** -0.5),
             up=n(E, I, H, std=H ** -0.5), down=n(E, H, I, std=I ** -0.5), w1=1 + 0.2 * n(H), scale=0.5 + 0.2 * n(H),
             w2=1 + 0.2 * n(H))
    return {k: v.to(dtype).to(DEV) for k, v in p.items()}, n(T, H).to(dtype).to(DEV), n(T, H).to(dtype).to(DEV)


def _forward64(p, idx, k):
    """out and y in FP64 for a fixed selection idx [T, k], differentiable."""
    unit = lambda v: v / ((v * v).mean(-1, keepdim=True) + EPS).sqrt()
    n = unit(p["x"]) * p["w0"]
    prob = torch.softmax(n @ p["router"], -1).gather(1, idx)
    prob = prob / prob.sum(-1, keepdim=True)
    f = 0
    for j in range(k):
        g = torch.einsum("th,tih->ti", n, p["gate"][idx[:, j]])
        u = torch.einsum("th,tih->ti", n, p["up"][idx[:, j]])
        f = f + prob[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, p["down"][idx[:, j]])
    out = p["x"] + 0.7 * p["scale"] * (unit(f) * p["w1"])
    return out, unit(out) * p["w2"]


def test_training_step_of_a_block(cuda_lib):
    moe = cuda_lib
    T, E, H, I, k = 37, 6, 64, 40, 2
    p, dout, dy = _layer(T, E, H, I, torch.float32, 3)
    join = dict(norm_weight=p["w1"], gate=p["scale"], next_weight=p["w2"], branch_scale=0.7, eps=EPS)
    ex = moe.Experts(p["gate"], p["up"], p["down"])

    n = moe.moe_block_norm(p["x"], p["w0"], eps=EPS)
    logits = n @ p["router"]
    idx, w, disp = moe.moe_route_dispatch(logits, k, True, n)
    yd, cache = moe.moe_experts_forward_training(ex, disp.x_dispatched, disp.offsets)
    f = moe.moe_combine(yd, disp.inv, w)
    out, y = moe.moe_block_join(f, p["x"], **join)

    j = moe.moe_block_join_backward(dout, f, dnormed=dy, joined=out, **join)
    dexp, dw = moe.moe_combine_backward(yd, disp.inv, disp.row_src, w, j.dbranch)
    eg = moe.moe_experts_backward(ex, cache, dexp)
    dlogits = moe.moe_router_backward(logits, idx, dw, moe.RouterWeightOptions("softmax", True))
    dn = moe.moe_dispatch_backward(eg.dx_dispatched, disp.inv, T, k) + dlogits @ p["router"].T
    g0 = moe.moe_block_norm_backward(dn, p["x"], p["w0"], eps=EPS, dresidual=j.dresidual)
    got = dict(x=g0.dx, w0=g0.dweight, router=n.T @ dlogits, gate=eg.dgate, up=eg.dup, down=eg.ddown, w1=j.dnorm_weight,
               scale=j.dgate, w2=j.dnext_weight)

    q = {name: f64(v).requires_grad_() for name, v in p.items()}
    ro, ry = _forward64(q, idx.cpu().long(), k)
    for a, b in ((out, ro), (y, ry)):
        assert float((f64(a) - b.detach()).norm() / b.detach().norm()) < 2.1e-3
    ((ro * f64(dout)).sum() + (ry * f64(dy)).sum()).backward()
    for name, v in q.items():
        assert float((f64(got[name]) - v.grad).norm() / v.grad.norm()) < 2.1e-3, name

    # clip over all gradients, then the optimizer on the experts' matrices
    grads = [got[name] for name in sorted(got)]
    norm = moe.moe_clip_grad_norm(grads, 0.5)
    ref = float(sum((v.grad ** 2).sum() for v in q.values()).sqrt())
    assert ref > 0.5 and abs(float(norm) - ref) < 2.1e-3 * ref
    rng = np.random.default_rng(4)
    for name in ("gate", "up", "down"):
        before, m = f64(p[name]).numpy(), torch.zeros_like(p[name])
        moe.moe_muon_step(p[name], got[name], m, lr=0.02, nesterov=False, weight_decay=0.1)
        rows, cols = p[name].shape[-2:]
        rate = float(np.float32(0.02)) * max(1.0, rows / cols) ** 0.5
        for e in range(E):
            g = f64(got[name])[e].numpy()
            o = block.newton_schulz(g)
            move = 2 * np.linalg.norm(block.newton_schulz_moved(g, rng) - o)
            want = (1 - 0.02 * 0.1) * before[e] - rate * o
            # keep, rate and the sum rounded once each, lr and weight_decay once more as FP32 values
            tol = 5 * 2.0 ** -24 * (np.abs(before[e]) + np.abs(rate * o)) + rate * move
            assert (np.abs(f64(p[name])[e].numpy() - want) <= tol).all(), name
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("T", [1, 16])
def test_decoding_step_eager_and_captured(cuda_lib, T):
    """norm, route + dispatch, experts, combine + join: the graph gives the eager call's bits, and the join in the
    combine's launch differs from the two calls by the combine's rounding to BF16 alone, half a step of the branch and,
    through its norm, as much again of the row, before out's own rounding of each."""
    moe = cuda_lib
    E, H, I, k = 16, 256, 96, 4
    p, _, _ = _layer(T, E, H, I, torch.bfloat16, 5)
    ex = moe.Experts(p["gate"], p["up"], p["down"])
    token = torch.rand(T, 1, device=DEV).to(torch.bfloat16)
    parts = dict(norm_weight=p["w1"], gate=token, next_weight=p["w2"], branch_scale=0.7, eps=EPS)
    router = p["router"].float()

    def step():
        n = moe.moe_block_norm(p["x"], p["w0"], eps=EPS)
        _, w, disp = moe.moe_route_dispatch(n.float() @ router, k, True, n)
        yd = moe.moe_experts_forward_dispatched(ex, disp.x_dispatched, disp.offsets)
        return moe.moe_combine_join(yd, disp.inv, w, p["x"], **parts), (yd, disp.inv, w)

    (out, y), rest = step()
    two = moe.moe_block_join(moe.moe_combine(*rest), p["x"], **parts)
    u = 2.0 ** -8
    branch = (f64(out) - f64(p["x"])).abs()
    tol = 3 * u * branch + 2 * u * f64(out).abs() + 2.0 ** -18 * f64(p["x"]).abs()
    assert ((f64(out) - f64(two[0])).abs() <= tol).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out2, y2), _ = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(y, y2)
