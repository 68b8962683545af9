"""The operators around the expert layer in its block, and the optimizer step
behind its backward, as measured cases.

Each case is one pass through an operator: the plain form in elementary torch
operations (``own`` false), or the library's call (``own`` true).

  norm        y = norm(x) * w before the block, or its backward (with the
              residual stream's gradient added to dx)
  join        after the block: out = alpha x + beta gate * (norm(f) * w), and
              the next block's norm(out) * w2, or the backward of both
  combine     the same with f = the routing-weighted sum of the experts' rows
  ortho       five Newton-Schulz steps on every matrix of a batch
  muon        momentum, the Newton-Schulz steps, and the weights' update
"""
from __future__ import annotations

import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
NS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Decode: 16 tokens into the block. A few microseconds: latency counts.
        dict(name="norm_decode_bf16", op="norm", back=False, dtype="bf16", vec="bf16", T=16, H=2048),
        # Training step of the coarse layer: the norm's backward joins the residual stream's gradient.
        dict(name="norm_backward_bf16", op="norm", back=True, dtype="bf16", vec="f32", T=8192, H=4096),
        # Decode: the experts' rows of 16 tokens x 8 back into the residual stream, gated per token, normed for the
        # next block.
        dict(name="combine_decode_bf16", op="combine", dtype="bf16", vec="bf16", T=16, H=2048, top_k=8, gate="token",
             post=True, next=True),
        # Fine-grained prefill.
        dict(name="combine_prefill_bf16", op="combine", dtype="bf16", vec="bf16", T=4096, H=2048, top_k=8,
             gate="none", post=True, next=True),
        # A long F16 prompt through a block with a learned scale per channel.
        dict(name="join_prompt_f16", op="join", back=False, dtype="f16", vec="f32", T=16384, H=2048, gate="channel",
             post=True, next=True),
        # Its backward at the coarse layer's size, every gradient.
        dict(name="join_backward_bf16", op="join", back=True, dtype="bf16", vec="f32", T=8192, H=4096,
             gate="channel", post=True, next=True),
        # Odd sizes, FP32, a gate of its own for every element (made by a condition).
        dict(name="join_backward_odd_f32", op="join", back=True, dtype="f32", vec="f32", T=333, H=1409,
             gate="element", post=True, next=True),
        # One router's gradient, 128 experts x 2048: a single small matrix, latency counts.
        dict(name="ortho_router_f32", op="ortho", dtype="f32", out="bf16", E=1, rows=128, cols=2048),
        # The gate gradients of the fine-grained layer.
        dict(name="ortho_experts_f32", op="ortho", dtype="f32", out="bf16", E=128, rows=768, cols=2048),
        # The gate gradients of the coarse layer: the largest products.
        dict(name="ortho_coarse_f32", op="ortho", dtype="f32", out="bf16", E=8, rows=14336, cols=4096),
        # BF16 weights and gradients, sizes that end inside every tile.
        dict(name="muon_ragged_bf16", op="muon", dtype="bf16", wdtype="bf16", E=7, rows=1184, cols=733, nesterov=True),
        # The down weights of the skewed layer, FP32 masters.
        dict(name="muon_down_f32", op="muon", dtype="f32", wdtype="f32", E=64, rows=2048, cols=1408, nesterov=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "join", "join", "combine", "ortho", "ortho", "muon"])
    if op in ("norm", "join", "combine"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), H=H)
        case["vec"] = rng.choice([case["dtype"], "f32"])
        most = min(16384, 33_554_432 // H)
        if op == "combine":
            case["top_k"] = rng.randint(1, 8)
            most = max(1, most // case["top_k"])
        else:
            case["back"] = rng.random() < 0.5
        case["T"] = _log_int(rng, 1, most)
        if op != "norm":
            case["gate"] = rng.choice(["none", "channel", "token", "element"])
            case["post"], case["next"] = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return case
    lo, hi = sorted((_log_int(rng, 16, 4096), _log_int(rng, 16, 8192)))
    if rng.random() < 0.6:
        lo, hi = (max(16, v // 16 * 16) for v in (lo, hi))
    # at most a tenth of the largest listed products and 300M elements
    E = min(128, int(1.5e12 // (5 * (3 * lo * lo * hi + lo ** 3))) + 1, 300_000_000 // (lo * hi) + 1)
    E = _log_int(rng, 1, E)
    rows, cols = (lo, hi) if rng.random() < 0.5 else (hi, lo)
    case = dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), E=E, rows=rows, cols=cols)
    if op == "ortho":
        case["out"] = rng.choice(["bf16", "bf16", "f16"])
    else:
        case["wdtype"] = rng.choice(["f32", "bf16"])
        case["nesterov"] = rng.random() < 0.7
    return case


def work(case):
    """Each input read once, each output written once; the symmetric products of a Newton-Schulz step counted half."""
    es = DTYPES[case["dtype"]].itemsize
    op = case["op"]
    if op in ("ortho", "muon"):
        n = case["E"] * case["rows"] * case["cols"]
        s, l = sorted((case["rows"], case["cols"]))
        flops = 5 * case["E"] * (3 * s * s * l + s ** 3)
        if op == "ortho":
            return {"bytes": n * (es + 2), "flops": flops}
        return {"bytes": n * (es + 8 + 2 * DTYPES[case["wdtype"]].itemsize), "flops": flops}
    T, H, n = case["T"], case["H"], case["T"] * case["H"]
    vs = DTYPES[case["vec"]].itemsize
    if op == "norm":
        if not case["back"]:
            return {"bytes": 2 * n * es + H * vs, "flops": 4 * n}
        return {"bytes": 4 * n * es + H * (vs + 4), "flops": 10 * n}
    gate = case["gate"]
    vecs = (int(case["post"]) + int(case["next"]) + int(gate == "channel")) * H + (T if gate == "token" else 0)
    element = n * es if gate == "element" else 0
    if op == "join" and case["back"]:
        # dout, f, and the gradients of x and f; out and dy where the next norm is there
        big = (4 + (2 if case["next"] else 0)) * n * es + 2 * element
        return {"bytes": big + vecs * (vs + 4), "flops": 30 * n}
    rows = case.get("top_k", 1)
    big = (rows + 2 + int(case["next"])) * n * es + element
    maps = T * rows * (4 + es) if op == "combine" else 0
    return {"bytes": big + maps + vecs * vs, "flops": (8 + 2 * rows) * n}


# ------------------------------------------------------------------ prepare

def _hidden(T, H, dtype, gen):
    """Hidden states: normal values with a few loud channels and a scale of its own for every token."""
    x = torch.randn(T, H, generator=gen, device=DEV)
    x[:, torch.randint(0, H, (max(1, H // 256),), generator=gen, device=DEV)] *= 20.0
    return (x * torch.exp(0.5 * torch.randn(T, 1, generator=gen, device=DEV))).to(dtype)


def _vector(n, dtype, gen):
    return (1.0 + 0.2 * torch.randn(n, generator=gen, device=DEV)).to(dtype)


def _gradients(case, gen):
    """Gradients of weight matrices: a few strong directions over noise."""
    E, r, c = case["E"], case["rows"], case["cols"]
    k = min(16, r, c)
    g = torch.randn(E, r, c, generator=gen, device=DEV)
    u = torch.randn(E, r, k, generator=gen, device=DEV) * torch.exp(-0.2 * torch.arange(k, device=DEV)) * 2.0
    return (torch.baddbmm(g, u, torch.randn(E, k, c, generator=gen, device=DEV)) * 1e-3).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("ortho", "muon"):
        st["grad"] = _gradients(case, gen)
        if op == "muon":
            E, r, c = case["E"], case["rows"], case["cols"]
            st["weight"] = (torch.randn(E, r, c, generator=gen, device=DEV) * c ** -0.5).to(DTYPES[case["wdtype"]])
            st["momentum"] = torch.randn(E, r, c, generator=gen, device=DEV) * 3e-3
        return st
    T, H = case["T"], case["H"]
    dt, vt = DTYPES[case["dtype"]], DTYPES[case["vec"]]
    if op == "norm":
        st["x"], st["w"] = _hidden(T, H, dt, gen), _vector(H, vt, gen)
        if case["back"]:
            st["dy"] = torch.randn(T, H, generator=gen, device=DEV).to(dt)
            st["dres"] = torch.randn(T, H, generator=gen, device=DEV).to(dt)
        return st
    st["w"] = _vector(H, vt, gen) if case["post"] else None
    st["w2"] = _vector(H, vt, gen) if case["next"] else None
    gate = case["gate"]
    st["gate"] = (None if gate == "none" else 0.3 * _vector(H, torch.float32, gen) if gate == "channel" else
                  torch.rand(T, 1, generator=gen, device=DEV) if gate == "token" else
                  0.5 * torch.randn(T, H, generator=gen, device=DEV))
    if gate != "none":
        st["gate"] = st["gate"].to(dt if gate == "element" else vt)
    st["alpha"], st["beta"] = 1.0, 0.7
    if op == "combine":
        n = T * case["top_k"]
        row_src = torch.randperm(n, generator=gen, device=DEV)
        inv = torch.empty_like(row_src)
        inv[row_src] = torch.arange(n, device=DEV)
        st["inv"] = inv.to(torch.int32)
        st["y"] = torch.randn(n, H, generator=gen, device=DEV).to(dt)
        st["weights"] = torch.softmax(torch.randn(T, case["top_k"], generator=gen, device=DEV), -1).to(dt)
        st["x"] = _hidden(T, H, dt, gen)
        return st
    st["f"] = torch.randn(T, H, generator=gen, device=DEV).to(dt)
    if not case["back"]:
        st["x"] = _hidden(T, H, dt, gen)
        return st
    st["out"] = _hidden(T, H, dt, gen) if case["next"] else None
    st["dout"] = torch.randn(T, H, generator=gen, device=DEV).to(dt)
    st["dy"] = torch.randn(T, H, generator=gen, device=DEV).to(dt) if case["next"] else None
    return st


# ------------------------------------------------------------------ the plain forms

def _f(t):
    return t.to(torch.float32)


def _rstd(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm_grad(v, w, dy):
    """(gradient of v, summed gradient of w) of v * rstd(v) * w, in FP32."""
    r = _rstd(v)
    wd = w * dy
    return r * (wd - v * (r * r) * (wd * v).mean(-1, keepdim=True)), (dy * v * r).sum(0)


def _join_plain(st, f, x):
    dt = x.dtype
    b = f * _rstd(f) * _f(st["w"]) if st["w"] is not None else f
    if st["gate"] is not None:
        b = b * _f(st["gate"])
    out = (st["alpha"] * _f(x) + st["beta"] * b).to(dt)
    if st["w2"] is None:
        return [out]
    o = _f(out)
    return [out, (o * _rstd(o) * _f(st["w2"])).to(dt)]


def _join_backward_plain(st):
    case = st["case"]
    dt = st["f"].dtype
    d = _f(st["dout"])
    dw = dw2 = dgate = None
    if st["w2"] is not None:
        dn, dw2 = _norm_grad(_f(st["out"]), _f(st["w2"]), _f(st["dy"]))
        d = d + dn
    dx = (st["alpha"] * d).to(dt)
    f = _f(st["f"])
    b = f * _rstd(f) * _f(st["w"]) if st["w"] is not None else f
    db = st["beta"] * d
    if st["gate"] is not None:
        t = db * b
        dgate = t.sum(0) if case["gate"] == "channel" else t.sum(-1, keepdim=True) if case["gate"] == "token" else t.to(dt)
        db = db * _f(st["gate"])
    if st["w"] is not None:
        db, dw = _norm_grad(f, _f(st["w"]), db)
    return {k: v for k, v in dict(dbranch=db.to(dt), dresidual=dx, dnorm_weight=dw, dgate=dgate,
                                  dnext_weight=dw2).items() if v is not None}


def _newton_schulz_plain(u):
    """Five steps on each matrix of u [E, r, c] in FP32."""
    a, b, c = NS
    x = u / ((u * u).sum((-2, -1), keepdim=True, dtype=torch.float64).sqrt() + NS_EPS).to(torch.float32)
    tall = x.shape[-2] > x.shape[-1]
    for _ in range(5):
        xt = x.transpose(-2, -1)
        g = xt @ x if tall else x @ xt
        p = b * g + c * (g @ g)
        x = a * x + (x @ p if tall else p @ x)
    return x


LR, MU, WD = 2e-3, 0.95, 0.1


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import moe_routing_swiglu_gb300 as moe

        if op == "norm":
            if case["back"]:
                return list(moe.moe_block_norm_backward(st["dy"], st["x"], st["w"], eps=EPS, dresidual=st["dres"]))
            return moe.moe_block_norm(st["x"], st["w"], eps=EPS)
        if op == "ortho":
            return moe.moe_orthogonalize(st["grad"], dtype=DTYPES[case["out"]], eps=NS_EPS)
        if op == "muon":
            moe.moe_muon_step(st["weight"], st["grad"], st["momentum"], lr=LR, momentum_decay=MU,
                              nesterov=case["nesterov"], weight_decay=WD, eps=NS_EPS)
            return [st["weight"], st["momentum"]]
        parts = dict(norm_weight=st["w"], gate=st["gate"], next_weight=st["w2"], residual_scale=st["alpha"],
                     branch_scale=st["beta"], eps=EPS)
        if op == "combine":
            got = moe.moe_combine_join(st["y"], st["inv"], st["weights"], st["x"], **parts)
        elif case["back"]:
            g = moe.moe_block_join_backward(st["dout"], st["f"], dnormed=st["dy"], joined=st["out"], **parts)
            return {k: v for k, v in g._asdict().items() if v is not None}
        else:
            got = moe.moe_block_join(st["f"], st["x"], **parts)
        return [t for t in got if t is not None]
    if op == "norm":
        x, w = _f(st["x"]), _f(st["w"])
        if case["back"]:
            dx, dw = _norm_grad(x, w, _f(st["dy"]))
            return [(dx + _f(st["dres"])).to(st["x"].dtype), dw]
        return (x * _rstd(x) * w).to(st["x"].dtype)
    if op == "ortho":
        return _newton_schulz_plain(_f(st["grad"])).to(DTYPES[case["out"]])
    if op == "muon":
        g, m = _f(st["grad"]), st["momentum"]
        m.mul_(MU).add_(g)
        o = _newton_schulz_plain(g + MU * m if case["nesterov"] else m)
        scale = math.sqrt(max(1.0, case["rows"] / case["cols"]))
        st["weight"].copy_((1.0 - LR * WD) * _f(st["weight"]) - LR * scale * o)
        return [st["weight"], m]
    if op == "combine":
        rows = _f(st["y"][st["inv"].long()]).unflatten(0, (case["T"], case["top_k"]))
        f = (rows * _f(st["weights"]).unsqueeze(-1)).sum(1)
        return _join_plain(st, f, st["x"])
    if case["back"]:
        return _join_backward_plain(st)
    return _join_plain(st, _f(st["f"]), st["x"])


# ------------------------------------------------------------------ exact

def _exact_unit(v):
    return v / (torch.linalg.vector_norm(v, dim=-1, keepdim=True).square() / v.shape[-1] + EPS).sqrt()


def _exact_newton_schulz(g):
    """One matrix in FP64, always on the side of fewer rows: X <- (aI + A (bI + cA)) X."""
    a, b, c = NS
    x = g.T if g.shape[0] > g.shape[1] else g
    x = x / (torch.linalg.vector_norm(x) + NS_EPS)
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for _ in range(5):
        gram = torch.einsum("ik,jk->ij", x, x)
        x = torch.einsum("ij,jk->ik", a * eye + torch.einsum("ij,jk->ik", gram, b * eye + c * gram), x)
    return x.T if g.shape[0] > g.shape[1] else x


def exact(case, seed):
    op = case["op"]
    if op in ("ortho", "muon") and work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    D = lambda t: None if t is None else t.double()
    if op == "ortho":
        return torch.stack([_exact_newton_schulz(D(g)) for g in st["grad"]])
    if op == "muon":
        mom = MU * D(st["momentum"]) + D(st["grad"])
        u = D(st["grad"]) + MU * mom if case["nesterov"] else mom
        scale = max(1.0, case["rows"] / case["cols"]) ** 0.5
        w = torch.stack([D(w) * (1 - LR * WD) - LR * scale * _exact_newton_schulz(m)
                         for w, m in zip(st["weight"], u)])
        return [w, mom]
    leaf = lambda t: None if t is None else t.double().requires_grad_()
    if op == "norm":
        x, w = leaf(st["x"]), leaf(st["w"])
        y = _exact_unit(x) * w
        if not case["back"]:
            return y.detach()
        dx, dw = torch.autograd.grad(y, (x, w), D(st["dy"]))
        return [dx + D(st["dres"]), dw]

    def branch(f, w, gate):
        b = f if w is None else _exact_unit(f) * w
        return st["beta"] * (b if gate is None else b * gate)

    if op == "join" and case["back"]:
        d = D(st["dout"])
        got = {}
        if case["next"]:
            o, w2 = leaf(st["out"]), leaf(st["w2"])
            do, got["dnext_weight"] = torch.autograd.grad(_exact_unit(o) * w2, (o, w2), D(st["dy"]))
            d = d + do
        got["dresidual"] = st["alpha"] * d
        parts = dict(dbranch=leaf(st["f"]), dnorm_weight=leaf(st["w"]), dgate=leaf(st["gate"]))
        b = branch(*parts.values())
        names = [k for k, v in parts.items() if v is not None]
        got.update(zip(names, torch.autograd.grad(b, [parts[k] for k in names], d)))
        return got
    if op == "combine":
        rows = st["inv"].long().view(case["T"], case["top_k"])
        f = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        for j in range(case["top_k"]):
            f += D(st["weights"])[:, j:j + 1] * D(st["y"])[rows[:, j]]
    else:
        f = D(st["f"])
    out = st["alpha"] * D(st["x"]) + branch(f, D(st["w"]), D(st["gate"]))
    return [out] if st["w2"] is None else [out, _exact_unit(out) * D(st["w2"])]
