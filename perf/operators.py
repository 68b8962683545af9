"""The 4-bit expert path's and the gradient clip's operators as measured cases.

Each case is one pass through an operator: the plain form in elementary torch
operations (``own`` false), or the library's call (``own`` true).

  quantize    values -> MXFP4 (blocks of 32 E2M1 elements with an E8M0 scale)
              -> the values the 4 bits stand for; with top_k > 0 the rows are
              written in dispatched order (one copy per chosen expert)
  gate_up     h = SiLU(x Wg^T) * (x Wu^T) per expert, MXFP4 operands
  down        y = h Wd^T per expert, MXFP4 operands
  grad_norm   the L2 norm over many tensors
  grad_clip   the norm, then every tensor times min(1, max_norm / norm)
"""
from __future__ import annotations

import functools
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Decode: 16 tokens' activations, quantised into the 8 rows each that
        # their experts read. A few microseconds: latency counts.
        dict(name="quantize_decode_bf16", op="quantize", dtype="bf16", rows=16, K=2048, top_k=8),
        # Ragged prefill, F16 activations, straight (no dispatch).
        dict(name="quantize_ragged_f16", op="quantize", dtype="f16", rows=1777, K=1408, top_k=0),
        # Prefill of the coarse layer: each of 8192 tokens to its two experts' rows.
        dict(name="quantize_prefill_bf16", op="quantize", dtype="bf16", rows=8192, K=4096, top_k=2),
        # Preparing a layer's gate weights: 128 experts x 768 rows, from FP32 masters.
        dict(name="quantize_weights_f32", op="quantize", dtype="f32", rows=98304, K=2048, top_k=0),
        # Decode step: 16 tokens x 8 of 128 experts; the touched weights' bytes count.
        dict(name="gate_up_decode_bf16", op="gate_up", dtype="bf16", T=16, E=128, top_k=8, H=2048, I=768, skew=0.0),
        # Fine-grained prefill, 256 rows an expert on average.
        dict(name="down_prefill_bf16", op="down", dtype="bf16", T=4096, E=128, top_k=8, H=2048, I=768, skew=0.0),
        # Skewed experts, ragged tails, F16.
        dict(name="gate_up_zipf_f16", op="gate_up", dtype="f16", T=16384, E=64, top_k=6, H=2048, I=1408, skew=1.2),
        # Odd token count, sizes that end inside every tile, FP32 outputs.
        dict(name="down_ragged_f32", op="down", dtype="f32", T=333, E=7, top_k=3, H=1184, I=736, skew=0.0),
        # Coarse prefill: the largest products.
        dict(name="gate_up_coarse_bf16", op="gate_up", dtype="bf16", T=8192, E=8, top_k=2, H=4096, I=14336, skew=0.0),
        # A router's and some norms' gradients: many small, odd tensors of two types.
        dict(name="grad_clip_small_mixed", op="grad_clip", dtype="mixed", tensors=60, total=1 << 20, clip=True),
        # BF16 gradients of a decode-sized layer, norm only (logged every step).
        dict(name="grad_norm_bf16", op="grad_norm", dtype="bf16", tensors=24, total=150_000_000, clip=True),
        # The training step's FP32 weight gradients of the fine-grained layer.
        dict(name="grad_clip_experts_f32", op="grad_clip", dtype="f32", tensors=3, total=603_979_776, clip=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // step * step if int(v) >= step else step))


def draw(rng):
    op = rng.choice(["quantize", "gate_up", "down", "grad_norm", "grad_clip"])
    if op == "quantize":
        K = _log_int(rng, 32, 14336, 32)
        rows = _log_int(rng, 1, min(98304, 200_000_000 // K))
        top_k = rng.choice([0, 0, 1, 2, 3, 8])
        if top_k:
            rows = max(1, rows // (2 * top_k))
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), rows=rows, K=K, top_k=top_k)
    if op in ("gate_up", "down"):
        E = rng.choice([1, 2, 5, 8, 16, 60, 64, 128])
        H = _log_int(rng, 256, 4096, 32)
        I = _log_int(rng, 256, min(14336, max(256, 400_000_000 // (E * H))), 32)
        T = _log_int(rng, 1, 16384)
        top_k = rng.randint(1, min(E, 8))
        T = max(1, min(T, 900_000_000_000 // (4 * top_k * H * I)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), T=T, E=E, top_k=top_k, H=H, I=I,
                    skew=rng.choice([0.0, 0.0, 0.8, 1.2]))
    return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32", "mixed"]),
                tensors=_log_int(rng, 1, 60 if op == "grad_clip" else 300), total=_log_int(rng, 1000, 300_000_000),
                clip=rng.random() < 0.75)


# ------------------------------------------------------------------ rows per expert, tensor sizes (from the case alone)

@functools.lru_cache(maxsize=64)
def _routing(T, E, top_k, skew):
    """Per token its top_k distinct experts, drawn with weights rank^-skew;
    returns the rows per expert."""
    rng = random.Random(f"route {T} {E} {top_k} {skew}")
    order = list(range(E))
    rng.shuffle(order)
    w = [0.0] * E
    for r, e in enumerate(order):
        w[e] = (r + 1.0) ** -skew
    cum = []
    s = 0.0
    for v in w:
        s += v
        cum.append(s)
    counts = [0] * E
    ids = range(E)
    for _ in range(T):
        chosen = set()
        if 2 * top_k > E:
            chosen = set(sorted(ids, key=lambda e: -w[e] * -math.log(1.0 - rng.random()))[:top_k])
        while len(chosen) < top_k:
            chosen.add(rng.choices(ids, cum_weights=cum)[0])
        for e in chosen:
            counts[e] += 1
    return tuple(counts)


@functools.lru_cache(maxsize=64)
def _sizes(tensors, total, dtype):
    """(elements, dtype name) of each gradient: the expert layer's three equal
    tensors, or a spread of sizes from one element up."""
    if tensors == 3 and dtype != "mixed":
        return tuple((total // 3, dtype) for _ in range(3))
    rng = random.Random(f"sizes {tensors} {total} {dtype}")
    w = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(tensors)]
    s = sum(w)
    kinds = ["f32", "bf16"] if dtype == "mixed" else [dtype]
    return tuple((max(1, int(total * v / s)), rng.choice(kinds)) for v in w)


def _pitch(K):
    return (K + 127) // 128 * 4


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["K"]
        out = case["rows"] * max(1, case["top_k"])
        # in once; out the codes, the scales and the values they stand for
        bytes_ = n * DTYPES[case["dtype"]].itemsize + out * (case["K"] // 2 + case["K"] // 32) + out * case["K"] * 2
        return {"bytes": bytes_, "flops": n}
    if op in ("gate_up", "down"):
        counts = _routing(case["T"], case["E"], case["top_k"], case["skew"])
        touched = sum(1 for c in counts if c)
        rows = sum(counts)
        H, I = case["H"], case["I"]
        K, N, mats = (H, I, 2) if op == "gate_up" else (I, H, 1)
        four = lambda n: n * (K // 2 + K // 32)
        return {"bytes": four(touched * mats * N) + four(rows) + rows * N * DTYPES[case["dtype"]].itemsize,
                "flops": 2 * mats * rows * N * K}
    nbytes = sum(n * DTYPES[d].itemsize for n, d in _sizes(case["tensors"], case["total"], case["dtype"]))
    n = sum(n for n, _ in _sizes(case["tensors"], case["total"], case["dtype"]))
    if op == "grad_norm":
        return {"bytes": nbytes + 4, "flops": 2 * n}
    # in once, out once (tensors beyond the on-chip memory are read again once the norm is known: 3 * nbytes)
    return {"bytes": 2 * nbytes + 4, "flops": 3 * n}


# ------------------------------------------------------------------ plain MXFP4

def _power_of_two(biased):
    """2^(biased - 127) in FP32 from its bits, biased in 0..254 (0: the subnormal 2^-127)."""
    return torch.where(biased > 0, biased.to(torch.int32) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _plain_quantize(x):
    """float [.., K] -> (E2M1 codes [.., K] int, biased exponents [.., K/32] int), in FP32."""
    v = x.to(torch.float32).unflatten(-1, (-1, 32))
    a = v.abs().amax(-1)
    _, ex = torch.frexp(a)                                    # a = m * 2^ex, m in [1/2, 1)
    byte = torch.where(a > 0, ex.to(torch.int32) - 3 + 127, 0).clamp(0, 254)
    m = (v * _power_of_two(254 - byte).unsqueeze(-1)).abs()
    code = torch.zeros_like(m, dtype=torch.int32)
    # ties go to the even mantissa: up across 0.75, 1.75, 3.5
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        code += (m >= border) if up else (m > border)
    code += torch.signbit(v).to(torch.int32) * 8
    bad = ~torch.isfinite(a)
    return torch.where(bad.unsqueeze(-1), 0, code).flatten(-2), torch.where(bad, 255, byte)


def _plain_values(code, byte, dtype):
    """E2M1 codes [.., K] and biased exponents [.., K/32] -> values in dtype."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=code.device)
    v = lut[code.long()].unflatten(-1, (-1, 32))
    s = torch.where(byte == 255, torch.nan, _power_of_two(byte.clamp(max=254)).to(dtype))
    return (v * s.unsqueeze(-1)).flatten(-2)


def _pack(code, byte, K):
    """Codes as bytes (element 2i in the low half), scales as bytes with rows of _pitch(K)."""
    c = code.unflatten(-1, (-1, 2))
    codes = (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8).contiguous()
    scales = torch.zeros(byte.shape[:-1] + (_pitch(K),), dtype=torch.uint8, device=byte.device)
    scales[..., :K // 32] = byte.to(torch.uint8)
    return codes, scales


def _unpack_values(codes, scales, K, dtype):
    c = codes.to(torch.int32)
    code = torch.stack((c & 15, c >> 4), -1).flatten(-2)
    return _plain_values(code, scales[..., :K // 32].to(torch.int32), dtype)


# ------------------------------------------------------------------ prepare

def _activations(rows, K, dtype, gen):
    """Normal activations with a few loud channels, as hidden states have."""
    x = torch.randn(rows, K, generator=gen, device=DEV)
    loud = torch.randint(0, K, (max(1, K // 256),), generator=gen, device=DEV)
    x[:, loud] *= 20.0
    return x.to(dtype)


def _mx_normal(shape, std, gen):
    """MXFP4 tensor (codes, scales) of N(0, std^2) values."""
    K = shape[-1]
    codes = torch.empty(shape[:-1] + (K // 2,), dtype=torch.uint8, device=DEV)
    scales = torch.empty(shape[:-1] + (_pitch(K),), dtype=torch.uint8, device=DEV)
    fc, fs = codes.view(-1, K // 2), scales.view(-1, _pitch(K))
    step = max(1, (1 << 26) // K)
    for r in range(0, fc.shape[0], step):
        n = min(step, fc.shape[0] - r)
        c, b = _plain_quantize(torch.randn(n, K, generator=gen, device=DEV) * std)
        fc[r:r + n], fs[r:r + n] = _pack(c, b, K)
    return codes, scales


def _row_maps(rows, top_k, gen):
    """A dispatch's maps for rows x top_k slots: (inv, row_src) of a random permutation."""
    n = rows * top_k
    row_src = torch.randperm(n, generator=gen, device=DEV)
    inv = torch.empty_like(row_src)
    inv[row_src] = torch.arange(n, device=DEV)
    return inv.to(torch.int32), row_src


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quantize":
        st["x"] = _activations(case["rows"], case["K"], DTYPES[case["dtype"]], gen)
        if case["top_k"]:
            st["inv"], st["row_src"] = _row_maps(case["rows"], case["top_k"], gen)
        return st
    if op in ("gate_up", "down"):
        E, H, I = case["E"], case["H"], case["I"]
        counts = _routing(case["T"], E, case["top_k"], case["skew"])
        st["counts"] = counts
        offs = [0]
        for c in counts:
            offs.append(offs[-1] + c)
        st["offsets"] = torch.tensor(offs, dtype=torch.int32, device=DEV)
        st["gate"] = _mx_normal((E, I, H), H ** -0.5, gen)
        st["up"] = _mx_normal((E, I, H), H ** -0.5, gen)
        st["down"] = _mx_normal((E, H, I), I ** -0.5, gen)
        K = H if op == "gate_up" else I
        act = _activations(offs[-1], K, torch.float32, gen)
        st["a"] = _pack(*_plain_quantize(act), K)
        if own:
            import moe_routing_swiglu_gb300 as moe

            st["experts"] = moe.ExpertsMxfp4(moe.Mxfp4(*st["gate"]), moe.Mxfp4(*st["up"]), moe.Mxfp4(*st["down"]))
            st["mx"] = moe.Mxfp4(*st["a"])
        return st
    grads = [(torch.randn(n, generator=gen, device=DEV) * 0.02).to(DTYPES[d])
             for n, d in _sizes(case["tensors"], case["total"], case["dtype"])]
    n = sum(g.numel() for g in grads)
    st["grads"] = grads
    # a clip that acts (half the expected norm) or one that leaves the gradients alone
    st["max_norm"] = 0.02 * math.sqrt(n) * (0.5 if case["clip"] else 2.0)
    if op == "grad_clip":
        st["out"] = [torch.empty_like(g) for g in grads]
    return st


# ------------------------------------------------------------------ run

def _experts_plain(st, dtype):
    """The experts' product per expert from the MXFP4 values in `dtype` arithmetic (FP32 or FP64)."""
    case = st["case"]
    H, I = case["H"], case["I"]
    K, N = (H, I) if case["op"] == "gate_up" else (I, H)
    a = _unpack_values(*st["a"], K, dtype)
    out = torch.zeros(a.shape[0], N, dtype=dtype, device=DEV)
    r = 0
    for e, c in enumerate(st["counts"]):
        if c:
            x = a[r:r + c]
            if case["op"] == "gate_up":
                g = x @ _unpack_values(st["gate"][0][e], st["gate"][1][e], K, dtype).T
                u = x @ _unpack_values(st["up"][0][e], st["up"][1][e], K, dtype).T
                out[r:r + c] = g / (1.0 + torch.exp(-g)) * u
            else:
                out[r:r + c] = x @ _unpack_values(st["down"][0][e], st["down"][1][e], K, dtype).T
        r += c
    return out


def _norm_plain(grads):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in grads:
        total = total + g.to(torch.float32).square().sum(dtype=torch.float64)
    return total.sqrt().to(torch.float32)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import moe_routing_swiglu_gb300 as moe

        if op == "quantize":
            q = moe.moe_mxfp4_quantize(st["x"], inv=st.get("inv"), top_k=max(1, case["top_k"]))
            return moe.moe_mxfp4_dequantize(q, torch.bfloat16)
        if op == "gate_up":
            return moe.moe_experts_mxfp4_gate_up(st["experts"], st["mx"], st["offsets"], dtype=DTYPES[case["dtype"]])
        if op == "down":
            return moe.moe_experts_mxfp4_down(st["experts"], st["mx"], st["offsets"], dtype=DTYPES[case["dtype"]])
        if op == "grad_norm":
            return moe.moe_grad_norm(st["grads"])
        norm = moe.moe_clip_grad_norm(st["grads"], st["max_norm"], out=st["out"])
        return [norm] + st["out"]
    if op == "quantize":
        code, byte = _plain_quantize(st["x"])
        v = _plain_values(code, byte, torch.float32).to(torch.bfloat16)
        return v[st["row_src"] // case["top_k"]] if case["top_k"] else v
    if op in ("gate_up", "down"):
        return _experts_plain(st, torch.float32).to(DTYPES[case["dtype"]])
    norm = _norm_plain(st["grads"])
    if op == "grad_norm":
        return norm
    coef = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm))
    return [norm] + [(g.to(torch.float32) * coef).to(g.dtype) for g in st["grads"]]


# ------------------------------------------------------------------ exact

def _exact_round4(y):
    """The nearest E2M1 value to y in [0, 8), ties to the even mantissa, saturated to 6: the grid's step is 1/2 below
    2, 1 below 4, 2 above (torch.round takes ties to even)."""
    step = torch.where(y < 2.0, 0.5, torch.where(y < 4.0, 1.0, 2.0)).to(torch.float64)
    return (torch.round(y / step) * step).clamp(max=6.0)


def exact(case, seed):
    w = work(case)
    if w["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, k = st["x"], case["top_k"]
        out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 25) // case["K"])
        for r in range(0, x.shape[0], step):
            v = x[r:r + step].double().unflatten(-1, (-1, 32))
            a = v.abs().amax(-1, keepdim=True)
            e = torch.where(a > 0, torch.floor(torch.log2(a)), torch.zeros_like(a)).clamp(min=-125)
            power = lambda n: ((n.long() + 1023) << 52).view(torch.float64)   # 2^n from its bits
            e = torch.where(power(e) > a, e - 1, torch.where(power(e + 1) <= a, e + 1, e)).clamp(min=-125)
            scale = power(e - 2)
            out[r:r + step] = (torch.sign(v) * _exact_round4(v.abs() / scale) * scale).flatten(-2)
        return out[st["row_src"] // k] if k else out
    if op in ("gate_up", "down"):
        H, I = case["H"], case["I"]
        K, N = (H, I) if op == "gate_up" else (I, H)
        half = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12, 0, -1, -2, -3, -4, -6, -8, -12], device=DEV).double() / 2

        def values(pair):
            codes, scales = pair
            v = torch.empty(codes.shape[0], K, dtype=torch.float64, device=DEV)
            v[:, 0::2] = half[(codes % 16).long()]
            v[:, 1::2] = half[(codes // 16).long()]
            return v * torch.exp2(scales[:, :K // 32].double() - 127).repeat_interleave(32, dim=1)

        at = lambda m, e: (st[m][0][e], st[m][1][e])
        out = torch.empty(sum(st["counts"]), N, dtype=torch.float64, device=DEV)
        lo = 0
        for e, c in enumerate(st["counts"]):
            if c == 0:
                continue
            x = values((st["a"][0][lo:lo + c], st["a"][1][lo:lo + c]))
            if op == "gate_up":
                g = torch.einsum("tk,nk->tn", x, values(at("gate", e)))
                u = torch.einsum("tk,nk->tn", x, values(at("up", e)))
                out[lo:lo + c] = g * torch.sigmoid(g) * u
            else:
                out[lo:lo + c] = torch.einsum("tk,nk->tn", x, values(at("down", e)))
            lo += c
        return out
    total = sum(torch.dot(g.double(), g.double()) for g in st["grads"])
    norm = torch.sqrt(total)
    if op == "grad_norm":
        return norm
    scale = min(1.0, st["max_norm"] / float(norm))
    return [norm] + [g.double() * scale for g in st["grads"]]
