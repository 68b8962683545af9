"""GPU checks of the norms around a block against the FP64 formulas (oracle/block.py).

Tolerances, relative to the sizes of a result's terms added up without their signs (oracle/block.py, *_size): a row sum
has at most 8 additions in a thread, 5 + 4 + 5 over the row's warps, products of at most 4 roundings each; with the
root, the division and the products after it every FP32 result is within 40 roundings, 40 * 2^-24 < 2^-18 of its size.
A column's sum over T rows adds (T + 16) 2^-24 at most. The combined branch adds top_k 2^-24 of sum |w y|. Then the
output's own rounding, half a step of its type. An output that underflows is off by half the type's smallest step."""
import numpy as np
import pytest
import torch

from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
REL = 2.0 ** -18
EPS = 1e-3

# one column; odd; one warp; several rows a block, ragged; whole blocks; odd block; one block of 4096; clusters of 2, 4, 8
SHAPES = [(1, 1), (5, 7), (9, 33), (19, 64), (37, 72), (3, 256), (17, 264), (16, 2048), (21, 1409), (7, 4096), (5, 4104),
          (3, 5001), (3, 8192), (2, 16390), (2, 32768)]
# more rows than one round of the blocks: rows come through shared memory, rounds ahead
LONG = [(20001, 64), (2500, 264), (1301, 2048), (2201, 1000), (1400, 1409), (700, 4104), (500, 8192), (330, 16392)]


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, size, extra=0.0):
    """|got - ref| within the rounding of got's type and `REL` (and extra) of size; NaN where ref is."""
    u = torch.finfo(got.dtype).eps / 2
    g = f64(got)
    assert g.shape == ref.shape
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    tol = u * np.abs(ref) + (REL * (1 + u) + extra) * size + torch.finfo(got.dtype).smallest_normal * u
    bad = ~np.isnan(ref) & ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - ref) / tol)[bad].max()))


def grads(rng, T, H, dtype):
    return torch.tensor(rng.normal(size=(T, H)), dtype=DTYPES[dtype], device=DEV)


def rows(rng, T, H, dtype, zeros=False):
    """Hidden states: a loud channel, a scale of its own for each row, one row of zeros if asked."""
    v = rng.normal(size=(T, H)) * np.exp(rng.normal(size=(T, 1)))
    v[:, rng.integers(H)] *= 20
    if zeros and T > 4:
        v[2] = 0
    return torch.tensor(v, dtype=DTYPES[dtype], device=DEV)


def vector(rng, n, dtype):
    return torch.tensor(1 + 0.3 * rng.normal(size=n), dtype=dtype, device=DEV)


@pytest.mark.parametrize("T,H", SHAPES + LONG)
@pytest.mark.parametrize("dtype,vec", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_norm_and_its_backward(cuda_lib, T, H, dtype, vec):
    moe = cuda_lib
    rng = np.random.default_rng(T * H)
    x, dy, dres = rows(rng, T, H, dtype, zeros=True), grads(rng, T, H, dtype), grads(rng, T, H, dtype)
    w = vector(rng, H, DTYPES[vec])
    y = moe.moe_block_norm(x, w, eps=EPS)
    ref = block.norm(f64(x), f64(w), EPS)
    check(y, ref, np.abs(ref))
    for extra in (dres, None):
        g = moe.moe_block_norm_backward(dy, x, w, eps=EPS, dresidual=extra)
        d = 0.0 if extra is None else f64(extra)
        dx, dw = block.norm_backward(f64(x), f64(w), f64(dy), EPS)
        sx, sw = block.norm_backward_size(f64(x), f64(w), np.abs(f64(dy)), EPS)
        check(g.dx, dx + d, sx + np.abs(d))
        check(g.dweight, dw, sw, (T + 16) * 2.0 ** -24)


def gate_of(rng, kind, T, H, dtype, vec):
    if kind == "none":
        return None
    shape = {"channel": (H,), "token": (T, 1), "element": (T, H)}[kind]
    return torch.tensor(rng.normal(size=shape), dtype=DTYPES[dtype if kind == "element" else vec], device=DEV)


def opt(t):
    return None if t is None else f64(t)


PARTS = [("none", True, True), ("channel", True, True), ("token", True, True), ("element", True, True),
         ("channel", False, True), ("token", True, False), ("element", False, False), ("none", False, False),
         ("token", False, True)]


def join_case(rng, T, H, dtype, vec, kind, post, nxt):
    p = dict(norm_weight=vector(rng, H, DTYPES[vec]) if post else None, gate=gate_of(rng, kind, T, H, dtype, vec),
             next_weight=vector(rng, H, DTYPES[vec]) if nxt else None, residual_scale=0.8, branch_scale=-1.25, eps=EPS)
    return rows(rng, T, H, dtype, zeros=True), rows(rng, T, H, dtype), p


def check_join(out, y, f, x, p, f_size=None):
    """out and y of a join of the FP64 branch f; f_size: how far f itself may be off, over its REL."""
    w, w2 = opt(p["norm_weight"]), opt(p["next_weight"])
    g = 1.0 if p["gate"] is None else f64(p["gate"])
    ref = block.join(f, f64(x), w, g, 0.8, -1.25, EPS)
    size = np.abs(0.8 * f64(x)) + np.abs(ref - 0.8 * f64(x))
    if f_size is not None:
        # f off by e: norm(f) moves by at most (|e| + |f| |e| rms / rms(f)) r w
        move = f_size
        if w is not None:
            r = block.rstd(f, EPS)
            move = r * np.abs(w) * (f_size + np.abs(f) * r * np.sqrt((f_size ** 2).mean(-1, keepdims=True)))
        size = size + 1.25 * np.abs(g) * move
    check(out, ref, size)
    if w2 is None:
        assert y is None
    else:   # the norm of what was stored
        ref = block.norm(f64(out), w2, EPS)
        check(y, ref, np.abs(ref))


def check_join_backward(moe, dout, dy, f, joined, p, got):
    T, H = f.shape
    g = np.ones((1, 1)) if p["gate"] is None else f64(p["gate"])
    args = (f64(dout) if dout is not None else np.zeros((T, H)), opt(dy), f64(f), opt(joined), opt(p["norm_weight"]), g,
            opt(p["next_weight"]), 0.8, -1.25, EPS)
    ref, size = block.join_backward(*args), block.join_backward_size(*args)
    cols = (T + 16) * 2.0 ** -24
    check(got.dbranch, ref.dbranch, size.dbranch)
    check(got.dresidual, ref.dresidual, size.dresidual)
    for name in ("dnorm_weight", "dnext_weight"):
        if getattr(ref, name) is None:
            assert getattr(got, name) is None
        else:
            check(getattr(got, name), getattr(ref, name), getattr(size, name), cols)
    if p["gate"] is None:
        assert got.dgate is None
    elif p["gate"].shape == (T, H):
        check(got.dgate, ref.dgate_full, size.dgate_full)
    elif p["gate"].dim() == 1:
        check(got.dgate, ref.dgate_full.sum(0), size.dgate_full.sum(0), cols)
    else:   # expanded into row sums: the sum of the sizes, with those of the projection on joined
        check(got.dgate, ref.dgate_full.sum(1, keepdims=True), size.dgate_full.sum(1, keepdims=True))


@pytest.mark.parametrize("T,H", SHAPES + LONG)
@pytest.mark.parametrize("kind,post,nxt", PARTS)
def test_join_and_its_backward(cuda_lib, T, H, kind, post, nxt):
    moe = cuda_lib
    if (T, H) in LONG and PARTS.index((kind, post, nxt)) > 5:
        pytest.skip("the shorter list of parts")
    i = (SHAPES + LONG).index((T, H)) + PARTS.index((kind, post, nxt))
    dtype, vec = [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32")][i % 4]
    rng = np.random.default_rng(T * H + i)
    f, x, p = join_case(rng, T, H, dtype, vec, kind, post, nxt)
    if kind == "element" and H == 1:
        p["gate"] = p["gate"].view(T, H)
    out, y = moe.moe_block_join(f, x, **p)
    check_join(out, y, f64(f), x, p)
    dout, dy = grads(rng, T, H, dtype), grads(rng, T, H, dtype)
    got = moe.moe_block_join_backward(dout, f, dnormed=dy if nxt else None, joined=out if nxt else None, **p)
    check_join_backward(moe, dout, dy if nxt else None, f, out if nxt else None, p, got)
    if nxt:
        got = moe.moe_block_join_backward(None, f, dnormed=dy, joined=out, **p)
        check_join_backward(moe, None, dy, f, out, p, got)


@pytest.mark.parametrize("T,k,H", [(1, 1, 64), (16, 8, 2048), (5, 3, 33), (3, 13, 5000), (130, 2, 96), (2, 5, 8192),
                                   (9001, 3, 64), (900, 8, 2048), (400, 2, 8192), (900, 40, 256), (700, 33, 33)])
@pytest.mark.parametrize("dtype,wdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("kind,post,nxt", [("token", True, True), ("none", False, True), ("channel", True, False)])
def test_combine_join(cuda_lib, T, k, H, dtype, wdt, kind, post, nxt):
    moe = cuda_lib
    rng = np.random.default_rng(T * H + k)
    _, x, p = join_case(rng, T, H, dtype, "f32", kind, post, nxt)
    yd = torch.tensor(rng.normal(size=(T * k, H)), dtype=DTYPES[dtype], device=DEV)
    inv = rng.permutation(T * k)
    wt = torch.tensor(rng.uniform(size=(T, k)), dtype=DTYPES[wdt], device=DEV)
    terms = f64(wt)[..., None] * f64(yd)[inv].reshape(T, k, H)
    out, y = moe.moe_combine_join(yd, torch.tensor(inv, dtype=torch.int32, device=DEV), wt, x, **p)
    check_join(out, y, terms.sum(1), x, p, np.abs(terms).sum(1) * (k * 2.0 ** -24 / REL))


def test_combine_join_in_fp32_is_the_join_of_the_combine(cuda_lib):
    """FP32 rows: the combine's rounding is its FP32 sum, so both ways give the same bits."""
    moe = cuda_lib
    rng = np.random.default_rng(3)
    f, x, p = join_case(rng, 40, 200, "f32", "f32", "token", True, True)
    yd = torch.tensor(rng.normal(size=(160, 200)), dtype=torch.float32, device=DEV)
    inv = torch.tensor(rng.permutation(160), dtype=torch.int32, device=DEV)
    wt = torch.rand(40, 4, device=DEV)
    for a, b in zip(moe.moe_combine_join(yd, inv, wt, x, **p),
                    moe.moe_block_join(moe.moe_combine(yd, inv, wt), x, **p)):
        assert torch.equal(a, b)


def test_a_bad_slot_or_row_stays_in_its_row(cuda_lib):
    moe = cuda_lib
    rng = np.random.default_rng(4)
    for T in (12, 6000):
        bad_slot(moe, rng, T)


def bad_slot(moe, rng, T):
    k, H = 2, 72
    f, x, p = join_case(rng, T, H, "bf16", "f32", "channel", True, True)
    yd = torch.tensor(rng.normal(size=(T * k, H)), dtype=torch.bfloat16, device=DEV)
    inv = torch.tensor(rng.permutation(T * k), dtype=torch.int32, device=DEV)
    wt = torch.rand(T, k, device=DEV)
    good = moe.moe_combine_join(yd, inv, wt, x, **p)
    inv[7] = -1                                            # 0xFFFFFFFF: not dispatched
    bad = moe.moe_combine_join(yd, inv, wt, x, **p)
    keep = [t for t in range(T) if t != 3]
    for a, b in zip(good, bad):
        assert torch.isnan(b[3]).all() and torch.equal(a[keep], b[keep])
    x2 = x.clone()
    x2[5, 3] = float("inf")
    y = moe.moe_block_norm(x2, p["next_weight"])
    assert torch.isnan(y[5, 3]) and (y[5, :3] == 0).all()  # inf / inf, finite / inf
    keep = [t for t in range(T) if t != 5]
    assert torch.equal(y[keep], moe.moe_block_norm(x, p["next_weight"])[keep])


def test_no_rows(cuda_lib):
    moe = cuda_lib
    w, x = torch.ones(40, device=DEV), torch.empty(0, 40, dtype=torch.bfloat16, device=DEV)
    assert moe.moe_block_norm(x, w).shape == (0, 40)
    assert (moe.moe_block_norm_backward(x, x, w).dweight == 0).all()
    out, y = moe.moe_block_join(x, x, norm_weight=w, next_weight=w, gate=w)
    assert out.shape == y.shape == (0, 40)
    g = moe.moe_block_join_backward(x, x, dnormed=x, joined=x, norm_weight=w, next_weight=w, gate=w)
    assert all((t == 0).all() for t in (g.dnorm_weight, g.dnext_weight, g.dgate))
    g = moe.moe_block_join_backward(x, x, norm_weight=w, gate=torch.empty(0, 1, device=DEV))
    assert (g.dnorm_weight == 0).all() and g.dgate.shape == (0, 1)


def test_in_place_and_the_rows_behind(cuda_lib):
    """Outputs in the inputs' place give the same bits, and rows past T stay as they were."""
    moe = cuda_lib
    rng = np.random.default_rng(5)
    for T, H, dtype in ((6, 2056, "bf16"), (3, 4200, "f16"), (11, 45, "f32"), (1500, 2048, "f16"), (400, 4104, "f32")):
        f, x, p = join_case(rng, T, H, dtype, "f32", "element", True, True)
        ref = moe.moe_block_join(f, x, **p)
        big = torch.full((T + 2, H), 7.0, dtype=x.dtype, device=DEV)
        big[:T] = x
        f2 = f.clone()
        out, y = moe.moe_block_join(f2, big[:T], out=big[:T], normed=f2, **p)
        assert torch.equal(big[:T], ref[0]) and torch.equal(f2, ref[1]) and (big[T:] == 7).all()
        dout, dy = grads(rng, T, H, dtype), grads(rng, T, H, dtype)
        ref = moe.moe_block_join_backward(dout, f, dnormed=dy, joined=out, **p)
        got = moe.moe_block_join_backward(dout, f, dnormed=dy, joined=out, dresidual=dout, dbranch=f, **p)
        for a, b in zip(ref, got):
            assert torch.equal(a, b)
        x2 = x.clone()
        assert torch.equal(moe.moe_block_norm(x2, p["norm_weight"], out=x2), moe.moe_block_norm(x, p["norm_weight"]))


def test_unaligned_rows_match_aligned_ones(cuda_lib):
    """Rows one element past a 16-byte boundary take the narrow loads: same sums in another order."""
    moe = cuda_lib
    rng = np.random.default_rng(6)
    T, H = 9, 520
    f, x, p = join_case(rng, T, H, "bf16", "f32", "token", True, True)
    off = torch.empty(T * H + 1, dtype=x.dtype, device=DEV)[1:].view(T, H)
    off.copy_(x)
    out, y = moe.moe_block_join(f, off, **p)
    check_join(out, y, f64(f), x, p)


def shifted(t, by, behind=0):
    """A copy of t that starts `by` elements into its memory, at the end of it but for `behind`."""
    room = torch.full((t.numel() + by + behind,), 7.0, dtype=t.dtype, device=DEV)
    view = room[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


# odd rows through shared memory, several rounds: many rows a block, one, a cluster's; H under a granule; H even but no
# multiple of 8; rows of whole granules at odd places
LOOSE = [(20003, 3), (21001, 63), (5003, 129), (2501, 518), (3001, 1023), (701, 4095), (403, 8191), (301, 16393),
         (2500, 264), (1301, 2048)]


@pytest.mark.parametrize("T,H", LOOSE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_off_granules_in_rounds(cuda_lib, T, H, dtype):
    moe = cuda_lib
    rng = np.random.default_rng(T + H)
    kind, post, nxt = PARTS[(T + len(dtype)) % 4]
    f, x, p = join_case(rng, T, H, dtype, "f32", kind, post, nxt)
    dout, dy = grads(rng, T, H, dtype), grads(rng, T, H, dtype)
    f, x, dout, dy = (shifted(t, by) for t, by in ((f, 1), (x, 3), (dout, 0), (dy, 7)))
    if kind == "element":
        p["gate"] = shifted(p["gate"], 5)
    out, y = moe.moe_block_join(f, x, **p)
    check_join(out, y, f64(f), x, p)
    joined = shifted(out, 2)
    check_join_backward(moe, dout, dy, f, joined, p, moe.moe_block_join_backward(dout, f, dnormed=dy, joined=joined, **p))
    w = p["norm_weight"]
    y = moe.moe_block_norm(x, w, eps=EPS)
    ref = block.norm(f64(x), f64(w), EPS)
    check(y, ref, np.abs(ref))
    g = moe.moe_block_norm_backward(dy, x, w, eps=EPS, dresidual=dout)
    dx, dw = block.norm_backward(f64(x), f64(w), f64(dy), EPS)
    sx, sw = block.norm_backward_size(f64(x), f64(w), np.abs(f64(dy)), EPS)
    check(g.dx, dx + f64(dout), sx + np.abs(f64(dout)))
    check(g.dweight, dw, sw, (T + 16) * 2.0 ** -24)
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("T,k,H", [(20003, 2, 3), (3001, 3, 129), (700, 8, 2047), (400, 3, 8191), (900, 32, 130),
                                   (900, 8, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combined_rows_off_granules_in_rounds(cuda_lib, T, k, H, dtype):
    moe = cuda_lib
    rng = np.random.default_rng(T + k)
    _, x, p = join_case(rng, T, H, dtype, "f32", "element" if k == 3 else "token", True, True)
    yd = shifted(torch.tensor(rng.normal(size=(T * k, H)), dtype=DTYPES[dtype], device=DEV), 1)
    x = shifted(x, 3)
    inv = rng.permutation(T * k)
    wt = torch.tensor(rng.uniform(size=(T, k)), dtype=torch.float32, device=DEV)
    terms = f64(wt)[..., None] * f64(yd)[inv].reshape(T, k, H)
    idx = torch.tensor(inv, dtype=torch.int32, device=DEV)
    out, y = moe.moe_combine_join(yd, idx, wt, x, **p)
    check_join(out, y, terms.sum(1), x, p, np.abs(terms).sum(1) * (k * 2.0 ** -24 / REL))
    idx[5] = T * k   # no such row: the token's rows are NaN, the others as they were
    o2, y2 = moe.moe_combine_join(yd, idx, wt, x, **p)
    bad = 5 // k
    keep = torch.arange(T, device=DEV) != bad
    assert torch.isnan(o2[bad]).all() and torch.isnan(y2[bad]).all()
    assert torch.equal(o2[keep], out[keep]) and torch.equal(y2[keep], y[keep])
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("T,H,dtype", [(5003, 129, "bf16"), (701, 4095, "f16"), (403, 8191, "bf16"), (3001, 1023, "f32")])
def test_loose_rows_in_place_and_the_rows_behind(cuda_lib, T, H, dtype):
    """The granules beside a row are being written by other blocks: the same bits as out of place, nothing else written."""
    moe = cuda_lib
    rng = np.random.default_rng(H)
    f, x, p = join_case(rng, T, H, dtype, "f32", "element", True, True)
    dout, dy = grads(rng, T, H, dtype), grads(rng, T, H, dtype)
    ref = moe.moe_block_join(f, x, **p)
    room = torch.full((T * H + 11,), 7.0, dtype=x.dtype, device=DEV)
    x2, f2 = room[3:3 + T * H].view(T, H), f.clone()
    x2.copy_(x)
    moe.moe_block_join(f2, x2, out=x2, normed=f2, **p)
    assert torch.equal(x2, ref[0]) and torch.equal(f2, ref[1])
    assert (room[:3] == 7).all() and (room[3 + T * H:] == 7).all()
    want = moe.moe_block_join_backward(dout, f, dnormed=dy, joined=ref[0], **p)
    d2, f2, j2, y2 = dout.clone(), f.clone(), ref[0].clone(), dy.clone()
    got = moe.moe_block_join_backward(d2, f2, dnormed=y2, joined=j2, dresidual=y2, dbranch=f2, **p)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    x2.copy_(x)
    moe.moe_block_norm(x2, p["norm_weight"], out=x2)
    assert torch.equal(x2, moe.moe_block_norm(x, p["norm_weight"]))
    assert (room[:3] == 7).all() and (room[3 + T * H:] == 7).all()
    assert moe.moe_device_status() == 0


def test_many_rows_and_far_offsets(cuda_lib):
    """More rows than one wave, and more than 2^31 elements: the last rows against the formula."""
    moe = cuda_lib
    T, H = 530_000, 4104
    x = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(3, H, device=DEV).to(torch.bfloat16)
    x[-3:] = tail
    w = vector(np.random.default_rng(1), H, torch.float32)
    y = moe.moe_block_norm(x, w, eps=EPS, out=x)
    ref = block.norm(f64(tail), f64(w), EPS)
    check(y[-3:], ref, np.abs(ref))
    ref = block.norm(np.ones((1, H)), f64(w), EPS)
    check(y[T // 2:T // 2 + 1], ref, np.abs(ref))


def test_streams_graphs_and_repeats(cuda_lib):
    """The same bits on another stream, from two captured graphs replayed together, and on every run."""
    moe = cuda_lib
    rng = np.random.default_rng(9)
    T, H = 2300, 1000
    f, x, p = join_case(rng, T, H, "bf16", "bf16", "channel", True, True)
    dout, dy = grads(rng, T, H, "bf16"), grads(rng, T, H, "bf16")
    p["gate"] = p["gate"].to(torch.bfloat16)

    def both(stream=None):
        out, y = moe.moe_block_join(f, x, stream=stream, **p)
        return [out, y, *moe.moe_block_join_backward(dout, f, dnormed=dy, joined=out, stream=stream, **p)]

    ref = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(ref, o))
    assert moe.moe_device_status() == 0


def test_refusals_of_the_binding(cuda_lib):
    moe = cuda_lib
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_block_norm(x[:, ::2], w[:32])
    with pytest.raises(ValueError):
        moe.moe_block_norm(x.cpu(), w)
    bad = [
        lambda: moe.moe_block_norm(x, w[:32]),
        lambda: moe.moe_block_norm(x, w.half()),
        lambda: moe.moe_block_norm(x.double(), w),
        lambda: moe.moe_block_norm(x, w, out=x.float()),
        lambda: moe.moe_block_norm(x, w, out=x.view(-1)[:0].view(0, 64)),
        lambda: moe.moe_block_join(x, x.float()),
        lambda: moe.moe_block_join(x, x, gate=torch.ones(3, 1, device=DEV)),
        lambda: moe.moe_block_join(x, x, gate=torch.ones(4, 64, device=DEV)),
        lambda: moe.moe_block_join(x, x, norm_weight=w, next_weight=w.bfloat16()),
        lambda: moe.moe_block_join(x, x, normed=x.clone()),
        lambda: moe.moe_block_join_backward(None, x),
        lambda: moe.moe_block_join_backward(x, x, next_weight=w),
        lambda: moe.moe_combine_join(x, torch.zeros(4, dtype=torch.int64, device=DEV), torch.ones(4, 1, device=DEV), x),
        lambda: moe.moe_combine_join(x, torch.zeros(8, dtype=torch.int32, device=DEV), torch.ones(4, 2, device=DEV), x),
    ]
    for call in bad:
        with pytest.raises(moe.MoeError):
            call()
