"""The training operators on the GPU against plain float64 forms.

Tolerances count roundings. A product of depth D accumulated in fp32, each
addition off by at most one unit in the last place (tensor cores may
truncate), is within D * 2^-23 * sum |a b| of the exact sum; a bf16 result
adds half a unit, 2^-8 of the value, and an fp32 one 2^-24."""
import math

import pytest
import torch

import sigmoid_group_limited_b200 as sgl

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
F8 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _offsets(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o.cuda()


# ------------------------------------------------------------------ grouped products
def _direct(direction, counts, a, b, out, accumulate):
    """(exact result, sum of magnitudes) per output, in float64; rows of no
    expert keep what `out` holds and get magnitude 0."""
    ref = out.to(F64)
    mag = torch.zeros_like(ref)
    lo = 0
    for e, c in enumerate(counts):
        hi = lo + c
        if direction == "wgrad":
            x, y = a[lo:hi].to(F64).t(), b[lo:hi].to(F64)
            at = e
        else:
            w = b[e].to(F64)
            x, y = a[lo:hi].to(F64), (w.t() if direction == "linear" else w)
            at = slice(lo, hi)
        if direction == "wgrad" or c:
            ref[at] = x @ y + (ref[at] if accumulate else 0)
            mag[at] = x.abs() @ y.abs()
        lo = hi
    return ref, mag


def _check_product(got, ref, mag, depth, touched, accumulate=False):
    assert torch.equal(got[~touched].to(F64), ref[~touched]), "an output of no expert changed"
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    acc = depth * 2.0 ** -23 * mag
    tol = acc + half * (ref.abs() + acc) + (2.0 ** -24 * (ref.abs() + mag) if accumulate else 0)
    bad = ((got.to(F64) - ref).abs() > tol) & touched
    assert not bad.any(), f"{int(bad.sum())} of {int(touched.sum())} off, first at {bad.nonzero()[0].tolist()}"


def _run(direction, a, b, offsets, out, accumulate=False, ws=None, stream=None):
    E = offsets.numel() - 1
    if ws is None:
        ws = sgl.alloc_linear_workspace(E, a.shape[0], 8, 8)
    if direction == "linear":
        sgl.moe_grouped_linear(a, offsets, b, out, ws, accumulate, stream)
    elif direction == "dgrad":
        sgl.moe_grouped_linear_dgrad(a, offsets, b, out, ws, accumulate, stream)
    else:
        sgl.moe_grouped_linear_wgrad(a, b, offsets, out, ws, accumulate, stream)
    return ws


def _product(direction, counts, N, K, out=BF, accumulate=False, spare=0, seed=0, pad=0):
    """Inputs and output of a product; pad: extra columns of the row-wise
    tensors (their row stride); spare rows hold NaN."""
    g = _gen(seed)
    R = sum(counts) + spare

    def rows(width, dtype=BF):
        t = _randn((R, width + pad), g, dtype)[:, :width]
        t[sum(counts):] = float("nan")
        return t

    if direction == "linear":
        a, b, o = rows(K), _randn((len(counts), N, K), g), rows(N, out)
    elif direction == "dgrad":
        a, b, o = rows(N), _randn((len(counts), N, K), g), rows(K, out)
    else:
        a, b, o = rows(N), rows(K), _randn((len(counts), N, K), g, out)
    if direction != "wgrad":
        o[sum(counts):] = 7.0
    return a, b, o


def _check(direction, counts, N, K, **kw):
    a, b, out = _product(direction, counts, N, K, **kw)
    acc = kw.get("accumulate", False)
    ref, mag = _direct(direction, counts, a, b, out, acc)
    total = sum(counts)
    ws = _run(direction, a, b, _offsets(counts), out, acc)
    assert sgl.moe_linear_read_error(ws) == 0
    touched = torch.ones_like(out, dtype=torch.bool)
    if direction != "wgrad":
        touched[total:] = False
    elif acc:
        touched[torch.tensor(counts) == 0] = False
    depth = {"linear": K, "dgrad": N, "wgrad": max(1, max(counts))}[direction]
    _check_product(out, ref, mag, depth, touched, acc)


DIRECTIONS = ("linear", "dgrad", "wgrad")
SHAPES = [  # counts, N, K
    ([1], 8, 8),
    ([0, 1, 0], 16, 64),
    ([3, 0, 1, 17], 72, 40),
    ([64, 63, 65, 1], 64, 64),
    ([127, 0, 128, 129, 5], 136, 200),
    ([255, 256, 257], 264, 136),
    ([300, 0, 0, 700], 768, 64),
    ([0, 0, 0, 33], 256, 2560),
    ([15, 16, 17, 31, 32, 33, 1, 0], 776, 328),
    ([1] * 8 + [0] * 24, 768, 2560),
    ([2, 0, 1, 5, 0, 0, 0, 4], 2560, 768),
    ([513], 512, 520),
]


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("counts,N,K", SHAPES, ids=lambda v: str(v)[:24])
def test_grouped_product(direction, counts, N, K):
    _check(direction, counts, N, K, seed=N + K)


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 1, 17], 72, 40), ([255, 0, 256, 257, 40], 264, 136),
                                        ([5, 1], 768, 2560)], ids=lambda v: str(v)[:24])
def test_grouped_product_fp32(direction, accumulate, counts, N, K):
    _check(direction, counts, N, K, out=F32, accumulate=accumulate, seed=3)


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_product_strides_and_spare_rows(direction, out):
    # row strides above the width, spare rows of NaN behind the last expert
    _check(direction, [40, 0, 131, 7], 200, 72, out=out, spare=60, pad=24, seed=5)
    _check(direction, [2, 0, 1], 200, 72, out=out, spare=300, pad=8, seed=6)


@pytest.mark.parametrize("direction", DIRECTIONS)
def test_grouped_product_many_experts(direction):
    g = torch.Generator().manual_seed(9)
    counts = torch.bincount(torch.randint(0, 1024, (3000,), generator=g) ** 2 // 1024, minlength=1024).tolist()
    _check(direction, counts, 64, 128, seed=9)


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_product_many_wide_tiles(direction, out):
    """Enough work for full-width tiles (narrower ones serve small calls): rows
    around the multiples of 256, several rounds per pair."""
    counts = [(e * 97) % 530 for e in range(56)] + [0, 255, 256, 257, 511, 512, 513, 1]
    n, k = (72, 776) if direction == "dgrad" else (776, 328)
    _check(direction, counts, n, k, out=out, seed=13, spare=33)


@pytest.mark.parametrize("out,accumulate", [(BF, False), (F32, False), (F32, True)])
@pytest.mark.parametrize("N,K", [(8, 8), (40, 264), (24, 776), (104, 1288), (72, 2568), (8, 7688)])
def test_few_rows(out, accumulate, N, K):
    """Up to 128 rows spread over the experts: every unit size (1 to 4 rows of
    an expert and their remainders), every number of slabs of K."""
    for counts in ([1], [0, 2], [3, 0, 4, 5, 0, 1], [1, 2, 3, 4, 5, 6, 7, 8, 9] + [0] * 9, [2] * 32 + [1] * 33,
                   [0] * 30 + [128] + [0], [0] * 31 + [129]):
        _check("linear", counts, N, K, out=out, accumulate=accumulate, seed=N + K, spare=len(counts) % 2, pad=8)


@pytest.mark.parametrize("direction", DIRECTIONS)
def test_grouped_product_long_depth(direction):
    # 2560 features and a contraction of thousands of rows
    _check(direction, [0, 4500, 3], 256, 2560, out=F32, seed=11)


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("counts", [[3, 0, 2], [40, 0, 150, 9]], ids=["few", "many"])
def test_spare_rows_in_front(direction, counts):
    """offsets[0] above zero: the rows before the first expert are spare."""
    lead, N, K = 21, 72, 136
    a, b, out = _product(direction, [lead] + counts, N, K, seed=7)
    off = _offsets([lead] + counts)[1:].clone()
    a[:lead] = float("nan")
    if direction == "wgrad":
        b[:lead] = float("nan")
        out = out[1:].contiguous()
    else:
        b = b[1:].contiguous()
        out[:lead] = 3.0
    ref, mag = _direct(direction, counts, a[lead:], b[lead:] if direction == "wgrad" else b,
                       out if direction == "wgrad" else out[lead:], False)
    ws = _run(direction, a, b, off, out)
    assert sgl.moe_linear_read_error(ws) == 0
    got = out if direction == "wgrad" else out[lead:]
    _check_product(got, ref, mag, 200, torch.ones_like(got, dtype=torch.bool))
    assert direction == "wgrad" or (out[:lead] == 3.0).all()


@pytest.mark.parametrize("direction", DIRECTIONS)
def test_no_rows_at_all(direction):
    counts, N, K = [0, 0, 0], 16, 24
    for spare in (0, 5):
        _check(direction, counts, N, K, spare=spare)
        _check(direction, counts, N, K, spare=spare, out=F32, accumulate=True)


def test_wgrad_keeps_non_finite_rows_to_their_expert():
    # expert 1's rows hold inf and NaN; its neighbours share its 64-row blocks
    counts, N, K = [37, 5, 90, 1], 136, 72
    for pos, val in ((0, float("inf")), (4, float("nan")), (2, float("-inf"))):
        a, b, out = _product("wgrad", counts, N, K, seed=4)
        clean = [t.clone() for t in (a, b)]
        a[37 + pos], b[37 + pos] = val, val
        _run("wgrad", a, b, _offsets(counts), out)
        ref, mag = _direct("wgrad", counts, *clean, out, False)
        touched = torch.ones_like(out, dtype=torch.bool)
        touched[1] = False
        assert not torch.isfinite(out[1]).any()
        ref[1] = out[1].to(F64).nan_to_num(0, 0, 0)
        out[1] = out[1].nan_to_num(0, 0, 0)
        _check_product(out, ref, mag, 90, touched)


@pytest.mark.parametrize("direction", ["linear", "dgrad"])
def test_non_finite_rows_stay_rows(direction):
    counts, N, K = [37, 5, 90], 136, 72
    a, b, out = _product(direction, counts, N, K, seed=4)
    ref, mag = _direct(direction, counts, a, b, out, False)
    a[40] = float("nan")
    _run(direction, a, b, _offsets(counts), out)
    assert torch.isnan(out[40]).all()
    touched = torch.ones_like(out, dtype=torch.bool)
    touched[40] = False
    out[40], ref[40] = 0, 0
    _check_product(out, ref, mag, max(N, K), touched)


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("offsets", [[0, 5, 3, 9, 12], [-4, 2, 6, 8, 12], [0, 4, 8, 12, 40],
                                     [50, 60, 70, 80, 90], [0, 2 ** 31 - 1, 4, 8, 12]])
def test_bad_offsets_are_reported_and_stay_inside(direction, offsets):
    """Offsets out of order or outside the rows: the error word, and no
    access outside the buffers (their neighbours keep their values)."""
    N, K, R = 72, 136, 12
    a, b, out = _product(direction, [3, 3, 3, 3], N, K, seed=2)
    guard = torch.full((3, out.numel()), 5.0, dtype=BF, device="cuda")
    guard[1] = out.reshape(-1)
    ws = _run(direction, a, b, torch.tensor(offsets, dtype=torch.int32).cuda(), guard[1].view(out.shape))
    assert sgl.moe_linear_read_error(ws) == 4
    assert sgl.moe_linear_read_error(ws) == 0
    assert (guard[0] == 5).all() and (guard[2] == 5).all()


@pytest.mark.parametrize("direction", DIRECTIONS)
@pytest.mark.parametrize("counts,N,K", [([3, 0, 1, 4], 768, 2560), ([200, 0, 300, 13], 264, 136)], ids=["few", "many"])
def test_same_bits_streams_and_graphs(direction, counts, N, K):
    """The same bits again, on another stream, and from two captured graphs
    that share a workspace and run at the same time."""
    a, b, out = _product(direction, counts, N, K, seed=8)
    off = _offsets(counts)
    ws = _run(direction, a, b, off, out)
    torch.cuda.synchronize()
    outs, graphs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = torch.zeros_like(out)
        _run(direction, a, b, off, o, ws=ws)
    outs.append(o)
    side.synchronize()
    o = torch.zeros_like(out)
    torch.cuda.synchronize()
    _run(direction, a, b, off, o, ws=ws, stream=side)
    outs.append(o)
    for _ in range(2):
        o = torch.zeros_like(out)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _run(direction, a, b, off, o, ws=ws)
        outs.append(o)
        graphs.append(gr)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert sgl.moe_linear_read_error(ws) == 0
    for o in outs:
        assert torch.equal(o, out)


@pytest.mark.parametrize("direction", DIRECTIONS)
def test_fp32_passes_add_in_order(direction):
    """Depths of several passes, overwriting and accumulating: the same bits
    every time, while another product keeps the GPU busy on another stream."""
    counts, N, K = [0, 2500, 3, 900], (264 if direction == "wgrad" else 2000), (2600 if direction == "linear" else 520)
    a, b, out = _product(direction, counts, N, K, out=F32, seed=8)
    off, base = _offsets(counts), out.clone()
    ref, mag = _direct(direction, counts, a, b, out, True)
    ws = _run(direction, a, b, off, out, True)
    depth = {"linear": K, "dgrad": N, "wgrad": 2500}[direction]
    touched = torch.ones_like(out, dtype=torch.bool)
    if direction == "wgrad":
        touched[0] = False
    _check_product(out, ref, mag, depth, touched, True)
    # the truncation of the tensor core's own sums is bounded by the passes, not by the depth
    err = float((out.to(F64) - ref)[touched].norm() / ref[touched].norm())
    assert err <= 768 / 16 * 2.0 ** -24, err
    side, other = torch.cuda.Stream(), torch.zeros_like(out)
    for _ in range(3):
        again = base.clone()
        torch.cuda.synchronize()
        _run(direction, a, b, off, other, ws=ws, stream=side)
        _run(direction, a, b, off, again, True, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(again, out)


def test_addresses_past_32_bits():
    """Row strides that put the last rows more than 2^31 elements from the first."""
    R, ld, N, K = 70001, 32768, 16, 24
    g = _gen(5)
    big = [torch.empty(R * ld, dtype=BF, device="cuda").view(R, ld) for _ in range(2)]
    x, y = big[0][:, :K], big[1][:, :N]
    x.copy_(_randn((R, K), g))
    W, off = _randn((2, N, K), g), _offsets([R - 300, 300])
    for direction, a, o in (("linear", x, y), ("dgrad", y, x)):
        a_in = a.clone()
        _run(direction, a, W, off, o)
        ref, mag = _direct(direction, [R - 300, 300], a_in, W, o.clone(), False)
        _check_product(o.contiguous(), ref, mag, 24, torch.ones_like(ref, dtype=torch.bool))
    dW = torch.empty(2, N, K, device="cuda")
    _run("wgrad", y, x, off, dW)
    ref, mag = _direct("wgrad", [R - 300, 300], y.contiguous(), x.contiguous(), dW, False)
    _check_product(dW, ref, mag, R, torch.ones_like(dW, dtype=torch.bool))
    h = big[1][:, 8:8 + K]
    sgl.moe_swiglu(x, x, h)
    ref = _swiglu_ref(x, x, 0.0, 1.0)
    assert ((h.to(F64) - ref).abs() <= (2.0 ** -8 + 2 * FAST) * ref.abs() + 1e-30).all()


def test_graph_follows_new_offsets():
    """A captured product reads the offsets when it runs: another split of the
    rows needs no new capture."""
    N, K, R = 264, 136, 400
    a, b, _ = _product("linear", [100] * 4, N, K, seed=8)
    off = _offsets([100] * 4)
    out = torch.zeros(R, N, dtype=BF, device="cuda")
    ws = _run("linear", a, b, off, out)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _run("linear", a, b, off, out, ws=ws)
    for counts in ([400, 0, 0, 0], [0, 1, 0, 399], [130, 2, 3, 100]):
        off.copy_(_offsets(counts))
        out.fill_(7.0)
        ref, mag = _direct("linear", counts, a, b, out, False)
        gr.replay()
        touched = torch.ones_like(out, dtype=torch.bool)
        touched[sum(counts):] = False
        _check_product(out, ref, mag, K, touched)


# ------------------------------------------------------------------ SwiGLU
def _swiglu_ref(g, u, limit, w, dh=None):
    """float64: h and, with dh, (dg, du, dw) and the magnitudes they are made of."""
    lim = limit if limit > 0 else math.inf
    g, u = g.to(F64), u.to(F64)
    a, b = g.clamp(-lim, lim), u.clamp(-lim, lim)
    s = torch.sigmoid(a)
    if dh is None:
        return w * a * s * b
    dh = dh.to(F64)
    dg = torch.where(g.abs() <= lim, w * dh * b * s * (1 + a * (1 - s)), torch.zeros_like(a))
    du = torch.where(u.abs() <= lim, w * dh * a * s, torch.zeros_like(a))
    mag = (w * dh * b).abs() * (s + (a * s).abs())
    return dg, du, dh * a * s * b, mag


# e^-a, the reciprocal and a handful of products: below 2^-18 relative for |a| <= 16
# (the argument's rounding alone costs |a| 2^-24), on every term of a sum
FAST = 2.0 ** -18


@pytest.mark.parametrize("limit", [0.0, 4.0, math.inf])
@pytest.mark.parametrize("R,I,spare,pad,weighted", [(1, 8, 0, 0, "perm"), (7, 768, 3, 0, "perm"),
                                                     (33, 136, 0, 16, "rows"), (300, 64, 11, 8, "none"),
                                                     (5, 4104, 1, 0, "perm"), (1000, 2048, 24, 0, "perm")])
def test_swiglu_and_gradients(limit, R, I, spare, pad, weighted):
    gen = _gen(R + I)
    cap = R + spare
    buf = _randn((cap, 2 * I + pad), gen, scale=2.5).clamp_(-16, 16)
    g, u = buf[:, :I], buf[:, I:2 * I]
    g[0, 0], u[0, 1] = 4.0, -4.0                       # on the limit: the gradient passes
    dh = _randn((cap, I + pad), gen)[:, :I]
    w = perm = dw = None
    wr = torch.ones(R, 1, dtype=F64, device="cuda")
    slots = torch.arange(R, device="cuda")
    if weighted != "none":
        w = torch.rand(cap + 5, generator=gen, device="cuda")
        dw = torch.full_like(w, 9.0)
        if weighted == "perm":
            perm = torch.randperm(cap + 5, generator=gen, device="cuda")[:cap].to(torch.int32)
            slots = perm[:R].long()
        wr = w.to(F64)[slots][:, None]
    rows = torch.tensor([R], dtype=torch.int32, device="cuda") if spare else None
    h = torch.full((cap, I + pad), 3.0, dtype=BF, device="cuda")[:, :I]
    dbuf = torch.full((cap, 2 * I + pad), 3.0, dtype=BF, device="cuda")
    dg, du = dbuf[:, :I], dbuf[:, I:2 * I]
    sgl.moe_swiglu(g, u, h, limit, w=w, perm=perm, rows=rows)
    sgl.moe_swiglu_backward(dh, g, u, dg, du, limit, w=w, perm=perm, dw=dw, rows=rows)
    ref = _swiglu_ref(g[:R], u[:R], limit, wr)
    assert ((h[:R].to(F64) - ref).abs() <= (2.0 ** -8 + 2 * FAST) * ref.abs()).all()
    rg, ru, rw, mag = _swiglu_ref(g[:R], u[:R], limit, wr, dh[:R])
    assert ((dg[:R].to(F64) - rg).abs() <= 2.0 ** -8 * (rg.abs() + 2 * FAST * mag) + 2 * FAST * mag).all()
    assert ((du[:R].to(F64) - ru).abs() <= (2.0 ** -8 + 2 * FAST) * ru.abs()).all()
    if dw is not None:
        got, want, terms = dw[slots].to(F64), rw.sum(1), rw.abs().sum(1)
        assert ((got - want).abs() <= (FAST + I * 2.0 ** -24) * terms).all()
        rest = torch.ones_like(dw, dtype=torch.bool)
        rest[slots] = False
        assert (dw[rest] == 9.0).all()
    for t in (h, dg, du):
        assert (t[R:] == 3.0).all()
    assert pad == 0 or (dbuf[:, 2 * I:] == 3.0).all()


def test_swiglu_gradient_against_differences():
    """The kernel's gradients against differences of the float64 forward: for
    a direction d, <grad, d> equals (f(x + t d) - f(x - t d)) / 2t up to
    O(t^2) and the bf16 rounding of each gradient entry."""
    gen = _gen(1)
    R, I, limit = 40, 72, 3.0
    g, u, dh = (_randn((R, I), gen, scale=1.5) for _ in range(3))
    for t in (g, u):  # keep t * d from crossing the limit
        near = (t.abs().float() - limit).abs() < 0.05
        t[near] = 1.0
    w = torch.rand(R, generator=gen, device="cuda") + 0.1
    dg, du, dw = torch.empty_like(g), torch.empty_like(g), torch.empty_like(w)
    sgl.moe_swiglu_backward(dh, g, u, dg, du, limit, w=w, dw=dw)
    t = 1e-4
    for seed in range(3):
        dir_g, dir_u = (torch.randn((R, I), generator=_gen(10 + seed + 50 * k), device="cuda", dtype=F64) for k in (0, 1))
        dir_w = torch.randn(R, generator=_gen(90 + seed), device="cuda", dtype=F64)

        def f(k):
            h = _swiglu_ref(g.to(F64) + k * dir_g, u.to(F64) + k * dir_u, limit, (w.to(F64) + k * dir_w)[:, None])
            return (h * dh.to(F64)).sum()

        diff = (f(t) - f(-t)) / (2 * t)
        parts = [dg.to(F64) * dir_g, du.to(F64) * dir_u, dw.to(F64) * dir_w]
        got = sum(p.sum() for p in parts)
        # independent roundings of the entries: 2^-8 each, here bounded by their sum in quadrature times 6
        tol = 6 * 2.0 ** -8 * math.sqrt(sum(float((p * p).sum()) for p in parts[:2])) + 1e-4 * abs(float(diff))
        assert abs(float(got - diff)) <= tol


def test_swiglu_in_place_nan_and_limits():
    gen = _gen(2)
    g, u = _randn((9, 64), gen), _randn((9, 64), gen)
    g[2, 3], u[4, 5] = float("nan"), float("nan")
    g[5, 6], g[5, 7], u[5, 8] = float("inf"), float("-inf"), float("inf")
    ref = _swiglu_ref(g, u, 4.0, 1.0)
    h = g.clone()
    sgl.moe_swiglu(h, u, h, 4.0)                       # h over g
    assert torch.isnan(h[2, 3]) and torch.isnan(h[4, 5])
    ok = ~torch.isnan(ref)
    assert torch.isfinite(h[ok]).all()
    assert ((h.to(F64) - ref).abs()[ok] <= (2.0 ** -8 + 2 * FAST) * ref.abs()[ok]).all()
    dh = _randn((9, 64), gen)
    rg, ru, _, mag = _swiglu_ref(g, u, 4.0, 1.0, dh)
    dg, du = g.clone(), u.clone()
    sgl.moe_swiglu_backward(dh, dg, du, dg, du, 4.0)   # gradients over g and u
    assert float(dg[5, 6]) == 0 and float(dg[5, 7]) == 0 and float(du[5, 8]) == 0
    ok = ~torch.isnan(mag)
    assert ((dg.to(F64) - rg).abs()[ok] <= 2.0 ** -8 * (rg.abs() + 2 * FAST * mag)[ok] + 2 * FAST * mag[ok]).all()


def test_swiglu_perm_outside_w_and_odd_row_counts():
    gen = _gen(3)
    g, u = _randn((6, 16), gen), _randn((6, 16), gen)
    w = torch.rand(4, generator=gen, device="cuda")
    perm = torch.tensor([0, 4, -1, 3, 2 ** 31 - 1, 1], dtype=torch.int32, device="cuda")
    guard = torch.full((12,), 9.0, device="cuda")
    dw = guard[4:8]
    h, dg, du = (torch.empty_like(g) for _ in range(3))
    sgl.moe_swiglu(g, u, h, w=w, perm=perm)
    sgl.moe_swiglu_backward(g, g, u, dg, du, w=w, perm=perm, dw=dw)
    bad = torch.tensor([False, True, True, False, True, False], device="cuda")
    for t in (h, dg, du):
        assert torch.isnan(t[bad]).all() and torch.isfinite(t[~bad]).all()
    assert (guard[:4] == 9).all() and (guard[8:] == 9).all() and float(dw[2]) == 9.0
    for n, live in ((-3, 0), (0, 0), (2, 2), (99, 6)):
        h.fill_(3.0)
        sgl.moe_swiglu(g, u, h, rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert (h[live:] == 3.0).all() and (live == 0 or (h[:live] != 3.0).any())


# ------------------------------------------------------------------ AdamW
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=7)


def _adam_tensor(n, gen, p=BF, g=BF, q8=False, master=False, wd=1.0):
    t = dict(p=_randn(n, gen, F32), g=_randn(n, gen, g, 1e-3), wd_scale=wd)
    if master:
        t["master"] = t["p"].clone()
    t["p"] = t["p"].to(p)
    if not q8:
        t["m"], t["v"] = _randn(n, gen, F32, 3e-4), torch.rand(n, generator=gen, device="cuda") * 1e-6
    else:
        b = -(-n // 256)
        t["m"] = (torch.randn(n, generator=gen, device="cuda") * 80).clamp_(-448, 448).to(F8)
        t["v"] = (torch.rand(n, generator=gen, device="cuda") * 448).to(F8)
        t["m_scale"] = torch.rand(b, generator=gen, device="cuda") * 1e-5
        t["v_scale"] = torch.rand(b, generator=gen, device="cuda") * 1e-5
    return t


def _per_element(scale, n):
    return scale.to(F64).repeat_interleave(256)[:n]


def _moments(t):
    n = t["p"].numel()
    if "m_scale" not in t:
        return t["m"].to(F64), t["v"].to(F64)
    return (t["m"].to(F64) * _per_element(t["m_scale"], n),
            (t["v"].to(F64) * _per_element(t["v_scale"], n)) ** 2)


def _check_adam(before, after, h, gs=1.0):
    """after against the float64 step of before. fp32 steps with rounded
    coefficients cost at most 6 roundings of 2^-24 for m and v; the update
    adds a square root, a reciprocal product and a fast division: below
    2^-19 of its magnitude."""
    n = before["p"].numel()
    m0, v0 = _moments(before)
    g = before["g"].to(F64) * gs
    p0 = before.get("master", before["p"]).to(F64)
    m = h["beta1"] * m0 + (1 - h["beta1"]) * g
    m_mag = h["beta1"] * m0.abs() + (1 - h["beta1"]) * g.abs()
    v = h["beta2"] * v0 + (1 - h["beta2"]) * g * g
    den = (v / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"]
    lr1 = h["lr"] / (1 - h["beta1"] ** h["step"])
    p = p0 * (1 - h["lr"] * h["weight_decay"] * before["wd_scale"]) - lr1 * m / den
    tol = 4 * 2.0 ** -24 * p0.abs() + 2.0 ** -19 * lr1 * m_mag / den
    if "master" in before:
        assert ((after["master"].to(F64) - p).abs() <= tol).all()
        assert torch.equal(after["p"], after["master"].to(BF))
    half = 2.0 ** -8 if after["p"].dtype == BF else 0.0
    assert ((after["p"].to(F64) - p).abs() <= tol + half * (p.abs() + tol)).all()
    if "m_scale" not in before:
        assert ((after["m"].to(F64) - m).abs() <= 6 * 2.0 ** -24 * m_mag).all()
        assert ((after["v"].to(F64) - v).abs() <= 8 * 2.0 ** -24 * v).all()
        return
    for key, x, mag, least in (("m", m, m_mag, 2.0 ** -10), ("v", v.sqrt(), v.sqrt(), 2.0 ** -9)):
        pad = torch.zeros(-(-n // 256) * 256, dtype=F64, device="cuda")
        pad[:n] = x.abs()
        top = pad.view(-1, 256).amax(1)
        want = torch.where(top < 2.0 ** -100, 0.0, top / 448)
        pad[:n] = mag
        assert ((after[key + "_scale"].to(F64) - want).abs() <= 8 * 2.0 ** -24 * pad.view(-1, 256).amax(1) / 448 * 2).all()
        s = _per_element(after[key + "_scale"], n)
        got = after[key].to(F64) * s
        # half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6), after fp32 roundings
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() * (1 + 2.0 ** -18) + least * s * (1 + 2.0 ** -18) + 2.0 ** -20 * mag).all()
        if key == "v":
            assert ((after["v"].to(F64) > 0) | (x == 0) | (s == 0)).all()


def _step(ts, **kw):
    before = [{k: (v.clone() if torch.is_tensor(v) else v) for k, v in t.items()} for t in ts]
    sgl.moe_adamw_step(sgl.make_adamw_tensors(ts), **{**HYPER, **kw})
    torch.cuda.synchronize()
    return before


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("p,master", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("g", [BF, F32])
def test_adamw(q8, p, master, g):
    gen = _gen(1)
    ts = [_adam_tensor(n, gen, p, g, q8, master, wd) for n, wd in
          ((1, 1.0), (7, 0.0), (8, 1.0), (255, 2.0), (256, 1.0), (257, 1.0), (2049, 0.0), (100003, 1.0))]
    for t, b in zip(ts, _step(ts)):
        _check_adam(b, t, HYPER)


def test_adamw_many_tensors_of_every_kind():
    """More tensors than one launch takes, empty ones among them, kinds mixed."""
    gen = _gen(2)
    kinds = [dict(p=p, g=g, q8=q, master=m) for p, m in ((BF, False), (BF, True), (F32, False)) for g in (BF, F32)
             for q in (False, True)]
    ts = [_adam_tensor((i * 37) % 700, gen, wd=float(i % 2), **kinds[i % len(kinds)]) for i in range(700)]
    assert any(t["p"].numel() == 0 for t in ts)
    for i, (t, b) in enumerate(zip(ts, _step(ts, grad_scale=0.5))):
        if t["p"].numel():
            _check_adam(b, t, HYPER, 0.5)


def test_adamw_neighbours_keep_their_values():
    """Views into larger buffers: nothing outside a tensor is written."""
    gen = _gen(3)
    for q8 in (False, True):
        t = _adam_tensor(300, gen, q8=q8)
        bufs = {}
        for k, v in list(t.items()):
            if torch.is_tensor(v):
                pad = 4 if k.endswith("_scale") else 32
                bufs[k] = torch.full((v.numel() + 2 * pad,), 1.0, device="cuda").to(v.dtype)
                bufs[k][pad:pad + v.numel()] = v
                t[k] = bufs[k][pad:pad + v.numel()]
        b = _step([t])[0]
        _check_adam(b, t, HYPER)
        for k, buf in bufs.items():
            pad = 4 if k.endswith("_scale") else 32
            assert (buf[:pad].float() == 1).all() and (buf[-pad:].float() == 1).all(), k


@pytest.mark.parametrize("q8", [False, True])
def test_adamw_past_32_bits(q8):
    """A tensor of more than 2^31 elements: its end moves as the same values do alone."""
    n, tail = 2 ** 31 + 700, 4096 + 700 % 256
    gen = _gen(8)
    small = _adam_tensor(tail, gen, BF, BF, q8)
    lo = n - tail
    assert lo % 256 == 0
    t = {}
    for k, x in small.items():
        if torch.is_tensor(x):
            scale = k.endswith("_scale")
            t[k] = torch.zeros(-(-n // 256) if scale else n, dtype=x.dtype, device="cuda")
            t[k].view(torch.uint8)[-x.numel() * x.element_size():] = x.view(torch.uint8)
    _step([t])
    _step([small])
    for k, x in small.items():
        if torch.is_tensor(x):
            assert torch.equal(t[k].view(torch.uint8)[-x.numel() * x.element_size():], x.view(torch.uint8)), k
    assert not t["p"][:lo:4097].any()


def test_adamw_zero_tiny_and_non_finite_blocks():
    gen = _gen(4)
    t = _adam_tensor(4 * 256, gen, F32, F32, True)
    for k in ("m", "v"):
        t[k].zero_()
    t["g"].zero_()
    t["g"][256:512] = 1e-33                     # below 2^-100 after (1 - beta1): the block's m is zero
    t["g"][512] = 1.0                           # a block whose other entries are 2^-30 of the largest
    t["g"][513:768] = 2.0 ** -30
    t["g"][800] = float("inf")
    p0 = t["p"].clone()
    _step([t], weight_decay=0.0)
    v = t["v"].to(F32)
    assert torch.equal(t["p"][:256], p0[:256]) and (t["m_scale"][:2] == 0).all() and float(t["v_scale"][0]) == 0
    assert (v[513:768] == 2.0 ** -9).all() and float(v[512]) == 448      # never rounded to zero
    assert torch.isfinite(t["p"][:768]).all()
    assert torch.isnan(t["m_scale"][3]) and torch.isnan(t["v_scale"][3])
    assert torch.isfinite(t["p"][768:800]).all() and torch.isnan(t["p"][800])
    u = _adam_tensor(512, gen, BF, BF)
    u["g"][3] = float("nan")
    _step([u])
    for k in ("p", "m", "v"):
        assert torch.isnan(u[k][3].float()) and torch.isfinite(torch.cat([u[k][:3], u[k][4:]]).float()).all()


def test_adamw_codes_follow_the_formula_bit_for_bit():
    """8-bit states: codes and scales equal those of the formula with every
    fp32 operation rounded by itself (what eager elementwise operations do),
    also at the borders between two codes; two million values a step meet
    some within an ulp or two of a border."""
    gen = _gen(7)
    n = 2_000_000 + 77
    pad = -(-n // 256) * 256
    for p, g in ((BF, BF), (F32, F32)):
        t = _adam_tensor(n, gen, p, g, True)
        h = sgl.make_adamw_tensors([t])

        def decode(q, s):
            full = torch.zeros(pad, device="cuda")
            full[:n] = q.to(F32)
            return full.view(-1, 256) * s[:, None]

        for step in (1, 2, 3):
            t["g"].copy_(_randn(n, gen, F32, 1e-3))
            grad = torch.zeros(pad, device="cuda")
            grad[:n] = t["g"].to(F32)
            m, v = decode(t["m"], t["m_scale"]), decode(t["v"], t["v_scale"])
            grad = grad.view(-1, 256)
            m = 0.9 * m + (1 - 0.9) * grad
            v = 0.95 * (v * v) + (1 - 0.95) * (grad * grad)
            sgl.moe_adamw_step(h, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=step)
            for key, x in (("m", m), ("v", v.sqrt())):
                top = x.abs().amax(1, keepdim=True)
                code = (x * (top.reciprocal() * 448)).to(F8)
                if key == "v":
                    code = torch.where((x > 0) & (code.to(F32) == 0), 2.0 ** -9, code.to(F32)).to(F8)
                assert torch.equal(t[key].view(torch.uint8), code.view(-1)[:n].view(torch.uint8)), (key, step)
                assert torch.equal(t[key + "_scale"], (top * torch.tensor(1.0 / 448, device="cuda")).view(-1)), (key, step)


def test_adamw_update_against_the_definition_over_steps():
    """Twenty steps with fp32 states follow a float64 AdamW of the same
    gradients: errors of 2^-19 of each update add up at most."""
    gen = _gen(5)
    n = 5000
    t = dict(p=_randn(n, gen, F32), g=torch.zeros(n, device="cuda"), m=torch.zeros(n, device="cuda"),
             v=torch.zeros(n, device="cuda"))
    h = sgl.make_adamw_tensors([t])
    p = t["p"].to(F64)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    for k in range(1, 21):
        t["g"].copy_(_randn(n, gen, F32))
        g = t["g"].to(F64)
        sgl.moe_adamw_step(h, lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=k)
        m, v = 0.9 * m + 0.1 * g, 0.99 * v + 0.01 * g * g
        p = p * (1 - 1e-3) - 1e-2 * (m / (1 - 0.9 ** k)) / ((v / (1 - 0.99 ** k)).sqrt() + 1e-8)
    # |m| may be far below its terms; 20 updates of at most about 4 lr each
    assert float((t["p"].to(F64) - p).abs().max()) <= 20 * (4 * 1e-2 * 2.0 ** -16 + 4 * 2.0 ** -24 * 5)


def test_adamw_graph_follows_the_schedule():
    """A captured step reads lr, bias corrections and gradient scale from
    `dyn` when it runs; each replay equals an eager step with host values."""
    gen = _gen(6)
    for q8 in (False, True):
        t = _adam_tensor(3000, gen, q8=q8, master=True)
        e = {k: (x.clone() if torch.is_tensor(x) else x) for k, x in t.items()}
        dyn = torch.zeros(4, device="cuda")
        h, he = sgl.make_adamw_tensors([t]), sgl.make_adamw_tensors([e])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sgl.moe_adamw_step(h, beta1=0.9, beta2=0.95, weight_decay=0.1, dyn=dyn)
        for k in (1, 2, 3):
            dyn.copy_(torch.tensor(sgl.adamw_dyn(1e-3 * k, 0.9, 0.95, k, 1.0 / k)))
            gr.replay()
            sgl.moe_adamw_step(he, lr=1e-3 * k, beta1=0.9, beta2=0.95, weight_decay=0.1, step=k, grad_scale=1.0 / k)
        torch.cuda.synchronize()
        for k, x in t.items():
            assert not torch.is_tensor(x) or torch.equal(x.view(torch.uint8), e[k].view(torch.uint8)), k


# ------------------------------------------------------------------ together
def test_expert_layer_forward_backward_and_step():
    """Routing, permutation, the experts from the separate operators, their
    gradients and an AdamW step, as a training step runs them: against the
    fused forward, float64 autograd and differences; then the fused forward
    on the updated weights."""
    import workloads
    from tests.helpers import run_staged, weights
    cfg = workloads.CONFIGS["tiny"].with_(T=150, limit_routed=3.0)
    d = workloads.generate(cfg, "cuda:0")
    T, E, K, H, I = cfg.T, cfg.E, cfg.K, cfg.H, cfg.I
    R = T * K
    ws = sgl.alloc_workspace(cfg, T)
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    sgl.moe_route(cfg, d["x"], d["Wr"], d["bias"], idx, w, ws)

    def experts_forward():
        st = run_staged(cfg, d, idx, w)
        offsets, perm = st["offsets"], st["perm"]
        x = d["x"][(perm // K).long()]
        lws = sgl.alloc_linear_workspace(E, R, I, H)
        gu = torch.empty(R, 2 * I, dtype=BF, device="cuda")
        g, u = gu[:, :I], gu[:, I:]
        h = torch.empty(R, I, dtype=BF, device="cuda")
        y = torch.empty(R, H, device="cuda")
        sgl.moe_grouped_linear(x, offsets, d["Wg"], g, lws)
        sgl.moe_grouped_linear(x, offsets, d["Wu"], u, lws)
        sgl.moe_swiglu(g, u, h, cfg.limit_routed, w=w.view(-1), perm=perm, rows=offsets[E:])
        sgl.moe_grouped_linear(h, offsets, d["Wd"], y, lws)
        assert sgl.moe_linear_read_error(lws) == 0
        # the fused forward keeps gate and up in fp32 and weighs the output: they differ by
        # the rounding of g, u and the weighted h (2^-8 each) on the way
        fused = st["y_slot"][perm.long()]
        assert float((y - fused).norm() / fused.norm()) <= 4 * 2.0 ** -8
        return x, offsets, perm, lws, g, u, h, y

    x, offsets, perm, lws, g, u, h, y = experts_forward()
    dy = _randn((R, H), _gen(3), BF)
    dh, dx = torch.empty_like(h), torch.empty(R, H, device="cuda")
    dgu = torch.empty(R, 2 * I, dtype=BF, device="cuda")
    dg, du = dgu[:, :I], dgu[:, I:]
    dw = torch.empty(R, device="cuda")
    dW = {k: torch.empty(d[k].shape, device="cuda") for k in ("Wg", "Wu", "Wd")}
    sgl.moe_grouped_linear_dgrad(dy, offsets, d["Wd"], dh, lws)
    sgl.moe_grouped_linear_wgrad(dy, h, offsets, dW["Wd"], lws)
    sgl.moe_swiglu_backward(dh, g, u, dg, du, cfg.limit_routed, w=w.view(-1), perm=perm, dw=dw, rows=offsets[E:])
    sgl.moe_grouped_linear_dgrad(dg, offsets, d["Wg"], dx, lws)
    sgl.moe_grouped_linear_dgrad(du, offsets, d["Wu"], dx, lws, accumulate=True)
    sgl.moe_grouped_linear_wgrad(dg, x, offsets, dW["Wg"], lws)
    sgl.moe_grouped_linear_wgrad(du, x, offsets, dW["Wu"], lws)
    assert sgl.moe_linear_read_error(lws) == 0

    ref = {k: d[k].to(F64).requires_grad_() for k in ("Wg", "Wu", "Wd")}
    xr, wr = x.to(F64).requires_grad_(), w.view(-1).to(F64).requires_grad_()
    e_of = torch.bucketize(torch.arange(R, device="cuda"), offsets[1:].long(), right=True)

    def loss(W, xx, ww):
        lim = cfg.limit_routed
        gg = torch.einsum("rk,rnk->rn", xx, W["Wg"][e_of]).clamp(-lim, lim)
        uu = torch.einsum("rk,rnk->rn", xx, W["Wu"][e_of]).clamp(-lim, lim)
        hh = ww[perm.long()][:, None] * torch.nn.functional.silu(gg) * uu
        return (torch.einsum("rn,rkn->rk", hh, W["Wd"][e_of]) * dy.to(F64)).sum()

    loss(ref, xr, wr).backward()
    # at most six bf16 roundings lie on a path (g, u, h, dh, dg or du), each 2^-8 of its
    # tensor's norm at most, passed on by SwiGLU with slopes up to about 1.1 times the weight
    for name, got, want in ([(k, dW[k], ref[k].grad) for k in dW] + [("x", dx, xr.grad), ("w", dw, wr.grad)]):
        err = float((got.to(F64) - want).norm() / want.norm())
        assert err <= 6 * 1.1 * 2.0 ** -8, (name, err)
    # and against differences of the loss along a direction in every weight
    with torch.no_grad():
        dirs = {k: torch.randn(d[k].shape, generator=_gen(11), device="cuda", dtype=F64) * 0.01 for k in dW}
        t = 1e-3
        f = [loss({k: ref[k] + s * t * dirs[k] for k in dW}, xr, wr) for s in (1, -1)]
        diff = float(f[0] - f[1]) / (2 * t)
        got = sum(float((dW[k].to(F64) * dirs[k]).sum()) for k in dW)
        scale = math.sqrt(sum(float(ref[k].grad.norm()) ** 2 * 0.01 ** 2 for k in dW))
        assert abs(got - diff) <= 6 * (6 * 1.1 * 2.0 ** -8) * scale + 0.02 * abs(diff)

    before = {k: d[k].clone() for k in dW}
    tensors = [dict(p=d[k], g=dW[k], m=torch.zeros(d[k].shape, device="cuda", dtype=F8),
                    v=torch.zeros(d[k].shape, device="cuda", dtype=F8),
                    m_scale=torch.zeros(-(-d[k].numel() // 256), device="cuda"),
                    v_scale=torch.zeros(-(-d[k].numel() // 256), device="cuda")) for k in dW]
    sgl.moe_adamw_step(sgl.make_adamw_tensors(tensors), lr=1e-2, weight_decay=0.1, step=1)
    for k in dW:  # first step: each weight with a gradient moves by lr against its sign, then decays
        moved = d[k].to(F64) - before[k].to(F64) * (1 - 1e-3)
        clear = dW[k].abs() > 1e-5
        want = -1e-2 * dW[k].sign().to(F64)
        tol = 2.0 ** -8 * (before[k].to(F64).abs() + 1e-2) + 1e-2 * 1e-3 + 1e-5
        assert ((moved - want).abs() <= tol)[clear].all()
        idle = (offsets[1:] == offsets[:-1]).nonzero()[:, 0]
        assert (dW[k][idle] == 0).all()
    experts_forward()
    assert weights(d) is not None
