"""The training operators at the ends of their ranges: gradient scales far
from one, second moments below the normal numbers, gates far below zero, long
contractions, large weights, forked captures, waits that give up."""
import time

import pytest
import torch

import sigmoid_group_limited_b200 as sgl
from tests.test_gpu_training import (BF, F8, F32, F64, HYPER, _adam_tensor, _check, _check_adam, _check_product, _direct,
                                     _gen, _offsets, _product, _randn, _run, _step)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ AdamW
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("g", [BF, F32])
@pytest.mark.parametrize("power", [66, -73])
@pytest.mark.parametrize("dyn", [False, True])
def test_adamw_scales_the_gradient_before_it_squares_it(q8, g, power, dyn):
    """Gradients whose square fp32 cannot hold, under a scale whose square it
    cannot hold either: the scaled gradient is around one."""
    gen = _gen(11)
    t = _adam_tensor(5000, gen, BF, g, q8, True)
    t["g"] = (torch.randn(5000, generator=gen, device="cuda") * 2.0 ** power).to(g)
    gs = 2.0 ** -power                                   # exact: one rounding less than the tolerance counts
    kw = dict(grad_scale=gs)
    if dyn:
        v = sgl.adamw_dyn(HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["step"], gs)
        kw = dict(dyn=torch.tensor(v, device="cuda"))
    before = _step([t], **kw)[0]
    assert torch.isfinite(t["v"].float()).all() and torch.isfinite(t["p"].float()).all()
    _check_adam(before, t, HYPER, gs)


@pytest.mark.parametrize("q8", [False, True])
def test_adamw_second_moments_below_the_normal_numbers(q8):
    """v' between 2^-130 and 2^-126 and no eps: the update is m over its root,
    not over zero. There v holds 19 bits or more, so its two or three
    roundings are 2^-19 of it at most, the root's 2^-20 each."""
    gen = _gen(12)
    n, beta1, beta2, lr, step = 2048, 0.9, 0.95, 1e-3, 5
    root = torch.exp2(torch.rand(n, generator=gen, device="cuda", dtype=F64) * 2 - 65)   # 2^-65 .. 2^-63
    t = dict(p=_randn(n, gen, F32), g=torch.zeros(n, device="cuda"))
    if q8:
        top = 2.0 ** -63 / 448
        t["v"] = (root / 2.0 ** -63 * 448).to(F8)
        t["m"] = (torch.rand(n, generator=gen, device="cuda") * 300 + 100).to(F8)
        t["v_scale"] = torch.full((n // 256,), top, device="cuda", dtype=F64).float()
        t["m_scale"] = torch.full((n // 256,), 2.0 ** -73, device="cuda")
        m = t["m"].to(F64) * 2.0 ** -73
        v = (t["v"].to(F64) * t["v_scale"].to(F64).repeat_interleave(256)) ** 2
    else:
        t["m"] = (torch.rand(n, generator=gen, device="cuda") + 0.5) * 2.0 ** -64
        t["v"] = (root * root).float()
        m, v = t["m"].to(F64), t["v"].to(F64)
    p0 = t["p"].to(F64)
    sgl.moe_adamw_step(sgl.make_adamw_tensors([t]), lr=lr, beta1=beta1, beta2=beta2, eps=0.0, step=step)
    up = lr / (1 - beta1 ** step) * beta1 * m / (beta2 * v / (1 - beta2 ** step)).sqrt()
    assert float(up.abs().min()) > 1e-4                  # far above the rounding of p
    assert ((t["p"].to(F64) - (p0 - up)).abs() <= 2 * 2.0 ** -24 * p0.abs() + 6 * 2.0 ** -20 * up.abs()).all()


def test_adamw_codes_with_zeros_and_a_gradient_scale():
    """8-bit states where much is zero (experts without rows, the first step):
    whole blocks, single elements, zero gradients on states that are not. Codes
    and scales equal those of the formula with every fp32 operation rounded by
    itself, under a gradient scale, too."""
    gen = _gen(18)
    n = 300 * 256 + 100
    blocks = -(-n // 256)
    t = _adam_tensor(n, gen, BF, F32, True)
    for k in ("m", "v"):
        t[k].view(torch.uint8)[:100 * 256] = 0               # idle from the start
        t[k].view(torch.uint8)[torch.rand(n, generator=gen, device="cuda") < 0.5] = 0
    h = sgl.make_adamw_tensors([t])

    def rows(x):
        full = torch.zeros(blocks * 256, device="cuda")
        full[:n] = x.to(F32)
        return full.view(-1, 256)

    gs = torch.tensor(0.37, device="cuda")
    for step in (1, 2, 3):
        t["g"].copy_(_randn(n, gen, F32, 1e-3))
        t["g"][:50 * 256] = 0
        t["g"][torch.rand(n, generator=gen, device="cuda") < 0.5] = 0
        g = rows(t["g"]) * gs
        m, v = rows(t["m"]) * t["m_scale"][:, None], rows(t["v"]) * t["v_scale"][:, None]
        m = 0.9 * m + (1 - 0.9) * g
        v = 0.95 * (v * v) + (1 - 0.95) * (g * g)
        sgl.moe_adamw_step(h, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=step, grad_scale=float(gs))
        assert torch.isfinite(t["p"].float()).all()
        for key, x in (("m", m), ("v", v.sqrt())):
            top = x.abs().amax(1, keepdim=True)
            code = (x * torch.where(top > 0, top.reciprocal() * 448, 0.0)).to(F8)
            if key == "v":
                code = torch.where((x > 0) & (code.to(F32) == 0), 2.0 ** -9, code.to(F32)).to(F8)
            # a product of zero and a negative number is -0, with or without the sum's sign
            same = t[key].view(torch.uint8) == code.view(-1)[:n].view(torch.uint8)
            zero = (t[key].to(F32) == 0) & (code.view(-1)[:n].to(F32) == 0)
            assert (same | zero).all(), (key, step)
            assert torch.equal(t[key + "_scale"], (top * torch.tensor(1.0 / 448, device="cuda")).view(-1)), (key, step)


# ------------------------------------------------------------------ SwiGLU
def test_swiglu_gates_far_below_zero():
    """No limit and gates down to -100: the sigmoid is below the normal
    numbers of fp32, its product with a large up value is not. e^a costs |a|
    2^-24 for its argument and a few 2^-23, and below 2^-126 a spacing of 2^-149;
    below -103.3 the sigmoid is zero."""
    gen = _gen(13)
    R, I = 64, 264
    g = -(torch.rand(R, I, generator=gen, device="cuda") * 22 + 80).to(BF)
    g[:, :8] = torch.tensor([-200.0, -3e38, 80.0, 100.0, 3e38, 0.0, -0.0, -1e-30], device="cuda").to(BF)
    u = (_randn((R, I), gen, F32) * 2.0 ** 20).to(BF)
    dh = _randn((R, I), gen)
    w = torch.rand(R, generator=gen, device="cuda") + 0.5
    h, dg, du, dw = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g), torch.empty_like(w)
    u[:, 4] = 1.0                                        # 3e38 w: stays finite
    w[:] = w.clamp(max=1.0)
    sgl.moe_swiglu(g, u, h, w=w)
    sgl.moe_swiglu_backward(dh, g, u, dg, du, w=w, dw=dw)
    a, b, d, ww = g.to(F64), u.to(F64), dh.to(F64), w.to(F64)[:, None]
    s = torch.sigmoid(a)
    rel, low = 128 * 2.0 ** -24 + 8 * 2.0 ** -23, 2.0 ** -149
    bf = 2.0 ** -134                                     # half the spacing of bf16 below its normal numbers

    def near(got, want, terms, floor):
        tol = 2.0 ** -8 * want.abs() + rel * terms + floor + bf
        past = want.abs() > torch.finfo(BF).max * (1 + 2.0 ** -8)        # no bf16 value: infinite
        assert torch.equal(got[past].to(F64), want[past].sign() * float("inf"))
        bad = ((got.to(F64) - want).abs() > tol) & ~past
        assert not bad.any(), (a[bad][:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())

    near(h, ww * a * s * b, (ww * a * s * b).abs(), (ww * a * b).abs() * low)
    near(du, ww * d * a * s, (ww * d * a * s).abs(), (ww * d * a).abs() * low)
    t = (ww * d * b).abs()
    near(dg, ww * d * b * s * (1 + a * (1 - s)), t * s * (1 + a.abs() * (1 - s)), t * (1 + a.abs()) * low)
    # the far gates alone
    far = torch.zeros_like(g)
    far[:] = -88.0
    sgl.moe_swiglu_backward(dh, far, u, dg, du, w=w, dw=dw)
    a = far.to(F64)
    terms = d * a * torch.sigmoid(a) * b
    err = (dw.to(F64) - terms.sum(1)).abs()
    assert (err <= (rel + I * 2.0 ** -24) * terms.abs().sum(1) + (d * a * b).abs().sum(1) * low).all()


# ------------------------------------------------------------------ long contractions
def _positive(shape, gen, dtype=BF):
    return (torch.rand(shape, generator=gen, device="cuda") + 0.5).to(dtype)


def test_wgrad_bf16_of_millions_of_rows():
    """One expert with 2^22 rows (the shared expert's case), terms of one sign.
    The tensor core cuts its sums; unbroken, that takes 2.3 % off here. In passes of
    at most 2^14 rows each addition is off by one unit, 2^-23, at most, on half
    of the sum on average, and adding 257 passes rounds by 2^-24 each."""
    gen = _gen(14)
    counts, N, K = [2 ** 22 + 37, 0, 50], 16, 24
    R = sum(counts)
    dy, x = _positive((R, N), gen), _positive((R, K), gen)
    dW = torch.empty(3, N, K, dtype=BF, device="cuda")
    ws = _run("wgrad", dy, x, _offsets(counts), dW)
    assert sgl.moe_linear_read_error(ws) == 0
    assert not dW[1].any()
    for e, (lo, hi) in ((0, (0, counts[0])), (2, (counts[0], R))):
        want = sum(dy[i:min(i + 2 ** 20, hi)].to(F64).t() @ x[i:min(i + 2 ** 20, hi)].to(F64) for i in range(lo, hi, 2 ** 20))
        err = (dW[e].to(F64) - want) / want
        assert float(err.abs().max()) <= 2.0 ** -8 + 2 ** 14 * 2.0 ** -24 + 257 * 2.0 ** -24


def test_wgrad_bf16_of_long_and_short_experts_together():
    """Experts of one and of several passes, whole and ragged, and none at all,
    over enough tiles that a pair takes long and short ones in turn; the same
    bits again. A pass is at most 1024 steps, each off by at most 17 units of
    2^-23 (16 products and the sum)."""
    gen = _gen(16)
    counts, N, K = [16385, 0, 300, 16384, 33333, 7, 49153], 1032, 2568
    R = sum(counts)
    dy, x = _randn((R, N), gen), _randn((R, K), gen)
    off = _offsets(counts)
    dW = torch.empty(len(counts), N, K, dtype=BF, device="cuda")
    ws = _run("wgrad", dy, x, off, dW)
    again = torch.full_like(dW, 7.0)
    _run("wgrad", dy, x, off, again, ws=ws)
    assert sgl.moe_linear_read_error(ws) == 0
    assert torch.equal(dW, again)
    lo = 0
    for e, c in enumerate(counts):
        want = dy[lo:lo + c].to(F64).t() @ x[lo:lo + c].to(F64)
        err = (dW[e].to(F64) - want).norm(dim=1)
        assert (err <= (2.0 ** -8 + 1024 * 17 * 2.0 ** -23) * want.norm(dim=1)).all(), e
        lo += c


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("direction,N,K", [("linear", 72, 16384), ("dgrad", 16384, 72), ("wgrad", 264, 136)])
def test_fp32_results_do_not_lose_with_depth(direction, N, K, accumulate):
    """Terms of one sign, a depth of one pass (768) and of many. A sum of passes
    of one sign is off by no more than its worst pass, relative to itself, and the
    P adds cost 2^-24 each; twice the first pass's error for the spread
    between passes. One unbroken sum has an error that grows with the depth: 6e-5
    at 16384 and 1e-4 at 20011, over twenty times the bound."""
    gen = _gen(15)
    depths = (768, 20011) if direction == "wgrad" else (768, 16384)
    errs = []
    for depth in depths:
        counts = [depth, 0, depth] if direction == "wgrad" else [40, 0, 300]
        n, k = (depth if direction == "dgrad" else N), (depth if direction == "linear" else K)
        R, E = sum(counts), len(counts)
        a = _positive((R, k if direction == "linear" else n), gen)
        b = _positive((R, k) if direction == "wgrad" else (E, n, k), gen)
        out = torch.zeros({"linear": (R, n), "dgrad": (R, k), "wgrad": (E, n, k)}[direction], device="cuda")
        ws = _run(direction, a, b, _offsets(counts), out, accumulate)
        assert sgl.moe_linear_read_error(ws) == 0
        want, _ = _direct(direction, counts, a, b, torch.zeros_like(out), False)
        errs.append(float((out.to(F64) - want).norm() / want.norm()))
    passes = -(-depths[1] // 768)
    assert errs[1] <= 2 * errs[0] + passes * 2.0 ** -24, errs


# ------------------------------------------------------------------ addresses and graphs
def test_weights_past_32_bits():
    """More than 2^32 weights: experts on both sides of 2^31 and 2^32 elements, few and
    many rows, and the clearing of experts without rows."""
    gen = _gen(3)
    E, N, K = 300, 4096, 4096
    live = (0, 128, 256, 257, 299)
    W = torch.zeros(E, N, K, dtype=BF, device="cuda")
    for e in live:
        W[e] = _randn((N, K), gen)
    dW = torch.empty(E, N, K, dtype=BF, device="cuda")
    for per in (8, 140):
        counts = [per if e in live else 0 for e in range(E)]
        off, R = _offsets(counts), per * len(live)
        x, dy = _randn((R, K), gen), _randn((R, N), gen)
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        for direction, a, out in (("linear", x, y), ("dgrad", dy, dx)):
            ws = _run(direction, a, W, off, out)
            ref, mag = _direct(direction, counts, a, W, out, False)
            _check_product(out, ref, mag, 4096, torch.ones_like(out, dtype=torch.bool))
        dW.fill_(3.0)
        _run("wgrad", dy, x, off, dW, ws=ws)
        assert sgl.moe_linear_read_error(ws) == 0
        for e in range(E):
            if e not in live:
                assert not dW[e].any(), e
        for i, e in enumerate(live):
            want = dy[i * per:(i + 1) * per].to(F64).t() @ x[i * per:(i + 1) * per].to(F64)
            mag = dy[i * per:(i + 1) * per].to(F64).abs().t() @ x[i * per:(i + 1) * per].to(F64).abs()
            _check_product(dW[e], want, mag, per, torch.ones_like(dW[e], dtype=torch.bool))


def test_captured_on_two_streams_that_join():
    """A capture that forks after a fill and joins before the next operator: the
    operators' launches have several predecessors, some of them no kernels."""
    x, W, _ = _product("linear", [100, 200], 72, 136, seed=19)
    off = _offsets([100, 200])
    y = [torch.empty(300, 72, dtype=BF, device="cuda") for _ in range(3)]
    h, want = torch.empty_like(y[0]), torch.empty_like(y[0])
    ws = _run("linear", x, W, off, y[2])
    sgl.moe_swiglu(y[2], y[2], want)
    torch.cuda.synchronize()
    side, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        main = torch.cuda.current_stream()
        y[0].zero_()
        side.wait_stream(main)
        _run("linear", x, W, off, y[0], ws=ws)
        with torch.cuda.stream(side):
            y[1].zero_()
            _run("linear", x, W, off, y[1], ws=ws)
        main.wait_stream(side)
        sgl.moe_swiglu(y[0], y[1], h)
    for _ in range(3):
        h.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[2]) and torch.equal(h, want)


# ------------------------------------------------------------------ waits that give up
@pytest.mark.parametrize("direction,counts,N,K,out", [
    ("linear", [40, 0, 300], 264, 2560, F32), ("dgrad", [40, 0, 300], 2560, 264, F32),
    ("wgrad", [2500, 37, 0, 900], 264, 136, F32), ("wgrad", [40007, 37], 264, 136, BF)])
def test_waits_run_out_and_report(direction, counts, N, K, out, monkeypatch):
    """The accumulators are never free again (their barriers wait for an arrival
    that does not come) and the waits' limit is about 1 ms: every role gives up,
    the call returns with the error word set, and the next one is right."""
    _check(direction, counts, N, K, out=out, seed=17)
    a, b, o = _product(direction, counts, N, K, out=out, seed=17)
    off = _offsets(counts)
    ws = sgl.alloc_linear_workspace(len(counts), a.shape[0], 8, 8)
    torch.cuda.synchronize()
    monkeypatch.setenv("SGL_MOE_TEST_WAIT_CYCLES", "2000000")
    monkeypatch.setenv("SGL_MOE_TEST_READY_EXTRA", "1")
    t0 = time.perf_counter()
    _run(direction, a, b, off, o, ws=ws)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    monkeypatch.delenv("SGL_MOE_TEST_WAIT_CYCLES")
    monkeypatch.delenv("SGL_MOE_TEST_READY_EXTRA")
    assert sgl.moe_linear_read_error(ws) == 2            # MOE_DEVERR_TIMEOUT
    assert sgl.moe_linear_read_error(ws) == 0
    _check(direction, counts, N, K, out=out, seed=17)
