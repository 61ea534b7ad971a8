"""The training operators at the ends of their ranges: gradient scales far
from one, long contractions."""
import pytest
import torch

import sigmoid_group_limited_b200 as sgl
from tests.test_gpu_training import BF, F32, F64, HYPER, _adam_tensor, _check_adam, _gen, _offsets, _run, _step

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
