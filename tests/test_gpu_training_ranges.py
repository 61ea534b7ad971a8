"""The training operators at the ends of their ranges: gradient scales far
from one."""
import pytest
import torch

import sigmoid_group_limited_b200 as sgl
from tests.test_gpu_training import BF, F32, HYPER, _adam_tensor, _check_adam, _gen, _step

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
