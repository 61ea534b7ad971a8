"""The training operators' binding at the ends of its ranges, without a GPU."""
import ctypes

import pytest
import torch

import sigmoid_group_limited_b200 as sgl

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _meta(shape, dtype=BF, stride=None):
    if stride is not None:
        return torch.empty_strided(shape, stride, dtype=dtype, device="meta")
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_31_bits_are_refused():
    """The C descriptors hold 32 bits: 2^32 + 5 rows must not become five."""
    R, ws = 2 ** 32 + 5, torch.zeros(256, dtype=torch.uint8)
    x, W, off = _meta((R, 8)), _meta((1, 8, 8)), _meta((2,), I32)
    wide = _meta((2, 8), stride=(2 ** 32 + 8, 1))
    one, two = _meta((1, 2 ** 32 + 8)), _meta((2, 8))
    over = _meta((2, 2 ** 32 + 8), stride=(8, 1))
    calls = [lambda: sgl.moe_grouped_linear(x, off, W, x, ws),
             lambda: sgl.moe_grouped_linear_dgrad(x, off, W, x, ws),
             lambda: sgl.moe_grouped_linear_wgrad(x, x, off, W, ws),
             lambda: sgl.moe_grouped_linear(wide, off, W, two, ws),
             lambda: sgl.moe_grouped_linear(two, off, W, wide, ws),
             lambda: sgl.moe_grouped_linear(one, off, _meta((1, 8, 2 ** 32 + 8)), _meta((1, 8)), ws),
             lambda: sgl.moe_grouped_linear(over, off, _meta((1, 8, 2 ** 32 + 8)), two, ws),
             lambda: sgl.moe_grouped_linear(two, _meta((2 ** 32 + 2,), I32), _meta((2 ** 32 + 1, 8, 8)), two, ws),
             lambda: sgl.moe_swiglu(x, x, x),
             lambda: sgl.moe_swiglu(wide, wide, two),
             lambda: sgl.moe_swiglu(two, two, wide),
             lambda: sgl.moe_swiglu(two, two, two, w=_meta((2 ** 32 + 2,), F32), perm=_meta((2,), I32)),
             lambda: sgl.moe_swiglu_backward(two, two, two, wide, wide),
             lambda: sgl.moe_swiglu_backward(wide, two, two, two, two)]
    for call in calls:
        with pytest.raises(ValueError, match="31 bits|E \\+ 1 entries"):
            call()
    for sizes in ((1, R, 8, 8), (2 ** 32 + 1, 8, 8, 8), (1, 8, 2 ** 32 + 8, 8), (1, 8, 8, 2 ** 32 + 8), (1, -2 ** 33 + 5, 8, 8)):
        with pytest.raises(sgl.MoEError):
            sgl.linear_workspace_size(*sizes)


@pytest.mark.parametrize("eps,status", [(1e-39, -1), (1e-50, -1), (5e-324, -1), (-0.0, -2), (0.0, -2), (2.0 ** -126, -2)])
def test_adamw_eps_is_zero_or_a_normal_number_of_fp32(eps, status):
    """A smaller eps would be divided by as an infinity's reciprocal, and an
    element that never had a gradient would become NaN. -2: what comes after the
    check, a tensor without addresses."""
    cfg = sgl.moe_adamw_cfg(1e-3, 0.9, 0.99, eps, 0.1, 1.0, 1, None)
    none = (sgl.moe_adamw_tensor * 1)(sgl.moe_adamw_tensor(None, None, None, None, None, None, None, 10, 0, 0, 0, 1.0))
    assert sgl.lib().moe_adamw_step(ctypes.byref(cfg), none, 1, None) == status
