"""The training operators' C-ABI without a GPU: descriptors, workspace sizes
and every refusal that comes before a launch."""
import ctypes

import pytest
import torch

import sigmoid_group_limited_b200 as sgl

A = 1 << 20  # an aligned fake "device" address: never dereferenced on these paths


def _linear(**kw):
    d = dict(E=4, R=10, N=16, K=24, ld_x=24, ld_y=16, out_type=0, accumulate=0)
    d.update(kw)
    return sgl.moe_linear_desc(*[d[k] for k, _ in sgl.moe_linear_desc._fields_])


BAD_LINEAR = [dict(E=0), dict(E=1025), dict(R=-1), dict(R=(1 << 25) + 1), dict(N=12), dict(N=0),
              dict(N=16392, ld_y=16392), dict(K=20), dict(K=-8), dict(ld_x=16), dict(ld_x=28),
              dict(ld_y=8), dict(ld_y=20), dict(out_type=2), dict(accumulate=1)]
CALLS = ("moe_grouped_linear", "moe_grouped_linear_dgrad", "moe_grouped_linear_wgrad")


@pytest.mark.parametrize("bad", BAD_LINEAR, ids=str)
def test_bad_linear_descriptor(bad):
    L, d = sgl.lib(), _linear(**bad)
    assert L.moe_linear_workspace_size(ctypes.byref(d)) == 0
    for f in CALLS:
        assert getattr(L, f)(ctypes.byref(d), A, A, A, A, A, 1 << 30, None) == -1


@pytest.mark.parametrize("f", CALLS)
def test_linear_pointers(f):
    L = sgl.lib()
    call = getattr(L, f)
    assert call(None, A, A, A, A, A, 1 << 30, None) == -1
    for kw in (dict(), dict(out_type=1), dict(out_type=1, accumulate=1)):
        d = _linear(**kw)
        need = L.moe_linear_workspace_size(ctypes.byref(d))
        assert need >= 256
        for i in range(4):
            for bad, st in ((None, -2), (A + 8, -3)):
                p = [A] * 4
                p[i] = bad
                assert call(ctypes.byref(d), *p, A, need, None) == st
        assert call(ctypes.byref(d), A, A, A, A, None, need, None) == -4
        assert call(ctypes.byref(d), A, A, A, A, A + 4, need, None) == -4
        assert call(ctypes.byref(d), A, A, A, A, A, need - 1, None) == -4
    # without rows the row-wise pointers may be NULL, the others not
    d = _linear(R=0)
    need = L.moe_linear_workspace_size(ctypes.byref(d))
    wg = f.endswith("wgrad")
    for p in ((A, A, None, A) if not wg else (A, A, A, None), (A, None, A, A)):
        p = (p[0], p[2], p[1], p[3]) if wg else p
        assert call(ctypes.byref(d), *p, A, need, None) == -2
    code = ctypes.c_int32(0)
    assert L.moe_linear_read_error(A, 256, None, None) == -2
    assert L.moe_linear_read_error(None, 256, None, ctypes.byref(code)) == -4
    assert L.moe_linear_read_error(A, 255, None, ctypes.byref(code)) == -4


@pytest.mark.parametrize("bad", [(-1, 8, 8, 8, 8, 0.), (4, 12, 16, 16, 16, 0.), (4, 0, 8, 8, 8, 0.),
                                 (4, 16, 8, 16, 16, 0.), (4, 16, 16, 20, 16, 0.),
                                 (4, 16, 16, 16, 16, float("nan")), ((1 << 25) + 1, 8, 8, 8, 8, 0.)])
def test_bad_swiglu_descriptor(bad):
    L, d = sgl.lib(), sgl.moe_swiglu_desc(*bad)
    assert L.moe_swiglu(ctypes.byref(d), A, A, None, None, 0, None, A, None) == -1
    assert L.moe_swiglu_backward(ctypes.byref(d), A, A, A, None, None, 0, None, A, A, None, None) == -1


def test_swiglu_pointers():
    L = sgl.lib()
    d = sgl.moe_swiglu_desc(4, 16, 16, 16, 16, 0.0)
    r = ctypes.byref(d)
    assert L.moe_swiglu(None, A, A, None, None, 0, None, A, None) == -1
    assert L.moe_swiglu(r, None, A, None, None, 0, None, A, None) == -2
    assert L.moe_swiglu(r, A, A, None, None, 0, None, None, None) == -2
    assert L.moe_swiglu(r, A, A + 8, None, None, 0, None, A, None) == -3
    assert L.moe_swiglu(r, A, A, A + 4, None, 0, None, A, None) == -3
    assert L.moe_swiglu(r, A, A, None, None, 0, A + 2, A, None) == -3
    assert L.moe_swiglu(r, A, A, A, A, -1, None, A, None) == -1
    assert L.moe_swiglu_backward(r, None, A, A, None, None, 0, None, A, A, None, None) == -2
    assert L.moe_swiglu_backward(r, A, A, A, None, None, 0, None, A, None, None, None) == -2
    assert L.moe_swiglu_backward(r, A, A, A, None, None, 0, None, A, A, A, None) == -2    # dw without w
    assert L.moe_swiglu_backward(r, A, A, A, A, None, 0, None, A, A, A + 4, None) == -3
    bad = sgl.moe_swiglu_desc(4, 16, 16, 16, 8, 0.0)                                      # ld_dg
    assert L.moe_swiglu_backward(ctypes.byref(bad), A, A, A, None, None, 0, None, A, A, None, None) == -1


def _tensor(**kw):
    d = dict(p=A, master=None, g=A, m=A, v=A, m_scale=None, v_scale=None, n=10, p_type=0, g_type=0,
             state_type=0, wd_scale=1.0)
    d.update(kw)
    return (sgl.moe_adamw_tensor * 1)(sgl.moe_adamw_tensor(*[d[k] for k, _ in sgl.moe_adamw_tensor._fields_]))


def _cfg(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=1, dyn=None)
    d.update(kw)
    return sgl.moe_adamw_cfg(*[d[k] for k, _ in sgl.moe_adamw_cfg._fields_])


@pytest.mark.parametrize("bad,status", [
    (dict(p_type=2), -1), (dict(g_type=-1), -1), (dict(state_type=2), -1), (dict(n=-1), -1),
    (dict(n=(1 << 40) + 1), -1), (dict(wd_scale=float("inf")), -1), (dict(p_type=1, master=A), -1),
    (dict(p=None), -2), (dict(g=None), -2), (dict(m=None), -2), (dict(v=None), -2),
    (dict(state_type=1), -2), (dict(state_type=1, m_scale=A), -2), (dict(p=A + 8), -3),
    (dict(master=A + 4), -3), (dict(g=A + 2), -3), (dict(m=A + 1), -3), (dict(v=A + 12), -3),
    (dict(state_type=1, m_scale=A + 2, v_scale=A), -3)], ids=str)
def test_bad_adamw_tensor(bad, status):
    assert sgl.lib().moe_adamw_step(ctypes.byref(_cfg()), _tensor(**bad), 1, None) == status


@pytest.mark.parametrize("bad", [dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=-1e-8),
                                 dict(eps=float("inf")), dict(step=0), dict(lr=float("nan")),
                                 dict(grad_scale=float("inf")), dict(weight_decay=float("nan"))], ids=str)
def test_bad_adamw_cfg(bad):
    assert sgl.lib().moe_adamw_step(ctypes.byref(_cfg(**bad)), _tensor(), 1, None) == -1


def test_adamw_list():
    L = sgl.lib()
    assert L.moe_adamw_step(None, _tensor(), 1, None) == -1
    assert L.moe_adamw_step(ctypes.byref(_cfg()), _tensor(), -1, None) == -1
    assert L.moe_adamw_step(ctypes.byref(_cfg()), None, 1, None) == -2
    assert L.moe_adamw_step(ctypes.byref(_cfg(dyn=A + 4)), _tensor(), 1, None) == -3
    sgl.moe_adamw_step(sgl.make_adamw_tensors([]))  # no tensors: nothing to do


def test_binding_refuses_what_it_cannot_describe():
    bf, f32 = torch.bfloat16, torch.float32
    x, W = torch.zeros(6, 24, dtype=bf), torch.zeros(4, 16, 24, dtype=bf)
    off, y = torch.zeros(5, dtype=torch.int32), torch.zeros(6, 16, dtype=bf)
    ws = torch.zeros(256, dtype=torch.uint8)
    for bad in ((x.to(f32), off, W, y), (x.t().contiguous().t(), off, W, y), (x, off.long(), W, y),
                (x, off[:4], W, y), (x, off, W.transpose(1, 2), y), (x, off, W, y[:5]), (x, off, W, y.half()),
                (x[:, :16], off, W, y), (x, off, W, y)):     # the last one: tensors on the CPU
        with pytest.raises(ValueError):
            sgl.moe_grouped_linear(*bad, ws)
    with pytest.raises(ValueError):
        sgl.moe_grouped_linear_dgrad(y, off, W, x[:, :16], ws)
    with pytest.raises(ValueError):
        sgl.moe_grouped_linear_wgrad(y, x, off, W.transpose(1, 2), ws)
    h = torch.zeros(6, 24, dtype=bf)
    w, perm = torch.zeros(6), torch.zeros(6, dtype=torch.int32)
    for bad in (dict(u=h[:5]), dict(h=h.float()), dict(w=w[:5]), dict(w=w.half()), dict(perm=perm),
                dict(w=w, perm=perm.long()), dict(w=w, perm=perm[:5]), dict(rows=perm[:0])):
        kw = dict(g=h, u=h, h=h)
        kw.update(bad)
        with pytest.raises(ValueError):
            sgl.moe_swiglu(**kw)
    with pytest.raises(ValueError):
        sgl.moe_swiglu_backward(h, h, h, h, h, dw=w)
    with pytest.raises(ValueError):
        sgl.moe_swiglu_backward(h, h, h, h, h, w=w, dw=w[:5])
    p = torch.zeros(300)
    q, s = p.to(torch.float8_e4m3fn), torch.zeros(2)
    for bad in (dict(m=q), dict(m=q, v=q), dict(m=q, v=q, m_scale=s, v_scale=s[:1]), dict(m_scale=s),
                dict(p=p.half()), dict(g=p[:299]), dict(master=p.to(bf)), dict()):
        kw = dict(p=p, g=p, m=p, v=p)
        kw.update(bad)
        with pytest.raises(ValueError):
            sgl.make_adamw_tensors([kw])


def test_dyn_values():
    assert sgl.adamw_dyn(0.1, 0.5, 0.75, 2, 3.0) == [0.1, 0.75, 0.4375 ** 0.5, 3.0]
