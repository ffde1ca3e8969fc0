"""What layer norm and linear attention refuse, on the host: the C ABI's argument checks and workspace
sizes (no GPU work is done), and the binding's."""
import ctypes
import os

import pytest
import torch

import recurrent_nets_amd as amd
from recurrent_nets_amd import linear_attention as la
from recurrent_nets_amd import slstm


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(slstm.lib_path()):
        pytest.fail("library not built: run `python -m recurrent_nets_amd.build`")
    return slstm.load()


PTR = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)


def _norm(lib, **kw):
    a = dict(x=PTR, xt=0, w=None, b=None, eps=1e-5, y=PTR, yt=1, m=None, r=None, rows=5, width=16, stream=None)
    a.update(kw)
    return lib.slstm_layer_norm_forward(*a.values())


def test_norm_forward_checks(lib):
    assert _norm(lib, rows=-1) == slstm.EINVAL
    assert _norm(lib, width=0) == slstm.EINVAL
    assert _norm(lib, width=(1 << 20) + 1) == slstm.EINVAL
    assert _norm(lib, xt=3) == slstm.EINVAL and _norm(lib, yt=-1) == slstm.EINVAL
    for eps in (-1e-5, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == slstm.EINVAL
    assert _norm(lib, x=None) == slstm.EINVAL and _norm(lib, y=None) == slstm.EINVAL
    assert _norm(lib, x=ODD) == slstm.EINVAL and _norm(lib, w=ODD) == slstm.EINVAL and _norm(lib, m=ODD) == slstm.EINVAL
    assert _norm(lib, rows=1 << 45, width=1 << 10) == slstm.EINVAL
    assert _norm(lib, rows=0, x=None, y=None) == slstm.OK  # nothing to do


def _norm_back(lib, **kw):
    a = dict(x=PTR, xt=0, g=PTR, gt=0, m=PTR, r=PTR, w=None, dx=PTR, dw=PTR, db=None, rows=5, width=16, ws=PTR, wsb=1 << 30,
             stream=None)
    a.update(kw)
    return lib.slstm_layer_norm_backward(*a.values())


def test_norm_backward_checks(lib):
    for name in ("x", "g", "m", "r", "dx"):
        assert _norm_back(lib, **{name: None}) == slstm.EINVAL
        assert _norm_back(lib, **{name: ODD}) == slstm.EINVAL
    assert _norm_back(lib, ws=None) == slstm.EINVAL
    assert _norm_back(lib, ws=ctypes.c_void_p(4096 + 64)) == slstm.EINVAL
    assert _norm_back(lib, wsb=16) == slstm.EWORKSPACE
    assert "needed" in lib.slstm_last_error().decode()
    assert lib.slstm_layer_norm_backward_workspace_bytes(5, 16) >= 2 * 16 * 4
    assert lib.slstm_layer_norm_backward_workspace_bytes(5, 0) == 0
    assert lib.slstm_layer_norm_backward_workspace_bytes(-1, 16) == 0


def _heads(data=4096, b=640, t=64, h=32):
    return la._Heads(data, b, t, h)


def _forward(lib, **kw):
    a = dict(q=_heads(), k=_heads(), v=_heads(), dt=1, g=PTR, per=0, s0=None, scale=1.0, out=_heads(), fin=None, B=2, T=10,
             H=2, dk=32, dv=32, cu=None, n=0, ws=PTR, wsb=1 << 30, stream=None)
    a.update(kw)
    refs = [ctypes.byref(x) if isinstance(x, la._Heads) else x for x in a.values()]
    return lib.slstm_linear_attention_forward(*refs)


def test_linear_forward_checks(lib):
    bad = [dict(B=0), dict(T=-1), dict(H=0), dict(dk=12), dict(dv=0), dict(dk=264), dict(dt=2), dict(q=None), dict(out=None),
           dict(v=_heads(data=0)), dict(k=_heads(data=4104)), dict(q=_heads(t=65)), dict(q=_heads(t=-64)),
           dict(k=_heads(t=1 << 24)), dict(g=None), dict(s0=ctypes.c_void_p(4100)), dict(fin=ctypes.c_void_p(4100)),
           dict(scale=float("inf")), dict(scale=float("nan")), dict(cu=PTR), dict(n=3), dict(cu=PTR, n=3),
           dict(cu=ctypes.c_void_p(4098), n=3, B=1)]
    for kw in bad:
        assert _forward(lib, **kw) == slstm.EINVAL, kw
        assert lib.slstm_last_error().decode()
    assert _forward(lib, T=4096, wsb=16) == slstm.EWORKSPACE  # few heads, many steps: segments
    assert _forward(lib, T=4096, ws=None) == slstm.EINVAL


def _step(lib, **kw):
    a = dict(q=_heads(), k=_heads(), v=_heads(), dt=0, g=PTR, per=0, state=PTR, slots=None, n=2, scale=1.0, out=PTR, B=2, H=2,
             dk=32, dv=32, stream=None)
    a.update(kw)
    return lib.slstm_linear_attention_step(*[ctypes.byref(x) if isinstance(x, la._Heads) else x for x in a.values()])


def test_linear_step_checks(lib):
    for kw in (dict(B=0), dict(state=None), dict(out=None), dict(n=1), dict(n=0, slots=PTR), dict(slots=ODD), dict(dk=20),
               dict(out=ctypes.c_void_p(4104)), dict(g=None)):
        assert _step(lib, **kw) == slstm.EINVAL, kw


def _backward(lib, **kw):
    a = dict(q=_heads(), k=_heads(), v=_heads(), dt=0, g=PTR, per=0, s0=None, scale=1.0, go=_heads(), gf=None, dq=_heads(),
             dk_=_heads(), dv_=_heads(), dg=PTR, ds=None, B=2, T=10, H=2, dk=32, dv=32, cu=None, n=0, ws=PTR, wsb=1 << 30,
             stream=None)
    a.update(kw)
    return lib.slstm_linear_attention_backward(*[ctypes.byref(x) if isinstance(x, la._Heads) else x for x in a.values()])


def test_linear_backward_checks(lib):
    for kw in (dict(go=None), dict(dq=None), dict(dk_=_heads(data=0)), dict(dv_=_heads(h=33)), dict(gf=ODD), dict(ds=ODD),
               dict(dg=ODD), dict(per=1), dict(ws=None), dict(dv=7)):
        assert _backward(lib, **kw) == slstm.EINVAL, kw
    assert _backward(lib, wsb=100) == slstm.EWORKSPACE


def test_linear_workspace_sizes(lib):
    f, b = lib.slstm_linear_attention_workspace_bytes, lib.slstm_linear_attention_backward_workspace_bytes
    assert f(256, 512, 8, 64, 64, 0) == 0     # heads enough for the GPU: one segment, no workspace
    assert f(1, 16384, 1, 128, 128, 0) > 0
    assert f(1, 16384, 1, 128, 128, 7) > 0
    assert f(2, 64, 1, 128, 128, 7) == 0      # packed sequences lie in one row
    assert f(1, 64, 1, 100, 128, 0) == 0 and b(0, 64, 1, 128, 128, 0) == 0
    assert b(256, 512, 8, 64, 64, 0) >= 2 * 256 * 512 * 8 * 4


def test_binding_refuses():
    q = torch.zeros(1, 4, 2, 16)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        amd.linear_attention_forward(q, q, q, g)
    with pytest.raises(ValueError, match="device tensor"):
        amd.linear_attention_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="device tensor"):
        amd.linear_attention_backward(q, q, q, g, q)
    with pytest.raises(ValueError, match="device tensor"):
        amd.layer_norm_forward(q)
    with pytest.raises(ValueError, match="device tensor"):
        amd.layer_norm_backward(q, q, q[..., 0], q[..., 0])
    with pytest.raises(ValueError, match="must be"):
        amd.linear_attention_forward(q[0], q[0], q[0], g)
    with pytest.raises(TypeError):
        amd.linear_attention_forward(q.half(), q.half(), q.half(), g)
    with pytest.raises(ValueError, match="share"):
        la._own(torch.zeros(1, 1, 2, 8).expand(1, 4, 2, 8), "dq")
