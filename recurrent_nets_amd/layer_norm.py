"""Layer norm over the last axis, forward and backward (the C ABI's slstm_layer_norm_*)."""
from __future__ import annotations

import torch

from .slstm import BF16, F32, _check, _dev, _ptr, _shape, _stream, alloc_workspace, load

_FLOATS = (torch.float32, torch.bfloat16)


def _dtype(t):
    return BF16 if t.dtype == torch.bfloat16 else F32


def _rows(x, name):
    """(leading shape, rows, width) of a dense (..., width) tensor."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must be (..., width) with width >= 1, got {tuple(x.shape)}")
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return tuple(x.shape[:-1]), rows, x.shape[-1]


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=None, mean=None, rstd=None,
                       want_stats=False, stream=None):
    """y = (x - mean) rstd weight + bias over the last axis of x (..., width), float32 or bfloat16;
    weight and bias (width) float32 or None. y has ``out_dtype`` (x's unless given; a float32
    residual stream gives the bfloat16 input of input_projection). Returns y, or (y, mean, rstd)
    with ``want_stats``: the float32 statistics of x's leading shape that layer_norm_backward
    takes."""
    L = load()
    _dev(x, "x", _FLOATS)
    _dev(weight, "weight", (torch.float32,))
    _dev(bias, "bias", (torch.float32,))
    lead, rows, width = _rows(x, "x")
    _shape(weight, "weight", (width,))
    _shape(bias, "bias", (width,))
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype, device=x.device)
    _dev(out, "out", _FLOATS)
    _shape(out, "out", x.shape)
    if want_stats and mean is None:
        mean = torch.empty(lead, dtype=torch.float32, device=x.device)
    if want_stats and rstd is None:
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _dev(t, name, (torch.float32,))
        _shape(t, name, lead)
    status = L.slstm_layer_norm_forward(_ptr(x), _dtype(x), _ptr(weight), _ptr(bias), float(eps), _ptr(out), _dtype(out),
                                        _ptr(mean), _ptr(rstd), rows, width, _stream(stream))
    _check(status, "slstm_layer_norm_forward")
    return (out, mean, rstd) if want_stats else out


def layer_norm_backward_workspace_bytes(rows: int, width: int) -> int:
    return int(load().slstm_layer_norm_backward_workspace_bytes(rows, width))


def layer_norm_backward(x, g_y, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, want_dweight=True,
                        want_dbias=True, workspace=None, stream=None):
    """Gradients of layer_norm_forward for the gradient g_y of y (x's shape, float32 or bfloat16):
    (dx in x's type, dweight (width) or None, dbias (width) or None), float32 sums over the rows
    in a fixed order. mean and rstd are the forward's."""
    L = load()
    _dev(x, "x", _FLOATS)
    _dev(g_y, "g_y", _FLOATS)
    _dev(weight, "weight", (torch.float32,))
    lead, rows, width = _rows(x, "x")
    _shape(g_y, "g_y", x.shape)
    _shape(weight, "weight", (width,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        _dev(t, name, (torch.float32,))
        _shape(t, name, lead)
    if dx is None:
        dx = torch.empty_like(x)
    if want_dweight and dweight is None:
        dweight = torch.empty(width, dtype=torch.float32, device=x.device)
    if want_dbias and dbias is None:
        dbias = torch.empty(width, dtype=torch.float32, device=x.device)
    _dev(dx, "dx", (x.dtype,))
    _shape(dx, "dx", x.shape)
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        _dev(t, name, (torch.float32,))
        _shape(t, name, (width,))
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = alloc_workspace(L.slstm_layer_norm_backward_workspace_bytes(rows, width), x.device)
    status = L.slstm_layer_norm_backward(_ptr(x), _dtype(x), _ptr(g_y), _dtype(g_y), _ptr(mean), _ptr(rstd), _ptr(weight),
                                         _ptr(dx), _ptr(dweight), _ptr(dbias), rows, width, _ptr(workspace),
                                         0 if workspace is None else workspace.numel() * workspace.element_size(),
                                         _stream(stream))
    _check(status, "slstm_layer_norm_backward")
    return dx, dweight, dbias
