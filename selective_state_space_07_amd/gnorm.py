"""torch-tensor front end of the group norm with an activation and a gate in
libmamba_scan (`group_norm_fwd` and its gradients `group_norm_bwd`): the norm
behind a scan, per head or over all channels, centered or RMS.

Marshalling only, as linattn.py: the entry points of include/mamba_gnorm.h do
the arithmetic.
"""
import ctypes

import torch

from . import _binding as _b
from .api import check_out
from .linattn import _io_of, _rows, _tensor, launch, scratch

EXPORTS = ("mamba_gnorm_fwd", "mamba_gnorm_bwd_workspace_bytes", "mamba_gnorm_bwd")
_ACT = {"none": 0, "silu": 1, "sigmoid": 2}
_F32 = torch.float32
_lib = None


def load():
    """The scan library with the signatures of include/mamba_gnorm.h declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _b.load()
    i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    head = [i64] + [i32] * 6 + [f32, vp, i64, vp, i64, vp, vp]
    lib.mamba_gnorm_fwd.restype = ctypes.c_int
    lib.mamba_gnorm_fwd.argtypes = head + [vp, vp]
    lib.mamba_gnorm_bwd.restype = ctypes.c_int
    lib.mamba_gnorm_bwd.argtypes = head + [vp, i64] + [vp] * 5 + [sz, vp]
    lib.mamba_gnorm_bwd_workspace_bytes.restype = sz
    lib.mamba_gnorm_bwd_workspace_bytes.argtypes = [i64] + [i32] * 5
    _lib = lib
    return lib


def _like(t, shape, name, dtype, device):
    if isinstance(t, torch.Tensor) and t.shape != shape:
        raise _b.MambaScanError(2, "%s must be %s (got %s)" % (name, list(shape), list(t.shape)))
    return _rows(t, name, dtype, device, len(shape) - 1, 1)


def _param(t, name, device, channels):
    if t is None:
        return None, 0
    t = _tensor(t, name, _F32, device)
    if t.shape != (channels,):
        raise _b.MambaScanError(2, "%s must be [%d] (got %s)" % (name, channels, list(t.shape)))
    t = t.contiguous()
    return t, t.data_ptr()


def _common(x, weight, bias, groups, z, activation, gate_first, center, eps):
    """The checked tensors, and the entry points' common arguments."""
    io, dtype, dev = _io_of(x, "x")
    act = _ACT.get(activation)
    if act is None:
        raise _b.MambaScanError(2, "activation must be one of %s (got %r)" % (sorted(_ACT), activation))
    if gate_first and z is None:
        raise _b.MambaScanError(1, "gate_first needs z")
    shape = x.shape
    if len(shape) < 1:
        raise _b.MambaScanError(2, "x must be [..., channels]")
    channels = shape[-1]
    x, xp, xs = _rows(x, "x", dtype, dev, len(shape) - 1, 1)
    gate = zp = zs = 0
    if z is not None:
        z, zp, zs = _like(z, shape, "z", dtype, dev)
        gate = 2 if gate_first else 1
    weight, wp = _param(weight, "weight", dev, channels)
    bias, bp = _param(bias, "bias", dev, channels)
    rows = x.numel() // channels if channels else 0
    return dev, x, (rows, channels, groups, io, act, gate, 1 if center else 0, eps, xp, xs, zp, zs, wp, bp), (z, weight, bias)


def group_norm_fwd(x, weight, bias, groups, z=None, *, eps=1e-5, activation="silu", gate_first=False, center=True,
                   out=None):
    """x [..., channels], normed over each group of channels // groups neighbouring channels of a row, times weight
    plus bias ([channels] float32, or None), with an activation ("silu", "sigmoid" or "none"): of the gate z (like x),
    which multiplies the result or, with gate_first, x before its norm; without z, of the result itself. center=False
    takes no mean off (RMS). x and z may be columns of a wider tensor; they are read in place. Returns y like x."""
    lib = _lib or load()
    dev, x, args, keep = _common(x, weight, bias, groups, z, activation, gate_first, center, eps)
    y = x.new_empty(x.shape) if out is None else check_out(out, "out", x.shape, x.dtype, x.device)
    launch(dev, "mamba_gnorm_fwd", lib, lib.mamba_gnorm_fwd, *args, y.data_ptr())
    return y


def group_norm_bwd(x, weight, bias, groups, dy, z=None, *, eps=1e-5, activation="silu", gate_first=False, center=True,
                   workspace=None):
    """Gradients of `group_norm_fwd` given dy = dL/dy (like x); the other arguments are the forward's.

    Returns a dict: dx (and dz, where z is given) like x, and dweight, dbias ([channels] float32) where weight and
    bias are given."""
    lib = _lib or load()
    dev, x, args, (z, weight, bias) = _common(x, weight, bias, groups, z, activation, gate_first, center, eps)
    shape = x.shape
    dy, dyp, dys = _like(dy, shape, "dy", x.dtype, dev)
    grads = {"dx": x.new_empty(shape)}
    dz = dw = db = 0
    if z is not None:
        grads["dz"] = x.new_empty(shape)
        dz = grads["dz"].data_ptr()
    if weight is not None:
        grads["dweight"] = torch.empty_like(weight)
        dw = grads["dweight"].data_ptr()
    if bias is not None:
        grads["dbias"] = torch.empty_like(bias)
        db = grads["dbias"].data_ptr()
    need = 0
    if dw or db:
        need = lib.mamba_gnorm_bwd_workspace_bytes(*args[:4], 1 if dw else 0, 1 if db else 0)
    ws, ws_bytes, keep = scratch(workspace, need, x)
    launch(dev, "mamba_gnorm_bwd", lib, lib.mamba_gnorm_bwd, *args, dyp, dys, grads["dx"].data_ptr(), dz, dw, db, ws,
           ws_bytes)
    return grads


def group_norm_workspace_bytes(rows, channels, groups, dtype, weight=True, bias=True):
    """Bytes of workspace `group_norm_bwd` needs for the gradients of weight and bias (where they are given)."""
    return int(load().mamba_gnorm_bwd_workspace_bytes(rows, channels, groups, {torch.float32: 0, torch.bfloat16: 1}[dtype],
                                                      int(weight), int(bias)))
