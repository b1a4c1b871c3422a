"""torch-tensor front end of the RMS norm with the residual's addition in
libmamba_scan (`add_rms_norm_fwd`, `add_rms_norm_fp8` with an output in 8 bits,
and the gradients `add_rms_norm_bwd`): what stands between two blocks.

Marshalling only, as linattn.py: the entry points of include/mamba_rmsnorm.h do
the arithmetic.
"""
import ctypes

import torch

from . import _binding as _b
from .api import _IO, check_out
from .linattn import _io_of, _rows, _tensor, launch, scratch

EXPORTS = ("mamba_rmsnorm_fwd", "mamba_rmsnorm_fp8", "mamba_rmsnorm_bwd_workspace_bytes", "mamba_rmsnorm_bwd")
_F32 = torch.float32
_FP8 = torch.float8_e4m3fn
_lib = None


def load():
    """The scan library with the signatures of include/mamba_rmsnorm.h declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _b.load()
    i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    lib.mamba_rmsnorm_fwd.restype = ctypes.c_int
    lib.mamba_rmsnorm_fwd.argtypes = [i64, i32, i32, i32, f32, vp, i64, vp, i64, vp, vp, vp, vp]
    lib.mamba_rmsnorm_fp8.restype = ctypes.c_int
    lib.mamba_rmsnorm_fp8.argtypes = [i64, i32, i32, i32, f32, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp]
    lib.mamba_rmsnorm_bwd_workspace_bytes.restype = sz
    lib.mamba_rmsnorm_bwd_workspace_bytes.argtypes = [i64] + [i32] * 4
    lib.mamba_rmsnorm_bwd.restype = ctypes.c_int
    lib.mamba_rmsnorm_bwd.argtypes = [i64, i32, i32, i32, f32, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, vp, sz, vp]
    _lib = lib
    return lib


def _weight(weight, dev, channels):
    if weight is None:
        return None, 0
    weight = _tensor(weight, "weight", _F32, dev)
    if weight.shape != (channels,):
        raise _b.MambaScanError(2, "weight must be [%d] (got %s)" % (channels, list(weight.shape)))
    weight = weight.contiguous()
    return weight, weight.data_ptr()


def _like(t, name, shape, dev):
    """(residual code, tensor, address, row stride) of a tensor on the residual's side"""
    code, dtype, _ = _io_of(t, name)
    if t.shape != shape:
        raise _b.MambaScanError(2, "%s must be %s (got %s)" % (name, list(shape), list(t.shape)))
    return code, dtype


def _forward(x, residual, weight, align, inplace):
    """The checked tensors and their addresses, and h."""
    io, dtype, dev = _io_of(x, "x")
    shape = x.shape
    nrow = len(shape) - 1
    if nrow < 0:
        raise _b.MambaScanError(2, "x must be [..., channels]")
    channels = shape[-1]
    x, xp, xs = _rows(x, "x", dtype, dev, nrow, align or x.element_size())
    res, rp, rs, h, hp = io, 0, 0, x, 0
    if inplace and residual is None:
        raise _b.MambaScanError(1, "inplace needs a residual")
    if residual is not None:
        res, rtype = _like(residual, "residual", shape, dev)
        if res > io:
            raise TypeError("residual must be float32 or like x (got %s)" % rtype)
        if inplace:
            h = check_out(residual, "residual", shape, rtype, x.device)
        residual, rp, rs = _rows(residual, "residual", rtype, dev, nrow, align or residual.element_size())
        if inplace and residual is not h:
            raise _b.MambaScanError(4, "the residual of an in-place call must be %d-byte aligned" % align)
        if not inplace:
            h = x.new_empty(shape, dtype=rtype)
        hp = h.data_ptr()
    weight, wp = _weight(weight, dev, channels)
    rows = x.numel() // channels if channels else 0
    return dev, x, h, rows, channels, io, res, (xp, xs, rp, rs, wp), hp, (x, residual, weight)


def add_rms_norm_fwd(x, residual, weight, *, eps=1e-5, inplace=False, out=None):
    """h = x + residual and its RMS norm y = h / sqrt(mean(h^2) + eps) * weight over the channels of each row. x
    [..., channels] float32 or bfloat16; residual like x, float32 or of x's type, or None (then h is x itself); weight
    [channels] float32, or None. x and residual may be columns of a wider tensor; they are read in place. With
    inplace=True h is written over the residual.
    Returns (y like x, h like the residual)."""
    lib = _lib or load()
    dev, x, h, rows, channels, io, res, args, hp, keep = _forward(x, residual, weight, 0, inplace)
    y = x.new_empty(x.shape) if out is None else check_out(out, "out", x.shape, x.dtype, x.device)
    launch(dev, "mamba_rmsnorm_fwd", lib, lib.mamba_rmsnorm_fwd, rows, channels, io, res, eps, *args, y.data_ptr(), hp)
    return y, h


def add_rms_norm_fp8(x, residual, weight, *, block=None, eps=1e-5, inplace=False):
    """`add_rms_norm_fwd` with y as float8_e4m3fn values times float32 scales: one scale for each row, or with block=128
    one for each 128 neighbouring channels of a row. channels must be a multiple of 16.
    Returns (y, scales [..., 1 or ceil(channels / 128)], h)."""
    lib = _lib or load()
    if block not in (None, 128):
        raise _b.MambaScanError(2, "block must be None or 128 (got %r)" % (block,))
    dev, x, h, rows, channels, io, res, args, hp, keep = _forward(x, residual, weight, 16, inplace)
    y = x.new_empty(x.shape, dtype=_FP8)
    scales = x.new_empty((*x.shape[:-1], -(-channels // block) if block else 1), dtype=_F32)
    launch(dev, "mamba_rmsnorm_fp8", lib, lib.mamba_rmsnorm_fp8, rows, channels, io, res, eps, block or 0, *args,
           y.data_ptr(), scales.data_ptr(), hp)
    return y, scales, h


def add_rms_norm_bwd(h, weight, dy, dh=None, *, eps=1e-5, workspace=None):
    """Gradients of `add_rms_norm_fwd` from the h that it returned, dy = dL/dy and dh = dL/dh as it comes from behind (like
    h, or None for zeros).

    Returns a dict: dresidual (like h) and dx (of dy's type; where the types agree the same tensor), and dweight
    ([channels] float32) where a weight is given."""
    lib = _lib or load()
    io, dtype, dev = _io_of(dy, "dy")
    shape = dy.shape
    nrow = len(shape) - 1
    if nrow < 0:
        raise _b.MambaScanError(2, "dy must be [..., channels]")
    channels = shape[-1]
    dy, dyp, dys = _rows(dy, "dy", dtype, dev, nrow, dy.element_size())
    res, rtype = _like(h, "h", shape, dev)
    if res > io:
        raise TypeError("h must be float32 or like dy (got %s)" % rtype)
    h, hp, hs = _rows(h, "h", rtype, dev, nrow, h.element_size())
    dhp = dhs = 0
    if dh is not None:
        _like(dh, "dh", shape, dev)
        dh, dhp, dhs = _rows(dh, "dh", rtype, dev, nrow, dh.element_size())
    weight, wp = _weight(weight, dev, channels)
    grads = {"dresidual": dy.new_empty(shape, dtype=rtype)}
    dxp = dwp = need = 0
    if res != io:
        grads["dx"] = dy.new_empty(shape)
        dxp = grads["dx"].data_ptr()
    else:
        grads["dx"] = grads["dresidual"]
    rows = dy.numel() // channels if channels else 0
    if weight is not None:
        grads["dweight"] = torch.empty_like(weight)
        dwp = grads["dweight"].data_ptr()
        need = lib.mamba_rmsnorm_bwd_workspace_bytes(rows, channels, io, res, 1)
    ws, ws_bytes, keep = scratch(workspace, need, dy)
    launch(dev, "mamba_rmsnorm_bwd", lib, lib.mamba_rmsnorm_bwd, rows, channels, io, res, eps, hp, hs, wp, dyp, dys, dhp, dhs,
           dxp, grads["dresidual"].data_ptr(), dwp, ws, ws_bytes)
    return grads


def add_rms_norm_workspace_bytes(rows, channels, dtype, residual_dtype=_F32):
    """Bytes of workspace `add_rms_norm_bwd` needs for the gradient of a weight."""
    return int(load().mamba_rmsnorm_bwd_workspace_bytes(rows, channels, _IO[dtype], _IO[residual_dtype], 1))
