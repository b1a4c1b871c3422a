"""torch-tensor front end of the short causal convolution in libmamba_scan
(`conv_fwd`, its gradients `conv_bwd`, and `conv_step` for one token): the
depthwise convolution over time in front of a Mamba-2 scan's x, B and C.

Marshalling only, as linattn.py: the entry points of include/mamba_conv.h do
the arithmetic.
"""
import ctypes

import torch

from . import _binding as _b
from .api import _IO, check_out
from .linattn import _f32, _ids, _io_of, _rows, _tensor, launch, scratch

EXPORTS = ("mamba_conv_fwd", "mamba_conv_bwd_workspace_bytes", "mamba_conv_bwd", "mamba_conv_step")
MAX_PARTS = 4  # MAMBA_CONV_MAX_PARTS
_ACT = {"none": 0, "silu": 1}
_F32 = torch.float32
_lib = None


def load():
    """The scan library with the signatures of include/mamba_conv.h declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _b.load()
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    head = [i32] * 6 + [vp, i64] + [vp] * 4 + [i32, vp, vp]
    lib.mamba_conv_fwd.restype = ctypes.c_int
    lib.mamba_conv_fwd.argtypes = head + [vp, vp]
    lib.mamba_conv_bwd_workspace_bytes.restype = sz
    lib.mamba_conv_bwd_workspace_bytes.argtypes = [i32] * 5
    lib.mamba_conv_bwd.restype = ctypes.c_int
    lib.mamba_conv_bwd.argtypes = head + [vp] * 7 + [sz, vp]
    lib.mamba_conv_step.restype = ctypes.c_int
    lib.mamba_conv_step.argtypes = [i32] * 5 + [vp, i64] + [vp] * 3 + [i32, vp, vp, vp, vp]
    _lib = lib
    return lib


def _act(activation):
    code = _ACT.get(activation)
    if code is None:
        raise _b.MambaScanError(2, "activation must be one of %s (got %r)" % (sorted(_ACT), activation))
    return code


def _weights(weight, bias, dev, channels):
    """(taps, the checked weight and bias, their addresses)"""
    weight = _tensor(weight, "weight", _F32, dev)
    if weight.dim() != 2 or weight.shape[0] != channels or weight.shape[1] < 1:
        raise _b.MambaScanError(2, "weight must be [%d, taps] (got %s)" % (channels, list(weight.shape)))
    weight, wp = _f32(weight, "weight", dev, weight.shape)
    bias, bp = _f32(bias, "bias", dev, (channels,))
    return weight.shape[1], weight, bias, wp, bp


def _sizes(split, channels):
    """The channels of each part."""
    if split is None:
        return [channels]
    split = [int(n) for n in split]
    if not 1 <= len(split) <= MAX_PARTS or min(split) < 1 or sum(split) != channels:
        raise _b.MambaScanError(2, "split must be 1 to %d positive numbers that add up to %d (got %s)" %
                                (MAX_PARTS, channels, split))
    return split


def _outs(x, lead, sizes, split, out):
    """The parts of y: the caller's, or new ones."""
    if out is None:
        return [x.new_empty((*lead, n)) for n in sizes]
    if split is None:
        out = [out]
    if not isinstance(out, (list, tuple)) or len(out) != len(sizes):
        raise _b.MambaScanError(2, "out must be %d tensors, one for each part" % len(sizes))
    return [check_out(o, "out", (*lead, n), x.dtype, x.device) for o, n in zip(out, sizes)]


def _array(kind, values):
    return (kind * len(values))(*values)


def conv_fwd(x, weight, bias=None, state=None, *, activation="silu", seq_idx=None, split=None, out=None,
             state_out=None, return_state=True):
    """Whole sequence: x [batch, seqlen, channels] (it may be columns of a wider tensor; it is read in place); weight
    [channels, taps] float32, taps 2 to 4, the last of which multiplies the newest token; bias [channels] float32 or
    None; state [batch, channels, taps - 1] float32, the inputs before the first token, oldest first, or None (zeros);
    activation "silu" or "none"; seq_idx [batch, seqlen] integer document ids or None (packed documents: the inputs
    before a token are zero wherever the id changes); split: channel counts, to get y as that many tensors (x, B and C
    of a Mamba-2 scan, for instance).
    Returns (y [batch, seqlen, channels] or a tuple of its parts, final state or None)."""
    lib = _lib or load()
    io, dtype, dev = _io_of(x, "x")
    act = _act(activation)
    if x.dim() != 3:
        raise _b.MambaScanError(2, "x must be [batch, seqlen, channels]")
    x, xp, xs = _rows(x, "x", dtype, dev, 2, x.element_size())
    batch, seqlen, channels = x.shape
    taps, weight, bias, wp, bp = _weights(weight, bias, dev, channels)
    state_shape = (batch, channels, taps - 1)
    state, sp = _f32(state, "state", dev, state_shape)
    seq_idx, ip = _ids(seq_idx, dev, batch, seqlen)
    sizes = _sizes(split, channels)
    ys = _outs(x, (batch, seqlen), sizes, split, out)
    if state_out is not None:
        check_out(state_out, "state_out", state_shape, _F32, x.device)
    elif return_state:
        state_out = x.new_empty(state_shape, dtype=_F32)
    launch(dev, "mamba_conv_fwd", lib, lib.mamba_conv_fwd, batch, seqlen, channels, taps, io, act, xp, xs, ip, wp, bp, sp,
           len(ys), _array(ctypes.c_int32, sizes), _array(ctypes.c_void_p, [y.data_ptr() for y in ys]),
           0 if state_out is None else state_out.data_ptr())
    return ys[0] if split is None else tuple(ys), state_out


def conv_bwd(x, weight, dy, bias=None, state=None, dstate=None, *, activation="silu", seq_idx=None, workspace=None):
    """Gradients of `conv_fwd` given dy = dL/dy (like x, or its parts along the channels, as `split` makes them) and
    dstate = dL/d(final state) (float32 like state, or None for zeros); the other arguments are the forward's.

    Returns a dict: dx (like x, contiguous), dweight, dbias (where a bias is given) and dstate (where a state is given:
    its gradient), float32."""
    lib = _lib or load()
    io, dtype, dev = _io_of(x, "x")
    act = _act(activation)
    if x.dim() != 3:
        raise _b.MambaScanError(2, "x must be [batch, seqlen, channels]")
    es = x.element_size()
    x, xp, xs = _rows(x, "x", dtype, dev, 2, es)
    batch, seqlen, channels = x.shape
    taps, weight, bias, wp, bp = _weights(weight, bias, dev, channels)
    state_shape = (batch, channels, taps - 1)
    state, sp = _f32(state, "state", dev, state_shape)
    dstate, dsp = _f32(dstate, "dstate", dev, state_shape)
    seq_idx, ip = _ids(seq_idx, dev, batch, seqlen)
    parts = list(dy) if isinstance(dy, (list, tuple)) else [dy]
    sizes, rows = [], []
    for p in parts:
        p = _tensor(p, "dy", dtype, dev)
        if p.dim() != 3 or p.shape[:2] != x.shape[:2]:
            raise _b.MambaScanError(2, "dy must be [%d, %d, channels] (got %s)" % (batch, seqlen, list(p.shape)))
        sizes.append(p.shape[2])
        rows.append(_rows(p, "dy", dtype, dev, 2, es))
    _sizes(sizes, channels)
    grads = {"dx": x.new_empty(x.shape), "dweight": torch.empty_like(weight)}
    dbp = dsi = 0
    if bias is not None:
        grads["dbias"] = torch.empty_like(bias)
        dbp = grads["dbias"].data_ptr()
    if state is not None:
        grads["dstate"] = torch.empty_like(state)
        dsi = grads["dstate"].data_ptr()
    ws, ws_bytes, keep = scratch(workspace, lib.mamba_conv_bwd_workspace_bytes(batch, seqlen, channels, taps, io), x)
    launch(dev, "mamba_conv_bwd", lib, lib.mamba_conv_bwd, batch, seqlen, channels, taps, io, act, xp, xs, ip, wp, bp, sp,
           len(rows), _array(ctypes.c_int32, sizes), _array(ctypes.c_void_p, [r[1] for r in rows]),
           _array(ctypes.c_int64, [r[2] for r in rows]), dsp, grads["dx"].data_ptr(), grads["dweight"].data_ptr(), dbp,
           dsi, ws, ws_bytes)
    return grads


def conv_step(x, weight, bias, state, *, activation="silu", split=None, inplace=False, out=None):
    """One token: x [batch, channels], state [batch, channels, taps - 1] float32 (required); weight, bias, activation and
    split as in `conv_fwd`. Functional by default (a new state is returned); with inplace=True the given state is
    updated and returned. Returns (y [batch, channels] or a tuple of its parts, state)."""
    lib = _lib or load()
    io, dtype, dev = _io_of(x, "x")
    act = _act(activation)
    if x.dim() != 2:
        raise _b.MambaScanError(2, "x must be [batch, channels]")
    if state is None:
        raise _b.MambaScanError(1, "conv_step needs a state")
    x, xp, xs = _rows(x, "x", dtype, dev, 1, x.element_size())
    batch, channels = x.shape
    taps, weight, bias, wp, bp = _weights(weight, bias, dev, channels)
    state_shape = (batch, channels, taps - 1)
    if inplace:
        new = check_out(state, "state", state_shape, _F32, x.device)
        sp = np = state.data_ptr()
    else:
        state, sp = _f32(state, "state", dev, state_shape)
        new = x.new_empty(state_shape, dtype=_F32)
        np = new.data_ptr()
    sizes = _sizes(split, channels)
    ys = _outs(x, (batch,), sizes, split, out)
    launch(dev, "mamba_conv_step", lib, lib.mamba_conv_step, batch, channels, taps, io, act, xp, xs, wp, bp, sp, len(ys),
           _array(ctypes.c_int32, sizes), _array(ctypes.c_void_p, [y.data_ptr() for y in ys]), np)
    return ys[0] if split is None else tuple(ys), new


def conv_workspace_bytes(batch, seqlen, channels, taps, dtype):
    """Bytes of workspace `conv_bwd` needs."""
    return int(load().mamba_conv_bwd_workspace_bytes(batch, seqlen, channels, taps, _IO[dtype]))
