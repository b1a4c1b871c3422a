"""torch-tensor front end of the Mamba-2 SSD scan in libmamba_scan (`ssd_fwd`,
its gradients `ssd_bwd`, and `ssd_step` for one token).

Marshalling only: checks devices, dtypes and shapes, makes tensors contiguous,
allocates outputs and the workspace, and passes raw device addresses plus
torch's current HIP stream to mamba2_ssd_fwd. The arithmetic is all in the
library's kernels.
"""
import torch

from . import _binding as _b
from .api import _IO, _addr, _dev, _io, check_out, check_workspace
from .linattn import _f32, _ids, _io_of, _rows, launch, scratch


def ssd_workspace_bytes(batch, seqlen, nheads, headdim, d_state, ngroups, dtype):
    return _b.mamba2_ssd_fwd_workspace_bytes(batch, seqlen, nheads, headdim, d_state, ngroups, _IO[dtype])


def ssd_fwd(x, dt, B, C, dt_bias, A, D, state=None, *, out=None, state_out=None, workspace=None,
            return_state=True, seq_idx=None):
    """x [batch, seqlen, nheads, headdim]; dt [batch, seqlen, nheads] (before dt_bias and
    softplus); B, C [batch, seqlen, ngroups, d_state]; dt_bias, A, D [nheads] float32;
    state [batch, nheads, headdim, d_state] float32 or None; seq_idx [batch, seqlen]
    integer document ids or None (packed documents: the state restarts from zero
    wherever the id changes, mamba2_ssd_fwd_seq).
    Returns (y like x, final state or None)."""
    io = _io(x)
    dtype = x.dtype
    x, dt = _dev(x, "x", dtype), _dev(dt, "dt", dtype)
    B, C = _dev(B, "B", dtype), _dev(C, "C", dtype)
    f32 = torch.float32
    dt_bias, A, D = _dev(dt_bias, "dt_bias", f32), _dev(A, "A", f32), _dev(D, "D", f32)
    state = _dev(state, "state", f32)
    if x.dim() != 4 or B.dim() != 4:
        raise _b.MambaScanError(2, "x must be [batch, seqlen, nheads, headdim] and B [batch, seqlen, ngroups, d_state]")
    batch, seqlen, nheads, headdim = x.shape
    ngroups, d_state = B.shape[2], B.shape[3]
    if dt.shape != (batch, seqlen, nheads) or C.shape != B.shape or B.shape[:2] != (batch, seqlen):
        raise _b.MambaScanError(2, "shape mismatch between x %s, dt %s and B/C %s" % (tuple(x.shape), tuple(dt.shape),
                                                                                    tuple(B.shape)))
    if dt_bias.shape != (nheads,) or A.shape != (nheads,) or D.shape != (nheads,):
        raise _b.MambaScanError(2, "dt_bias, A and D must be [%d]" % nheads)
    if state is not None and state.shape != (batch, nheads, headdim, d_state):
        raise _b.MambaScanError(2, "state must be [%d, %d, %d, %d]" % (batch, nheads, headdim, d_state))
    y = check_out(out, "out", x.shape, dtype, x.device) if out is not None else torch.empty_like(x)
    if state_out is not None:
        check_out(state_out, "state_out", (batch, nheads, headdim, d_state), f32, x.device)
    if return_state and state_out is None:
        state_out = torch.empty(batch, nheads, headdim, d_state, device=x.device, dtype=f32)
    workspace = check_workspace(workspace, x.device)
    ws_need = _b.mamba2_ssd_fwd_workspace_bytes(batch, seqlen, nheads, headdim, d_state, ngroups, io)
    if workspace is None and ws_need:
        workspace = torch.empty(ws_need, device=x.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    stream = torch.cuda.current_stream(x.device).cuda_stream
    if seq_idx is None:
        _b.mamba2_ssd_fwd(batch, seqlen, nheads, headdim, d_state, ngroups, io, _addr(x), _addr(dt), _addr(B),
                          _addr(C), _addr(dt_bias), _addr(A), _addr(D), _addr(state), _addr(y), _addr(state_out),
                          _addr(workspace), ws_bytes, stream)
    else:
        if isinstance(seq_idx, torch.Tensor) and seq_idx.dtype in (torch.int64, torch.int16, torch.int8, torch.uint8):
            seq_idx = seq_idx.to(torch.int32)
        seq_idx = _dev(seq_idx, "seq_idx", torch.int32)
        if seq_idx.shape != (batch, seqlen):
            raise _b.MambaScanError(2, "seq_idx must be [%d, %d]" % (batch, seqlen))
        _b.mamba2_ssd_fwd_seq(batch, seqlen, nheads, headdim, d_state, ngroups, io, _addr(x), _addr(dt), _addr(B),
                              _addr(C), _addr(seq_idx), _addr(dt_bias), _addr(A), _addr(D), _addr(state), _addr(y),
                              _addr(state_out), _addr(workspace), ws_bytes, stream)
    return y, state_out


def ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, d_state, ngroups, dtype):
    return _b.mamba2_ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, d_state, ngroups, _IO[dtype])


def ssd_bwd(x, dt, B, C, dt_bias, A, D, dy, state=None, dstate=None, *, seq_idx=None, workspace=None):
    """Gradients of `ssd_fwd` given dy = dL/dy (like x) and dstate = dL/d(final state) ([batch, nheads, headdim, d_state]
    float32, or None for zeros); the other arguments are the forward's, with A at most 0. x, dt, B, C and dy may be
    columns of wider tensors; they are read in place.

    Returns a dict: dx, ddt, dB, dC (dtype and shape of x, dt, B, C; dB and dC are summed over the heads of a group),
    ddt_bias, dA, dD ([nheads] float32) and, where a state is given, dstate (float32, its gradient)."""
    lib = _b.load()
    io, dtype, dev = _io_of(x, "x")
    x, xp, xs = _rows(x, "x", dtype, dev, 2, 16)
    dt, dtp, dts = _rows(dt, "dt", dtype, dev, 2, x.element_size())
    B, Bp, Bs = _rows(B, "B", dtype, dev, 2, 16)
    C, Cp, Cs = _rows(C, "C", dtype, dev, 2, 16)
    dy, dyp, dys = _rows(dy, "dy", dtype, dev, 2, 16)
    if x.dim() != 4 or B.dim() != 4:
        raise _b.MambaScanError(2, "x must be [batch, seqlen, nheads, headdim] and B [batch, seqlen, ngroups, d_state]")
    batch, seqlen, nheads, headdim = x.shape
    ngroups, d_state = B.shape[2:]
    if dt.shape != (batch, seqlen, nheads) or C.shape != B.shape or B.shape[:2] != (batch, seqlen) or dy.shape != x.shape:
        raise _b.MambaScanError(2, "shape mismatch between x %s, dy %s, dt %s, B %s and C %s" %
                                tuple(tuple(t.shape) for t in (x, dy, dt, B, C)))
    state_shape = (batch, nheads, headdim, d_state)
    dt_bias, dbp = _f32(dt_bias, "dt_bias", dev, (nheads,))
    A, Ap = _f32(A, "A", dev, (nheads,))
    D, Dp = _f32(D, "D", dev, (nheads,))
    state, sp = _f32(state, "state", dev, state_shape)
    dstate, dsp = _f32(dstate, "dstate", dev, state_shape)
    seq_idx, ip = _ids(seq_idx, dev, batch, seqlen)
    grads = {"dx": x.new_empty(x.shape), "ddt": x.new_empty(dt.shape), "dB": x.new_empty(B.shape),
             "dC": x.new_empty(B.shape)}
    for n in ("ddt_bias", "dA", "dD"):
        grads[n] = x.new_empty(nheads, dtype=torch.float32)
    dsi = 0
    if state is not None:
        grads["dstate"] = x.new_empty(state_shape, dtype=torch.float32)
        dsi = grads["dstate"].data_ptr()
    sizes = (batch, seqlen, nheads, headdim, d_state, ngroups, io)
    ws, ws_bytes, keep = scratch(workspace, lib.mamba2_ssd_bwd_workspace_bytes(*sizes), x)
    launch(dev, "mamba2_ssd_bwd", lib, lib.mamba2_ssd_bwd, *sizes, xp, xs, dtp, dts, Bp, Bs, Cp, Cs, ip, dbp, Ap, Dp, sp,
           dyp, dys, dsp, *(grads[n].data_ptr() for n in ("dx", "ddt", "dB", "dC", "ddt_bias", "dA", "dD")), dsi, ws,
           ws_bytes)
    return grads


def ssd_step(x, dt, B, C, dt_bias, A, D, state, *, inplace=False, out=None):
    """One token: x [batch, nheads, headdim], dt [batch, nheads], B, C [batch, ngroups,
    d_state], state [batch, nheads, headdim, d_state] float32 (required).
    Functional by default (a new state is returned); with inplace=True the given
    state is updated and returned."""
    io = _io(x)
    dtype = x.dtype
    x, dt = _dev(x, "x", dtype), _dev(dt, "dt", dtype)
    B, C = _dev(B, "B", dtype), _dev(C, "C", dtype)
    f32 = torch.float32
    dt_bias, A, D = _dev(dt_bias, "dt_bias", f32), _dev(A, "A", f32), _dev(D, "D", f32)
    if state is None:
        raise _b.MambaScanError(1, "ssd_step needs a state")
    if inplace and not state.is_contiguous():
        raise _b.MambaScanError(2, "in-place step needs a contiguous state tensor")
    state = _dev(state, "state", f32)
    if x.dim() != 3 or B.dim() != 3:
        raise _b.MambaScanError(2, "x must be [batch, nheads, headdim] and B [batch, ngroups, d_state]")
    batch, nheads, headdim = x.shape
    ngroups, d_state = B.shape[1], B.shape[2]
    if dt.shape != (batch, nheads) or C.shape != B.shape or B.shape[0] != batch:
        raise _b.MambaScanError(2, "shape mismatch between x, dt and B/C")
    if dt_bias.shape != (nheads,) or A.shape != (nheads,) or D.shape != (nheads,):
        raise _b.MambaScanError(2, "dt_bias, A and D must be [%d]" % nheads)
    if state.shape != (batch, nheads, headdim, d_state):
        raise _b.MambaScanError(2, "state must be [%d, %d, %d, %d]" % (batch, nheads, headdim, d_state))
    y = check_out(out, "out", x.shape, dtype, x.device) if out is not None else torch.empty_like(x)
    so = state if inplace else torch.empty_like(state)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    _b.mamba2_ssd_step(batch, nheads, headdim, d_state, ngroups, io, _addr(x), _addr(dt), _addr(B), _addr(C),
                       _addr(dt_bias), _addr(A), _addr(D), _addr(state), _addr(y), _addr(so), stream)
    return y, so
