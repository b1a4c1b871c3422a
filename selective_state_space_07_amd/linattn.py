"""torch-tensor front end of linear attention with a decay for each head in
libmamba_scan (`lin_attn_fwd`, its gradients `lin_attn_bwd`, and
`lin_attn_step` for one token).

Marshalling only: checks devices, dtypes and shapes, passes row strides where
the library can read a tensor in place (columns of one projection's output) and
makes others contiguous, allocates outputs and the workspace, and passes raw
device addresses plus torch's current HIP stream to the entry points of
include/mamba_linattn.h. The arithmetic is all in the library's kernels.
"""
import ctypes
import math

import torch

from . import _binding as _b
from .api import _IO, check_out, check_workspace

EXPORTS = ("mamba_linattn_fwd_workspace_bytes", "mamba_linattn_fwd", "mamba_linattn_bwd_workspace_bytes",
           "mamba_linattn_bwd", "mamba_linattn_step")
_MAX_STRIDE = 1 << 24
_F32 = torch.float32
_lib = None


def load():
    """The scan library with the signatures of include/mamba_linattn.h declared."""
    global _lib
    if _lib is not None:
        return _lib
    lib = _b.load()
    i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    rows = [vp, i64]
    for name in ("mamba_linattn_fwd_workspace_bytes", "mamba_linattn_bwd_workspace_bytes"):
        getattr(lib, name).restype = sz
        getattr(lib, name).argtypes = [i32] * 7
    lib.mamba_linattn_fwd.restype = ctypes.c_int
    lib.mamba_linattn_fwd.argtypes = [i32] * 7 + [f32] + rows * 3 + [vp] * 6 + [sz, vp]
    lib.mamba_linattn_bwd.restype = ctypes.c_int
    lib.mamba_linattn_bwd.argtypes = [i32] * 7 + [f32] + rows * 3 + [vp] * 3 + rows + [vp] * 6 + [sz, vp]
    lib.mamba_linattn_step.restype = ctypes.c_int
    lib.mamba_linattn_step.argtypes = [i32] * 6 + [f32] + rows * 3 + [vp] * 5
    _lib = lib
    return lib


# The current stream's address without the wrapper objects of torch.cuda (a
# call of one token takes few microseconds on the GPU).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _tensor(t, name, dtype, device):
    """Check that t is a tensor of `dtype` on GPU number `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise _b.MambaScanError(7, "%s must be on the GPU (got %s); there is no CPU path" % (name, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.get_device() != device:
        raise _b.MambaScanError(7, "%s is on %s, expected cuda:%d" % (name, t.device, device))
    return t


def _io_of(x, name):
    """(io code, dtype, GPU number) that a call's first io tensor sets for the others."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    io = _IO.get(x.dtype)
    if io is None:
        raise TypeError("io tensors must be float32 or bfloat16 (got %s)" % x.dtype)
    return io, x.dtype, x.get_device() if x.is_cuda else -1


def row_stride(shape, strides, nrow):
    """Elements between consecutive rows of a tensor whose first `nrow` dims number its rows and whose other
    dims are one row's elements in order; 0 where the rows are not so laid out."""
    want = 1
    for n, s in zip(reversed(shape[nrow:]), reversed(strides[nrow:])):
        if n != 1 and s != want:
            return 0
        want *= n
    step = 0
    count = 1
    for n, s in zip(reversed(shape[:nrow]), reversed(strides[:nrow])):
        if n != 1:
            if step == 0:
                step = s // count if s % count == 0 else 0
                if step < want or step > _MAX_STRIDE:
                    return 0
            elif s != step * count:
                return 0
        count *= n
    return step or want


def _rows(t, name, dtype, device, nrow, align):
    """(the tensor or a contiguous copy of it, its address, its row stride), readable in place by the library."""
    t = _tensor(t, name, dtype, device)
    at = t.data_ptr()
    shape = t.shape
    if not at % align:
        if t.is_contiguous():
            return t, at, math.prod(shape[nrow:])
        step = row_stride(shape, t.stride(), nrow)
        if step and not step * t.element_size() % align:
            return t, at, step
    t = t.clone(memory_format=torch.contiguous_format)
    return t, t.data_ptr(), math.prod(shape[nrow:])


def _f32(t, name, device, shape):
    """(a float32 tensor of `shape`, contiguous and 16-byte aligned, its address); (None, 0) for None."""
    if t is None:
        return None, 0
    t = _tensor(t, name, _F32, device)
    if t.shape != shape:
        raise _b.MambaScanError(2, "%s must be %s (got %s)" % (name, list(shape), list(t.shape)))
    at = t.data_ptr()
    if at % 16 or not t.is_contiguous():
        t = t.clone(memory_format=torch.contiguous_format)
        at = t.data_ptr()
    return t, at


def _ids(seq_idx, device, batch, seqlen):
    if seq_idx is None:
        return None, 0
    if isinstance(seq_idx, torch.Tensor) and seq_idx.dtype in (torch.int64, torch.int16, torch.int8, torch.uint8):
        seq_idx = seq_idx.to(torch.int32)
    seq_idx = _tensor(seq_idx, "seq_idx", torch.int32, device)
    if seq_idx.shape != (batch, seqlen):
        raise _b.MambaScanError(2, "seq_idx must be [%d, %d]" % (batch, seqlen))
    seq_idx = seq_idx.contiguous()
    return seq_idx, seq_idx.data_ptr()


def launch(device, what, lib, fn, *args):
    """Call an entry point with GPU number `device` current and its current stream as the last argument."""
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return launch(device, what, lib, fn, *args)
    stream = _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    status = fn(*args, stream)
    if status:
        _b._check(lib, status, what)


def scratch(workspace, need, x):
    """(address, bytes, tensor) of the caller's workspace or, where it is None, of a new one of `need` bytes; on the
    device of x."""
    if workspace is None:
        if not need:
            return 0, 0, None
        workspace = x.new_empty(need, dtype=torch.uint8)
        return workspace.data_ptr(), need, workspace
    workspace = check_workspace(workspace, x.device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _sizes(q, k, v):
    if q.dim() != 4 or v.dim() != 4:
        raise _b.MambaScanError(2, "q and k must be [batch, seqlen, ngroups, d_k] and v [batch, seqlen, nheads, d_v]")
    qs, vs = q.shape, v.shape
    if k.shape != qs or vs[:2] != qs[:2]:
        raise _b.MambaScanError(2, "shape mismatch between q %s, k %s and v %s" % (tuple(qs), tuple(k.shape), tuple(vs)))
    batch, seqlen, ngroups, d_k = qs
    return batch, seqlen, vs[2], ngroups, d_k, vs[3]


def _scale(scale, d_k):
    """The factor of q.k (any number for a d_k of 0, which the library refuses)."""
    return scale if scale is not None else d_k ** -0.5 if d_k else 1.0


def lin_attn_workspace_bytes(batch, seqlen, nheads, ngroups, d_k, d_v, dtype, backward=False):
    """Bytes of workspace `lin_attn_fwd` (or, with `backward`, `lin_attn_bwd`) needs."""
    lib = load()
    fn = lib.mamba_linattn_bwd_workspace_bytes if backward else lib.mamba_linattn_fwd_workspace_bytes
    return int(fn(batch, seqlen, nheads, ngroups, d_k, d_v, _IO[dtype]))


def lin_attn_fwd(q, k, v, log_decay, state=None, *, scale=None, seq_idx=None, out=None, state_out=None,
                 workspace=None, return_state=True):
    """Whole sequence: q, k [batch, seqlen, ngroups, d_k]; v [batch, seqlen, nheads, d_v]; log_decay [nheads]
    float32 (at most 0); state [batch, nheads, d_v, d_k] float32 or None (zeros); scale: a number, d_k ** -0.5 if
    None; seq_idx [batch, seqlen] integer document ids or None (packed documents: the state restarts from zero
    wherever the id changes). q, k and v may be columns of one wider tensor; they are read in place.
    Returns (y like v, final state or None)."""
    lib = _lib or load()
    io, dtype, dev = _io_of(q, "q")
    q, qp, qs = _rows(q, "q", dtype, dev, 2, 16)
    k, kp, ks = _rows(k, "k", dtype, dev, 2, 16)
    v, vp, vs = _rows(v, "v", dtype, dev, 2, 16)
    batch, seqlen, nheads, ngroups, d_k, d_v = sizes = _sizes(q, k, v)
    state_shape = (batch, nheads, d_v, d_k)
    log_decay, gp = _f32(log_decay, "log_decay", dev, (nheads,))
    state, sp = _f32(state, "state", dev, state_shape)
    seq_idx, ip = _ids(seq_idx, dev, batch, seqlen)
    y = q.new_empty(v.shape) if out is None else check_out(out, "out", v.shape, dtype, q.device)
    if state_out is not None:
        check_out(state_out, "state_out", state_shape, _F32, q.device)
    elif return_state:
        state_out = q.new_empty(state_shape, dtype=_F32)
    ws, ws_bytes, keep = scratch(workspace, lib.mamba_linattn_fwd_workspace_bytes(*sizes, io), q)
    launch(dev, "mamba_linattn_fwd", lib, lib.mamba_linattn_fwd, *sizes, io, _scale(scale, d_k),
           qp, qs, kp, ks, vp, vs, ip, gp, sp, y.data_ptr(), 0 if state_out is None else state_out.data_ptr(), ws,
           ws_bytes)
    return y, state_out


def lin_attn_bwd(q, k, v, log_decay, dy, state=None, dstate=None, *, scale=None, seq_idx=None, workspace=None):
    """Gradients of `lin_attn_fwd` given dy = dL/dy (like v) and dstate = dL/d(final state) ([batch, nheads, d_v, d_k]
    float32, or None for zeros); the other arguments are the forward's.

    Returns a dict: dq, dk, dv (dtype and shape of q, k, v; dq and dk are summed over the heads of a group) and,
    where a state is given, dstate (float32, its gradient). The decays are constants: they get no gradient."""
    lib = _lib or load()
    io, dtype, dev = _io_of(q, "q")
    q, qp, qs = _rows(q, "q", dtype, dev, 2, 16)
    k, kp, ks = _rows(k, "k", dtype, dev, 2, 16)
    v, vp, vs = _rows(v, "v", dtype, dev, 2, 16)
    dy, dyp, dys = _rows(dy, "dy", dtype, dev, 2, 16)
    batch, seqlen, nheads, ngroups, d_k, d_v = sizes = _sizes(q, k, v)
    if dy.shape != v.shape:
        raise _b.MambaScanError(2, "dy must be %s (got %s)" % (list(v.shape), list(dy.shape)))
    state_shape = (batch, nheads, d_v, d_k)
    log_decay, gp = _f32(log_decay, "log_decay", dev, (nheads,))
    state, sp = _f32(state, "state", dev, state_shape)
    dstate, dsp = _f32(dstate, "dstate", dev, state_shape)
    seq_idx, ip = _ids(seq_idx, dev, batch, seqlen)
    dq, dk, dv = q.new_empty(q.shape), q.new_empty(q.shape), q.new_empty(v.shape)
    grads = {"dq": dq, "dk": dk, "dv": dv}
    dsi = 0
    if state is not None:
        grads["dstate"] = q.new_empty(state_shape, dtype=_F32)
        dsi = grads["dstate"].data_ptr()
    ws, ws_bytes, keep = scratch(workspace, lib.mamba_linattn_bwd_workspace_bytes(*sizes, io), q)
    launch(dev, "mamba_linattn_bwd", lib, lib.mamba_linattn_bwd, *sizes, io, _scale(scale, d_k),
           qp, qs, kp, ks, vp, vs, ip, gp, sp, dyp, dys, dsp, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dsi, ws,
           ws_bytes)
    return grads


def lin_attn_step(q, k, v, log_decay, state, *, scale=None, inplace=False, out=None):
    """One token: q, k [batch, ngroups, d_k], v [batch, nheads, d_v], state [batch, nheads, d_v, d_k] float32
    (required). Functional by default (a new state is returned); with inplace=True the given state is updated and
    returned. Returns (y like v, state)."""
    lib = _lib or load()
    io, dtype, dev = _io_of(q, "q")
    es = q.element_size()
    q, qp, qs = _rows(q, "q", dtype, dev, 1, es)
    k, kp, ks = _rows(k, "k", dtype, dev, 1, es)
    v, vp, vs = _rows(v, "v", dtype, dev, 1, es)
    if state is None:
        raise _b.MambaScanError(1, "lin_attn_step needs a state")
    if q.dim() != 3 or v.dim() != 3:
        raise _b.MambaScanError(2, "q and k must be [batch, ngroups, d_k] and v [batch, nheads, d_v]")
    q_shape, v_shape = q.shape, v.shape
    if k.shape != q_shape or v_shape[0] != q_shape[0]:
        raise _b.MambaScanError(2, "shape mismatch between q %s, k %s and v %s" % (tuple(q_shape), tuple(k.shape),
                                                                                 tuple(v_shape)))
    batch, ngroups, d_k = q_shape
    nheads, d_v = v_shape[1:]
    state_shape = (batch, nheads, d_v, d_k)
    log_decay, gp = _f32(log_decay, "log_decay", dev, (nheads,))
    if inplace:
        new = check_out(state, "state", state_shape, _F32, q.device)
        sp = np = state.data_ptr()
    else:
        state, sp = _f32(state, "state", dev, state_shape)
        new = q.new_empty(state_shape, dtype=_F32)
        np = new.data_ptr()
    y = q.new_empty(v_shape) if out is None else check_out(out, "out", v_shape, dtype, q.device)
    launch(dev, "mamba_linattn_step", lib, lib.mamba_linattn_step, batch, nheads, ngroups, d_k, d_v, io,
           _scale(scale, d_k), qp, qs, kp, ks, vp, vs, gp, sp, y.data_ptr(), np)
    return y, new
