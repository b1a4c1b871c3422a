"""fp64 CPU oracle of the short causal convolution and of its gradients.

TEST INFRASTRUCTURE ONLY: the test suite uses it; the HIP product path never
imports it and shares no code with it.

Token by token, with the window of the last taps - 1 inputs, which is emptied
where a document begins: u = bias + sum of tap times input, y = silu(u) or u.
The gradients go back through the same windows. Inputs are upcast to float64
(exact for fp32 and bf16 values).
"""
import numpy as np

from .linattn import f64


def sigmoid(u):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-u))


def act(u, kind):
    return u * sigmoid(u) if kind == "silu" else u


def act_grad(u, kind):
    s = sigmoid(u)
    return s * (1 + u * (1 - s)) if kind == "silu" else np.ones_like(u)


def _begins(seq_idx, batch, seqlen):
    """[seqlen, batch]: a document begins at this token (the first one continues the state)."""
    begins = np.zeros((seqlen, batch), dtype=bool)
    if seq_idx is not None:
        ids = f64(seq_idx)
        begins[1:] = (ids[:, 1:] != ids[:, :-1]).T
    return begins


def _start(state, batch, channels, past):
    return np.zeros((batch, channels, past)) if state is None else f64(state).copy()


def oracle_fwd(x, weight, bias=None, state=None, seq_idx=None, activation="silu"):
    """x [batch, seqlen, channels], weight [channels, taps], state [batch, channels, taps - 1] (oldest first) or None.
    Returns float64 (y, final state)."""
    x, weight = f64(x), f64(weight)
    batch, seqlen, channels = x.shape
    past = weight.shape[1] - 1
    begins = _begins(seq_idx, batch, seqlen)
    window = _start(state, batch, channels, past)
    y = np.empty_like(x)
    for t in range(seqlen):
        window = np.where(begins[t][:, None, None], 0.0, window)
        full = np.concatenate([window, x[:, t, :, None]], 2)
        u = (full * weight).sum(2) + (0.0 if bias is None else f64(bias))
        y[:, t] = act(u, activation)
        window = full[:, :, 1:]
    return y, window


def oracle_step(x, weight, bias, state, activation="silu"):
    y, new = oracle_fwd(f64(x)[:, None], weight, bias, state, None, activation)
    return y[:, 0], new


def oracle_bwd(x, weight, dy, bias=None, state=None, dstate=None, seq_idx=None, activation="silu"):
    """Gradients as a dict: dx, dweight, dbias, dstate (of the incoming state)."""
    x, weight, dy = f64(x), f64(weight), f64(dy)
    batch, seqlen, channels = x.shape
    past = weight.shape[1] - 1
    begins = _begins(seq_idx, batch, seqlen)
    windows = []
    window = _start(state, batch, channels, past)
    for t in range(seqlen):
        window = np.where(begins[t][:, None, None], 0.0, window)
        windows.append(np.concatenate([window, x[:, t, :, None]], 2))
        window = windows[-1][:, :, 1:]
    dx, dweight, dbias = np.empty_like(x), np.zeros_like(weight), np.zeros(channels)
    back = _start(dstate, batch, channels, past)  # gradient of the window behind the token
    for t in reversed(range(seqlen)):
        u = (windows[t] * weight).sum(2) + (0.0 if bias is None else f64(bias))
        du = dy[:, t] * act_grad(u, activation)
        dweight += (du[:, :, None] * windows[t]).sum(0)
        dbias += du.sum(0)
        full = du[:, :, None] * weight
        full[:, :, 1:] += back
        dx[:, t] = full[:, :, past]
        back = np.where(begins[t][:, None, None], 0.0, full[:, :, :past])
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dstate": back}
