"""fp64 CPU oracle of linear attention with a decay for each head, and of its
gradients.

TEST INFRASTRUCTURE ONLY: the test suite uses it; the HIP product path never
imports it and shares no code with it.

Token by token, with the state S [d_v, d_k] of each head: S = lam S + v k^T,
y = scale S q, and for the gradients, from the last token to the first,
R = lam R + scale dy q^T, dk = R^T v, dv = R k, and dq = scale S^T dy. Inputs
are upcast to float64 (exact for fp32 and bf16 values).
"""
import numpy as np


def f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().cpu().double().numpy()
    return np.asarray(a, dtype=np.float64)


def _heads(t, nheads):
    return np.repeat(t, nheads // t.shape[2], axis=2)


def _keep(seq_idx, batch, seqlen):
    """[seqlen, batch, 1, 1, 1]: 0 where a document begins, else 1 (the first token continues the incoming state)."""
    keep = np.ones((seqlen, batch, 1, 1, 1))
    if seq_idx is not None:
        ids = f64(seq_idx)
        keep[1:, :, 0, 0, 0] = (ids[:, 1:] == ids[:, :-1]).T
    return keep


def _start(state, batch, nheads, d_v, d_k):
    return np.zeros((batch, nheads, d_v, d_k)) if state is None else f64(state).copy()


def oracle_fwd(q, k, v, log_decay, state=None, scale=None, seq_idx=None):
    """q, k [batch, seqlen, ngroups, d_k], v [batch, seqlen, nheads, d_v], log_decay [nheads], state [batch, nheads,
    d_v, d_k] or None. Returns float64 (y like v, final state)."""
    q, k, v = f64(q), f64(k), f64(v)
    batch, seqlen, nheads, d_v = v.shape
    d_k = q.shape[3]
    scale = d_k ** -0.5 if scale is None else scale
    q, k = _heads(q, nheads), _heads(k, nheads)
    lam = np.exp(f64(log_decay))[None, :, None, None]
    keep = _keep(seq_idx, batch, seqlen)
    S = _start(state, batch, nheads, d_v, d_k)
    y = np.empty_like(v)
    for t in range(seqlen):
        # chosen, not multiplied: what stood before a document's first token is gone, whatever it was
        S = np.where(keep[t] > 0, lam * S, 0.0) + v[:, t, :, :, None] * k[:, t, :, None, :]
        y[:, t] = scale * (S * q[:, t, :, None, :]).sum(-1)
    return y, S


def oracle_step(q, k, v, log_decay, state, scale=None):
    y, S = oracle_fwd(f64(q)[:, None], f64(k)[:, None], f64(v)[:, None], log_decay, state, scale)
    return y[:, 0], S


def oracle_bwd(q, k, v, log_decay, dy, state=None, dstate=None, scale=None, seq_idx=None):
    """Gradients as a dict: dq, dk (summed over each group's heads), dv, dstate (of the incoming state)."""
    q, k, v, dy = f64(q), f64(k), f64(v), f64(dy)
    batch, seqlen, nheads, d_v = v.shape
    ngroups, d_k = q.shape[2:]
    scale = d_k ** -0.5 if scale is None else scale
    qh, kh = _heads(q, nheads), _heads(k, nheads)
    lam = np.exp(f64(log_decay))[None, :, None, None]
    keep = _keep(seq_idx, batch, seqlen)
    S = _start(state, batch, nheads, d_v, d_k)
    dq, dk, dv = np.empty_like(qh), np.empty_like(kh), np.empty_like(v)
    for t in range(seqlen):
        S = lam * keep[t] * S + v[:, t, :, :, None] * kh[:, t, :, None, :]
        dq[:, t] = scale * (S * dy[:, t, :, :, None]).sum(-2)
    R = _start(dstate, batch, nheads, d_v, d_k)
    for t in reversed(range(seqlen)):
        R = R + scale * dy[:, t, :, :, None] * qh[:, t, :, None, :]
        dk[:, t] = (R * v[:, t, :, :, None]).sum(-2)
        dv[:, t] = (R * kh[:, t, :, None, :]).sum(-1)
        R = lam * keep[t] * R
    shared = lambda a: a.reshape(batch, seqlen, ngroups, nheads // ngroups, d_k).sum(3)  # noqa: E731
    return {"dq": shared(dq), "dk": shared(dk), "dv": dv, "dstate": R}
