"""fp64 CPU oracle of the gradients of the Mamba-2 SSD scan.

TEST INFRASTRUCTURE ONLY: the test suite uses it; the HIP product path never
imports it and shares no code with it.

Token by token: the states S forwards, and from the last token to the first
R_t = dy_t C_t^T + a_{t+1} R_{t+1}, the gradient of S_t; then dC = S^T dy,
dB = delta R^T x, dx = delta R B + D dy, and of the decay's exponent
g_t = a_t <R_t, S_{t-1}>, so that ddelta = x . R B + A g. Inputs are upcast to
float64 (exact for fp32 and bf16 values).
"""
import numpy as np

from .linattn import f64


def oracle_ssd_bwd(x, dt, B, C, dt_bias, A, D, dy, state=None, dstate=None, seq_idx=None, magnitudes=False):
    """The arguments of ssd_bwd. Returns a dict of float64: dx, ddt, dB, dC, ddt_bias, dA, dD, dstate. With `magnitudes`
    the sums of the absolute values of all terms instead, and beside them g, and the tokens' terms `inside` whose running
    sums g may be taken from, all at least as large as what they bound."""
    x, dt, B, C, dt_bias, A, D, dy = map(f64, (x, dt, B, C, dt_bias, A, D, dy))
    batch, L, H, P = x.shape
    G, N = B.shape[2:]
    rep = H // G
    v = dt + dt_bias
    delta = np.logaddexp(0.0, v)
    decay = np.exp(delta * A)
    sig = 1 / (1 + np.exp(-v))
    if magnitudes:
        x, B, C, dy, A, D = map(np.abs, (x, B, C, dy, A, D))
        state, dstate = (None if s is None else np.abs(f64(s)) for s in (state, dstate))
    Bh, Ch = np.repeat(B, rep, 2), np.repeat(C, rep, 2)
    keep = np.ones((L, batch, 1, 1, 1))  # 0 where a document begins
    if seq_idx is not None:
        ids = f64(seq_idx)
        keep[1:, :, 0, 0, 0] = (ids[:, 1:] == ids[:, :-1]).T
    a = decay.transpose(1, 0, 2)[..., None, None] * keep
    start = np.zeros((batch, H, P, N)) if state is None else f64(state)
    before, S, dC = [], start, np.empty((batch, L, H, N))
    for t in range(L):
        S = np.where(keep[t] > 0, a[t] * S, 0.0)
        before.append(S)  # the decayed state that the token's input is added to
        S = S + (delta[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None]
        dC[:, t] = np.einsum("bhpn,bhp->bhn", S, dy[:, t])
    R = np.zeros((batch, H, P, N)) if dstate is None else f64(dstate)
    dB, RB, g = np.empty_like(dC), np.empty_like(x), np.empty_like(delta)
    for t in reversed(range(L)):
        R = R + dy[:, t][..., None] * Ch[:, t, :, None]
        dB[:, t] = delta[:, t, :, None] * np.einsum("bhpn,bhp->bhn", R, x[:, t])
        RB[:, t] = np.einsum("bhpn,bhn->bhp", R, Bh[:, t])
        g[:, t] = (R * before[t]).sum((-1, -2))
        R = np.where(keep[t] > 0, a[t] * R, 0.0)
    direct = (RB * x).sum(-1)
    ddt = (direct + A * g) * sig
    shared = lambda q: q.reshape(batch, L, G, rep, N).sum(3)  # noqa: E731
    got = {"dx": delta[..., None] * RB + D[:, None] * dy, "ddt": ddt, "dB": shared(dB), "dC": shared(dC),
           "ddt_bias": ddt.sum((0, 1)), "dA": (g * delta).sum((0, 1)), "dD": (dy * x).sum((0, 1, 3)), "dstate": R}
    if magnitudes:
        got.update(g=g, inside=(dC * Ch).sum(-1) + delta * direct, delta=delta, sig=sig, v=v)
    return got
