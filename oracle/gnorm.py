"""fp64 CPU oracle of the group norm with an activation and a gate.

TEST INFRASTRUCTURE ONLY: the test suite uses it; the HIP product path never
imports it and shares no code with it. Gradients are written out, not taken by
differentiation; inputs are upcast to float64.
"""
import numpy as np

from .linattn import f64


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def act(kind, z):
    return z if kind == "none" else z * sigmoid(z) if kind == "silu" else sigmoid(z)


def act_grad(kind, z):
    if kind == "none":
        return np.ones_like(z)
    s, c = sigmoid(z), sigmoid(-z)
    return s * (1 + z * c) if kind == "silu" else s * c


def _norm(x, weight, bias, groups, z, eps, activation, gate_first, center):
    c = x.shape[-1]
    u = x * act(activation, z) if gate_first else x
    u = u.reshape(-1, groups, c // groups)
    if center:
        u = u - u.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    hat = (u * r).reshape(x.shape)
    n = hat * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return hat, r, n


def oracle_fwd(x, weight, bias, groups, z=None, eps=1e-5, activation="silu", gate_first=False, center=True):
    x, z, weight, bias = f64(x), f64(z), f64(weight), f64(bias)
    _, _, n = _norm(x, weight, bias, groups, z, eps, activation, gate_first, center)
    if z is None:
        return act(activation, n)
    return n if gate_first else n * act(activation, z)


def oracle_bwd(x, weight, bias, groups, dy, z=None, eps=1e-5, activation="silu", gate_first=False, center=True):
    """A dict: dx, dz (where z is given), dweight, dbias."""
    x, z, weight, bias, dy = f64(x), f64(z), f64(weight), f64(bias), f64(dy)
    hat, r, n = _norm(x, weight, bias, groups, z, eps, activation, gate_first, center)
    dn, dz = dy, None
    if z is None:
        dn = dy * act_grad(activation, n)
    elif not gate_first:
        dn = dy * act(activation, z)
        dz = dy * n * act_grad(activation, z)
    c = x.shape[-1]
    dhat = (dn * (1.0 if weight is None else weight)).reshape(-1, groups, c // groups)
    h = hat.reshape(dhat.shape)
    du = dhat - h * (dhat * h).mean(-1, keepdims=True)
    if center:
        du = du - dhat.mean(-1, keepdims=True)
    du = (du * r).reshape(x.shape)
    if gate_first:
        dz = du * x * act_grad(activation, z)
        du = du * act(activation, z)
    g = {"dx": du, "dweight": (dn * hat).reshape(-1, c).sum(0), "dbias": dn.reshape(-1, c).sum(0)}
    return g if z is None else dict(g, dz=dz)
