"""fp64 CPU oracle of the RMS norm with the residual's addition, of its 8-bit
output and of its gradients.

TEST INFRASTRUCTURE ONLY: the test suite uses it; the HIP product path never
imports it and shares no code with it. Inputs are upcast to float64 (exact for
fp32 and bf16 values).
"""
import numpy as np

from .linattn import f64


def oracle_fwd(x, residual, weight, eps=1e-5):
    """Returns float64 (y, h)."""
    h = f64(x) if residual is None else f64(x) + f64(residual)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * f64(weight)), h


def oracle_scales(y, block=None):
    """The scales [..., blocks] of float64 outputs y, and the scale of each of its elements."""
    n = y.shape[-1]
    block = block or n
    scales = np.stack([np.abs(y[..., i:i + block]).max(-1) for i in range(0, n, block)], -1) / 448.0
    scales = np.where(scales == 0, 1.0, np.maximum(scales, 2.0 ** -126))
    return scales, np.repeat(scales, block, -1)[..., :n]


def oracle_bwd(h, weight, dy, dh=None, eps=1e-5):
    """Gradients as a dict: d (of x and of the residual), dweight."""
    h, dy = f64(h), f64(dy)
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    hat = h * r
    dn = dy if weight is None else dy * f64(weight)
    d = r * (dn - hat * (dn * hat).mean(-1, keepdims=True))
    return {"d": d if dh is None else d + f64(dh),
            "dweight": (dy * hat).reshape(-1, h.shape[-1]).sum(0)}
