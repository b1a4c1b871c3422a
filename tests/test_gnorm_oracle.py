"""The fp64 oracle of the gated group norm against torch's float64 functions,
autograd and central differences."""
import itertools

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import gnorm as gn

ACT = {"none": lambda t: t, "silu": F.silu, "sigmoid": torch.sigmoid}


@pytest.mark.parametrize("act,gate,center", itertools.product(ACT, ["none", "after", "first"], [True, False]))
def test_against_torch(act, gate, center):
    r = torch.Generator().manual_seed(1)
    x, z, dy = (torch.randn(6, 12, generator=r, dtype=torch.float64, requires_grad=True) for _ in range(3))
    w, b = (torch.randn(12, generator=r, dtype=torch.float64, requires_grad=True) for _ in range(2))
    u = x * ACT[act](z) if gate == "first" else x
    if center:
        n = F.group_norm(u, 3, w, b, 1e-5)
    else:
        v = u.unflatten(1, (3, 4))
        n = (v * torch.rsqrt(v.pow(2).mean(-1, keepdim=True) + 1e-5)).flatten(1) * w + b
    y = n * ACT[act](z) if gate == "after" else ACT[act](n) if gate == "none" else n
    kw = dict(activation=act, gate_first=gate == "first", center=center)
    zz = None if gate == "none" else z
    np.testing.assert_allclose(gn.oracle_fwd(x, w, b, 3, zz, **kw), y.detach().numpy(), rtol=1e-12, atol=1e-13)
    got = gn.oracle_bwd(x, w, b, 3, dy, zz, **kw)
    leaves = {"x": x, "weight": w, "bias": b, **({} if zz is None else {"z": z})}
    want = torch.autograd.grad(y, list(leaves.values()), dy.detach())
    assert set(got) == {"d" + n for n in leaves}
    for name, t in zip(leaves, want):
        np.testing.assert_allclose(got["d" + name], t.numpy(), rtol=1e-9, atol=1e-11, err_msg=name)
    # central differences along a random direction
    for name, t in leaves.items():
        d = torch.randn(t.shape, generator=r, dtype=torch.float64)
        at = lambda s: {n: (v + s * d if n == name else v).detach() for n, v in leaves.items()}  # noqa: E731
        f = lambda s: (gn.oracle_fwd(at(s)["x"], at(s)["weight"], at(s)["bias"], 3, at(s).get("z"), **kw)  # noqa: E731
                       * dy.detach().numpy()).sum()
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs(slope - (got["d" + name] * d.numpy()).sum()) < 1e-6 * (1 + abs(slope)), name
