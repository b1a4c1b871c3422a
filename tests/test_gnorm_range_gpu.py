"""The group norm on the GPU over values whose squares, or whose sum, leave
float32. Scaled by a power of two, values that large are ordinary ones, and all
that follows is scaled exactly: outputs are bit for bit those of the ordinary
values without an eps (which is nothing beside them), dx is smaller by the same
power (to a step of what float32 holds there), and the parameters' gradients are
the same."""
import numpy as np
import pytest
import torch

from oracle import gnorm as gn
from tests.test_gnorm_gpu import BF, DT, U, bwd, fwd, gpu, make, say

pytestmark = pytest.mark.gpu

# lanes of one wave; single elements, few and many a lane; a workgroup; read anew (16-byte pieces, single elements)
SHAPES = [(48, 4), (130, 10), (600, 2), (1536, 1), (2500, 1), (16384, 1), (16383, 1)]


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [66, 124])
def test_large_values(power, shape, dtype, gate):
    c, groups = shape
    say("large", power, shape, dtype, gate)
    a = make(9, c, groups, DT[dtype], gate, seed=91)
    big = torch.ones(9, 1)
    big[[1, 4, 5, 8]] = 2.0 ** power  # beside ordinary rows, in the same waves
    for center in (True, False):
        kw = dict(gate_first=gate == "first", center=center)
        d, e = gpu(a), gpu(dict(a, x=(a["x"].float() * big).to(DT[dtype])))
        large = big[:, 0] > 1
        y, g = fwd(e, **kw), bwd(e, **kw)
        y0, g0 = fwd(d, eps=0.0, **kw), bwd(d, eps=0.0, **kw)
        y1, g1 = fwd(d, **kw), bwd(d, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y[large], y0[large]) and torch.equal(y[~large], y1[~large])
        # what lies below 2^-126 is held in steps of 2^-149 (bfloat16: 2^-133), and rounded to one on its way
        step = (2.0 ** -149 if dtype == "f32" else 2.0 ** -133) if power > 100 else 0.0
        assert ((g["dx"][large].double() * 2.0 ** power - g0["dx"][large].double()).abs() <= step * 2.0 ** power).all()
        assert torch.equal(g["dx"][~large], g1["dx"][~large])
        if gate != "none":
            assert torch.equal(g["dz"][large], g0["dz"][large]) and torch.equal(g["dz"][~large], g1["dz"][~large])
        # sums over rows of both kinds: the terms are those of the two calls
        b = {n: t[large.cuda()] if n in ("x", "z", "dy") and t is not None else t for n, t in d.items()}
        o = {n: t[~large.cuda()] if n in ("x", "z", "dy") and t is not None else t for n, t in d.items()}
        gb, go = bwd(b, eps=0.0, **kw), bwd(o, **kw)
        for n in ("dweight", "dbias"):
            torch.testing.assert_close(g[n], gb[n] + go[n], rtol=16 * U, atol=64 * U * float(g[n].abs().max()))


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [-60, -74, -100])
def test_small_values_without_eps(power, shape, dtype, gate):
    """Values whose squares lose bits, or vanish, beside ordinary ones and a row of zeros (0 / 0)."""
    c, groups = shape
    say("small", power, shape, dtype, gate)
    a = make(9, c, groups, DT[dtype], gate, seed=93)
    little = torch.ones(9, 1)
    little[[1, 4, 5, 8]] = 2.0 ** power
    small = little[:, 0] < 1
    for center in (True, False):
        kw = dict(gate_first=gate == "first", center=center, eps=0.0)
        d, e = gpu(a), gpu(dict(a, x=(a["x"].float() * little).to(DT[dtype])))
        y, g = fwd(e, **kw), bwd(e, **kw)
        y0, g0 = fwd(d, **kw), bwd(d, **kw)
        e["x"][2] = 0
        y2 = fwd(e, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.isfinite(y).all()
        assert torch.equal(g["dx"][small].double() * 2.0 ** power, g0["dx"][small].double())
        assert torch.equal(g["dx"][~small], g0["dx"][~small])
        for n in ("dweight", "dbias", "dz"):
            assert n not in g or torch.equal(g[n], g0[n]), n
        assert torch.isnan(y2[2]).all() and torch.equal(y2[3:], y[3:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_at_the_ends_of_the_type(shape, dtype):
    """A row of the lowest value, one of the highest, one with a single lowest value, one of both in turn."""
    c, groups = shape
    a = make(6, c, groups, DT[dtype], "after", seed=92)
    f = torch.finfo(DT[dtype])
    a["x"][0], a["x"][1], a["x"][2, 3], a["x"][3, ::2], a["x"][3, 1::2] = f.min, f.max, f.min, f.min, f.max
    d = gpu(a)
    for center in (True, False):
        y, g = fwd(d, center=center), bwd(d, center=center)
        torch.cuda.synchronize()
        got = y.cpu().double().numpy()
        want = gn.oracle_fwd(a["x"], a["weight"], a["bias"], groups, a["z"], center=center)
        assert np.isfinite(got).all() and all(torch.isfinite(t).all() for t in g.values())
        hat = np.abs(gn._norm(gn.f64(a["x"]), None, None, groups, None, 1e-5, "silu", False, center)[0])
        size = ((1 + hat) * np.abs(gn.f64(a["weight"])) + np.abs(gn.f64(a["bias"]))) * (1 + np.abs(gn.f64(a["z"])))
        # Rows 0 and 1, centered, are all mean. A bfloat16 value times any number of channels, and its division, are
        # exact in float32: the bias alone is left. Of a float32 one its sum's rounding may be left, over itself.
        rows = slice(2 if center and dtype == "f32" else 0, 6)
        tol = (c // groups + 80) * 2 * U * size + (BF * np.abs(want) if dtype == "bf16" else 0)
        assert (np.abs(got - want) <= tol)[rows].all(), center
