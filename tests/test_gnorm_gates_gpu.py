"""The group norm where its activation is far from 0: gates and normed values
that close a channel (down to the lowest value of the type and to -inf) and that
leave it as it is, in every way an activation enters, forwards and backwards,
for groups held by a few lanes, by a workgroup, and read anew by each pass.

silu(z) = z / (1 + e^-z) and its derivative go to 0 towards -inf; that is also
what is expected here at -inf itself, where the products of the formula have no
value.

Bounds as in test_gnorm_gpu.py. An activation's relative error is counted there
for exponents of at most 9 or so; the exponent of e^-z is -z log2 e, off by three
roundings of itself, which is 3 |z| u of e^-z. Below 2^-126 a result may be
flushed to 0."""
import numpy as np
import pytest
import torch

from oracle import gnorm as gn
from tests.test_gnorm_gpu import BF, DT, U, bwd, check, close, fwd, gpu, magnitudes, make, say

pytestmark = pytest.mark.gpu

# lanes of one wave; single elements; a workgroup; read anew (16-byte pieces, single elements)
SHAPES = [(48, 4), (130, 10), (1536, 1), (16384, 1), (16383, 1)]
CLOSED = [-80.0, -200.0, -1e4, -1e30, "lowest"]


def value(v, dtype):
    return torch.finfo(dtype).min if v == "lowest" else v


def some(c, groups, seed):
    """About a third of the channels, never a whole group."""
    m = torch.rand(c, generator=torch.Generator().manual_seed(seed)) < 0.3
    m[::c // groups] = False
    if not m.any():
        m[1] = True
    return m


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("gate", ["after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_closed_gates(shape, dtype, gate, act):
    """A closed channel is 0, and neither its group's statistics nor its gradients see it as anything else."""
    c, groups = shape
    say("closed gates", shape, dtype, gate, act)
    a = make(len(CLOSED), c, groups, DT[dtype], gate, seed=41)
    shut = some(c, groups, 42)
    for row, v in enumerate(CLOSED):
        a["z"][row, shut] = value(v, DT[dtype])
    d = gpu(a)
    kw = dict(activation=act, gate_first=gate == "first", center=gate != "first")
    y, g = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    check(a, y, g, **kw)
    for t in (g["dz"], y if gate == "after" else g["dx"]):
        assert (t[:, shut.cuda()].abs() <= 2.0 ** -100).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_normed_values_far_from_zero(shape, dtype):
    """Without a gate the activation is of the normed value itself, which a bias takes anywhere."""
    c, groups = shape
    for v in CLOSED + [80.0, 200.0, 1e4]:
        a = make(3, c, groups, DT[dtype], "none", seed=43)
        far = some(c, groups, 44)
        a["bias"][far] = value(v, torch.float32)
        d = gpu(a)
        y, g = fwd(d), bwd(d)
        torch.cuda.synchronize()
        say("bias", v)
        if v == "lowest" or v < 0:
            # a normed value moves n by up to 10 or so: silu(-70) and its derivative are below 2^-90
            for t in (y[:, far.cuda()], g["dbias"][far.cuda()], g["dweight"][far.cuda()]):
                assert (t.abs() <= 2.0 ** -90).all()
            # to the others the closed channels are as good as without a gradient
            b = dict(a, dy=a["dy"].masked_fill(far, 0.0), bias=a["bias"].masked_fill(far, 0.0))
            want = gn.oracle_bwd(b["x"], b["weight"], b["bias"], groups, b["dy"])
            close(g["dx"], want["dx"], magnitudes(b)["dx"], b, "dx")
        else:
            check(a, y, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_open_gates(shape, dtype):
    """silu of a large gate is the gate, and its derivative 1."""
    c, groups = shape
    a = make(3, c, groups, DT[dtype], "after", seed=45)
    wide = some(c, groups, 46)
    for row, v in enumerate((80.0, 1e4, 1e30)):
        a["z"][row, wide] = v
    d = gpu(a)
    y, g = fwd(d), bwd(d)
    torch.cuda.synchronize()
    check(a, y, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_small_gates_keep_their_digits(shape, dtype):
    """silu of -85 .. -20 is right relative to itself, not only beside the others."""
    c, groups = shape
    a = make(4, c, groups, DT[dtype], "after", seed=47, affine=False)
    a["z"] = -(20 + 65 * torch.rand(4, c, generator=torch.Generator().manual_seed(48))).to(DT[dtype])
    d = gpu(a)
    y, n = fwd(d), fwd(d, activation="none")
    torch.cuda.synchronize()
    z = a["z"].double().numpy()
    silu = z / (1 + np.exp(-z))
    # activation "none" multiplies by z itself: n, once more rounded
    want = n.cpu().double().numpy() / z * silu
    rel = (3 * np.abs(z) + 80) * U + (2 * BF * (1 + BF) if dtype == "bf16" else 0)
    err = np.abs(y.cpu().double().numpy() - want)
    assert (err <= rel * np.abs(want) + 128 * 2.0 ** -126).all()


@pytest.mark.parametrize("gate", ["after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gates_of_minus_infinity(shape, dtype, gate):
    """A gate of -inf closes as the lowest value does, bit for bit."""
    c, groups = shape
    a = make(3, c, groups, DT[dtype], gate, seed=49)
    shut = some(c, groups, 50)
    kw = dict(gate_first=gate == "first", center=gate != "first")
    out = []
    for v in (torch.finfo(DT[dtype]).min, -float("inf")):
        a["z"][:, shut] = v
        d = gpu(a)
        out.append((fwd(d, **kw), bwd(d, **kw)))
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.isfinite(out[0][0]).all()
    for n in out[0][1]:
        assert torch.equal(out[0][1][n], out[1][1][n]), n


@pytest.mark.parametrize("gate", ["after", "first", "none"])
def test_nan_gates_stay_nan(gate):
    a = make(4, 96, 4, torch.float32, gate, seed=51)
    if gate == "none":
        a["bias"][5] = float("nan")
    else:
        a["z"][:, 5] = float("nan")
    d = gpu(a)
    y, g = fwd(d, gate_first=gate == "first"), bwd(d, gate_first=gate == "first")
    torch.cuda.synchronize()
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, 24:]).all()
    assert torch.isnan(g["dz" if gate != "none" else "dx"][:, 5]).all() and torch.isfinite(g["dx"][:, 24:]).all()
