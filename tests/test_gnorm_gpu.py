"""The gated group norm on the GPU against the fp64 oracle: every output at
group sizes that fill a lane's pieces and that do not, one wave and a whole
workgroup per group, each gate, activation and io type, strided and unaligned
rows, rows that hold NaN, graphs.

The bounds are counted, not fitted. With u = 2^-24 and gs channels a group:
a sum over the group is within gs u of the sum of its magnitudes, an
activation within 40 u of itself (three roundings of an exponent of at most 9
or so, and the instructions' own). So the centered value times its reciprocal
deviation is within C u (1 + kappa) (1 + |xh|), C = gs + 80 and kappa the root
mean square of the group before its mean is taken off, over its deviation (the
amplification of the mean's error); what follows multiplies magnitudes. A
bfloat16 output is rounded once more (2^-8 of itself)."""
import sys

import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import gnorm as gn

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make(rows, c, groups, dtype, gate, seed=0, affine=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = dict(x=(rnd(rows, c) + 0.5 * rnd(c)).to(dtype), z=rnd(rows, c).to(dtype) if gate != "none" else None,
             weight=1 + 0.3 * rnd(c) if affine else None, bias=0.3 * rnd(c) if affine else None, groups=groups,
             dy=rnd(rows, c).to(dtype))
    return a


def gpu(a):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in a.items()}


def fwd(a, **kw):
    return ms.group_norm_fwd(a["x"], a["weight"], a["bias"], a["groups"], a["z"], **kw)


def bwd(a, **kw):
    return ms.group_norm_bwd(a["x"], a["weight"], a["bias"], a["groups"], a["dy"], a["z"], **kw)


def magnitudes(a, activation="silu", gate_first=False, center=True, eps=1e-5):
    """What each output's error is counted in units of C u."""
    f = gn.f64
    x, z, dy = f(a["x"]), f(a["z"]), f(a["dy"])
    c, G = x.shape[-1], a["groups"]
    w = np.ones(c) if a["weight"] is None else np.abs(f(a["weight"]))
    b = np.zeros(c) if a["bias"] is None else np.abs(f(a["bias"]))
    ga = np.ones_like(x) if z is None else 1 + np.abs(gn.act(activation, z))
    raw = x * gn.act(activation, z) if gate_first else x
    hat, r, _ = gn._norm(x, None, None, G, z, eps, activation, gate_first, center)
    kappa = np.sqrt((raw.reshape(r.shape[0], G, -1) ** 2).mean(-1, keepdims=True)) * r
    grow = np.broadcast_to(1 + kappa, (r.shape[0], G, c // G)).reshape(x.shape)
    H = (1 + np.abs(hat)) * grow
    n = H * w + b
    after = z is not None and not gate_first
    m = {"y": 1.1 * n * (ga if after else 1)}
    dn = 1.1 * np.abs(dy) * (ga if after else 1) * (1 if z is not None else 1 + n)
    dh = (dn * w).reshape(r.shape[0], G, -1)
    Hg = H.reshape(dh.shape)
    dx = (2 * r * (dh + dh.mean(-1, keepdims=True) + Hg * (dh * Hg).mean(-1, keepdims=True))).reshape(x.shape)
    m["dx"] = dx * (ga if gate_first else 1)
    if z is not None:
        m["dz"] = 1.1 * (dx * np.abs(x) if gate_first else np.abs(dy) * n)
    m["dweight"], m["dbias"] = (dn * H).sum(0), dn.sum(0)
    return m


def close(got, want, size, a, what, rows=0, rounded=True):
    got = got.detach().cpu().double().numpy()
    C = a["x"].shape[-1] // a["groups"] + 80 + rows
    tol = C * U * size + 1e-30
    if rounded and a["x"].dtype == torch.bfloat16:
        tol = tol + BF * np.abs(want)
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    at = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), "%s: %g off at %s, %g allowed" % (what, err[at], at, tol[at])


def check(a, y, grads, **kw):
    args = (a["x"], a["weight"], a["bias"], a["groups"])
    m = magnitudes(a, **kw)
    if y is not None:
        close(y, gn.oracle_fwd(*args, a["z"], **kw), m["y"], a, "y")
    if grads is None:
        return
    want = gn.oracle_bwd(*args, a["dy"], a["z"], **kw)
    names = {"dx"} | ({"dz"} if a["z"] is not None else set())
    names |= ({"dweight"} if a["weight"] is not None else set()) | ({"dbias"} if a["bias"] is not None else set())
    assert set(grads) == names
    for n in grads:
        par = n in ("dweight", "dbias")
        close(grads[n], want[n], m[n], a, n, rows=a["x"].shape[0] if par else 0, rounded=not par)


SHAPES = [
    # rows, channels, groups
    (1, 1, 1), (1, 8, 1), (3, 8, 8), (5, 24, 3), (7, 96, 12), (64, 64, 1), (13, 130, 10), (77, 1000, 8),
    (33, 1536, 12), (9, 1536, 1), (6, 1600, 5), (11, 1028, 1),
    (4, 2500, 2), (2, 2056, 1), (3, 4096, 1), (2, 8192, 1), (3, 16384, 1), (2, 16383, 1),  # a workgroup per group
    (20000, 16, 2), (4100, 48, 1),  # many rows of few channels
]


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_fwd_and_bwd(shape, dtype, gate):
    say("group norm", shape, dtype, gate)
    a = make(*shape, DT[dtype], gate, seed=sum(shape))
    d = gpu(a)
    kw = dict(gate_first=gate == "first", center=gate != "first")
    y, g = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    check(a, y, g, **kw)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
def test_activations(gate, act, center):
    a = make(21, 192, 4, torch.float32, gate, seed=3)
    d = gpu(a)
    kw = dict(activation=act, gate_first=gate == "first", center=center, eps=1e-3)
    y, g = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    check(a, y, g, **kw)


@pytest.mark.parametrize("have", ["weight", "bias", "neither"])
def test_without_parameters(have):
    a = make(40, 96, 3, torch.bfloat16, "after", seed=4)
    a.update({n: None for n in ("weight", "bias") if n != have})
    d = gpu(a)
    y, g = fwd(d), bwd(d)
    torch.cuda.synchronize()
    check(a, y, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_columns_of_one_projection_and_odd_offsets(dtype):
    """x, z and dy as columns of one tensor, aligned and not, and with more leading dims."""
    wide = torch.randn(3, 20, 3 * 192 + 8, generator=torch.Generator().manual_seed(5)).to(DT[dtype]).cuda()
    w, b = torch.randn(192, device="cuda"), torch.randn(192, device="cuda")
    for off in (0, 1, 8):
        x, z, dy = (wide[..., off + i * 192:off + (i + 1) * 192] for i in range(3))
        y = ms.group_norm_fwd(x, w, b, 6, z)
        g = ms.group_norm_bwd(x, w, b, 6, dy, z)
        torch.cuda.synchronize()
        assert y.shape == x.shape
        a = dict(x=x.reshape(60, 192).cpu(), z=z.reshape(60, 192).cpu(), dy=dy.reshape(60, 192).cpu(), weight=w.cpu(),
                 bias=b.cpu(), groups=6)
        check(a, y.view(60, 192), {n: t.view(60, 192) if t.dim() == 3 else t for n, t in g.items()})
    x = wide[..., :192]
    assert torch.equal(ms.group_norm_fwd(x[:, 3], w, b, 6), ms.group_norm_fwd(x[:, 3].contiguous(), w, b, 6))
    assert torch.equal(ms.group_norm_fwd(x.transpose(0, 1), w, b, 6), ms.group_norm_fwd(x, w, b, 6).transpose(0, 1))
    assert torch.equal(ms.group_norm_fwd(x[0, 0], w, b, 6), ms.group_norm_fwd(x, w, b, 6)[0, 0])


@pytest.mark.parametrize("c,groups", [(192, 4), (4096, 1)])
def test_rows_are_their_own(c, groups):
    """NaN and infinities in one row and group stay there; a constant group (deviation 0) gives the bias."""
    a = make(37, c, groups, torch.float32, "after", seed=6)
    d = gpu(a)
    y0, g0 = fwd(d), bwd(d)
    d["x"] = d["x"].clone()
    d["x"][5, 3] = float("nan")
    d["x"][9, 3] = float("inf")
    d["x"][11] = 2.5
    y1, g1 = fwd(d), bwd(d)
    torch.cuda.synchronize()
    rest = [i for i in range(37) if i not in (5, 9, 11)]
    assert torch.equal(y1[rest], y0[rest]) and torch.equal(g1["dx"][rest], g0["dx"][rest])
    gs = c // groups
    assert torch.isnan(y1[5, :gs]).all() and torch.equal(y1[5, gs:], y0[5, gs:])
    want = gn.oracle_fwd(d["x"][11:12].cpu(), a["weight"], a["bias"], groups, a["z"][11:12])
    assert np.allclose(y1[11].cpu().numpy(), want[0], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 17])
def test_eps_zero_and_rows_that_do_not_fill_a_wave(rows):
    a = make(rows, 40, 5, torch.float32, "none", seed=7)
    d = gpu(a)
    y, g = fwd(d, eps=0.0), bwd(d, eps=0.0)
    torch.cuda.synchronize()
    check(a, y, g, eps=0.0)


def test_is_deterministic_and_ignores_the_workspace():
    a = make(3000, 768, 3, torch.bfloat16, "after", seed=8)
    d = gpu(a)
    g0 = bwd(d)
    n = ms.group_norm_workspace_bytes(3000, 768, 3, torch.bfloat16)
    g1 = bwd(d, workspace=torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda"))
    out = torch.empty_like(d["x"])
    assert fwd(d, out=out) is out
    torch.cuda.synchronize()
    assert torch.equal(out, fwd(d))
    for n in g0:
        assert torch.equal(g0[n], g1[n]), n


def test_streams_and_captured_graphs():
    a = make(500, 512, 8, torch.bfloat16, "first", seed=9)
    d = gpu(a)
    kw = dict(gate_first=True, center=False)
    y0, g0 = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((fwd(d, **kw), bwd(d, **kw)))
        graphs.append(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        for y, g in outs:
            y.zero_(), [t.zero_() for t in g.values()]
        graphs[i % 2].replay()
        with torch.cuda.stream(side):
            ge = bwd(d, **kw)
        graphs[(i + 1) % 2].replay()
        torch.cuda.synchronize()
        for y, g in outs + [(y0, ge)]:
            assert torch.equal(y, y0) and all(torch.equal(g[n], g0[n]) for n in g0)


def test_rows_past_2_31_elements():
    wide = torch.empty(150, 1 << 24, dtype=torch.bfloat16, device="cuda")
    a = make(150, 256, 2, torch.bfloat16, "after", seed=10)
    v = dict(a, weight=a["weight"].cuda(), bias=a["bias"].cuda())
    for i, n in enumerate(("x", "z", "dy")):
        v[n] = wide[:, i * 256:(i + 1) * 256]
        v[n].copy_(a[n])
    y, g = fwd(v), bwd(v)
    torch.cuda.synchronize()
    check(a, y, g)
