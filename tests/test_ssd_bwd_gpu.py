"""Gradients of the Mamba-2 SSD scan on the GPU against the fp64 oracle: every
output at lengths around the tile and chunk edges, d_state 64 and 128, both io
types, shared and own groups, heads split over workgroups and not, carried
states and their gradients, packed documents, strided rows, steep and slow
decays, other documents' infinities and NaN, streams and captured graphs, and
against differences of the library's own forward.

The bounds are counted, not fitted. With U = 2^-24, a term goes through the
roundings of its dot products (64 + d_state), of sums over a chunk (256), over
chunks and over a group's heads, of its decays (the exponent stands up to |cs|
from 0 and is rounded, delta A with it; delta itself is within 2 |v| + 12 of
itself, for softplus' exponential and logarithm), and 40 more: each output is
within that many U of the sum of its terms' magnitudes, which the oracle gives.
g may be a difference of running sums over a tile: its bound has the tile's
terms besides. For bfloat16 io a product that meets the matrix cores in two
parts is off by 2^-17 of itself, 128 U, for outputs in io; those are then rounded,
by 2^-8 at most."""
import sys

import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
import workloads
from oracle.linattn import f64
from oracle.ssd_bwd import oracle_ssd_bwd

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
KEYS = workloads.SSD_KEYS
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make(b, L, H, G, N, dtype, seed=0, state=False, docs=0, a_range=(1.0, 16.0), dt_range=(1e-3, 1e-1)):
    a = workloads.make_ssd(b, L, H, 64, N, G, DT[dtype], seed=seed, a_range=a_range, dt_range=dt_range)
    g = torch.Generator().manual_seed(seed + 100)
    a["dy"] = torch.randn(b, L, H, 64, generator=g).to(DT[dtype])
    a["state"] = torch.randn(b, H, 64, N, generator=g) if state else None
    a["dstate"] = torch.randn(b, H, 64, N, generator=g) if state else None
    a["seq_idx"] = torch.cumsum(torch.rand(b, L, generator=g) < 1.0 / docs, 1).to(torch.int32) if docs else None
    return a


def gpu(a):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in a.items()}


def call(a, **kw):
    return ms.ssd_bwd(*(a[n] for n in KEYS), a["dy"], a["state"], a["dstate"], seq_idx=a["seq_idx"], **kw)


def bounds(a):
    """What each output may be off, but for the rounding to the io type."""
    size = oracle_ssd_bwd(**a, magnitudes=True)
    b, L, H, _ = a["x"].shape
    G, N = a["B"].shape[2:]
    delta, A = size["delta"], np.abs(f64(a["A"]))
    ends = list(range(0, L, 256)) + [L]
    span = max((delta[:, lo:hi] * A).sum(1).max() for lo, hi in zip(ends, ends[1:]))
    of_delta = 2 * np.abs(size["v"]).max() + 12
    n = (64 + N) + 256 + len(ends) + H // G + (of_delta + 3) * (1 + min(span, 104.0)) + 40
    wide = 128 if a["x"].dtype == torch.bfloat16 else 0
    inside = size["inside"]
    tile = np.stack([inside[:, t // 64 * 64:t // 64 * 64 + 64].sum(1) for t in range(L)], 1)
    g = n * U * (size["g"] + tile)
    ddt = n * U * size["ddt"] + A * g * size["sig"]
    tol = {m: (n + wide) * U * size[m] for m in ("dx", "dB", "dC")}
    tol.update(ddt=ddt, dstate=n * U * size["dstate"], dD=(n + b * L) * U * size["dD"],
               ddt_bias=ddt.sum((0, 1)) + (b * L + 8) * U * size["ddt_bias"],
               dA=(g * delta).sum((0, 1)) + (n + b * L) * U * size["dA"])
    return tol


def check(a, got, what):
    want, tol = oracle_ssd_bwd(**a), bounds(a)
    io = a["x"].dtype
    names = {"dx", "ddt", "dB", "dC", "ddt_bias", "dA", "dD"} | ({"dstate"} if a["state"] is not None else set())
    assert set(got) == names
    for n in sorted(names):
        rounded = io == torch.bfloat16 and n in ("dx", "ddt", "dB", "dC")
        assert got[n].dtype == (io if n in ("dx", "ddt", "dB", "dC") else torch.float32)
        t = tol[n] + (BF * (np.abs(want[n]) + tol[n]) if rounded else 0) + 1e-37
        v = f64(got[n])
        assert v.shape == want[n].shape and np.isfinite(v).all(), what + " " + n
        err = np.abs(v - want[n])
        at = np.unravel_index(np.argmax(err / t), err.shape)
        assert (err <= t).all(), "%s %s: %g off at %s, %g allowed" % (what, n, err[at], at, t[at])


SHAPES = [
    # batch, seqlen, heads, groups, d_state, state
    (1, 1, 1, 1, 64, True), (2, 2, 2, 1, 128, False), (1, 15, 3, 3, 64, True), (1, 16, 2, 2, 128, True),
    (1, 63, 4, 2, 64, False), (2, 64, 2, 1, 128, True), (1, 65, 6, 1, 64, True), (1, 129, 3, 1, 128, False),
    (2, 191, 2, 2, 64, True), (1, 192, 5, 1, 64, False), (1, 255, 2, 1, 128, True), (1, 256, 4, 2, 64, True),
    (1, 257, 3, 1, 128, True), (2, 300, 8, 1, 64, False), (1, 513, 2, 1, 128, True), (3, 770, 2, 2, 64, True),
    (17, 70, 8, 4, 64, True), (1, 1300, 24, 1, 64, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_gradients(i, dtype):
    b, L, H, G, N, st = SHAPES[i]
    say("ssd_bwd", SHAPES[i], dtype)
    a = make(b, L, H, G, N, dtype, seed=i, state=st)
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "ssd")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,docs,N", [(64, 8, 64), (200, 1, 64), (256, 30, 128), (300, 60, 64), (520, 200, 128), (700, 500, 64)])
def test_packed_documents(L, docs, N, dtype):
    say("packed", L, docs, N, dtype)
    a = make(2, L, 4, 2, N, dtype, seed=L, state=True, docs=docs)
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "packed")


@pytest.mark.parametrize("cuts", [[64], [63, 64, 65], [256], [128, 256, 257], [1], [299], [10, 20, 266]])
def test_documents_at_the_edges(cuts):
    a = make(1, 300, 2, 1, 64, "f32", seed=5, state=True)
    ids = torch.zeros(1, 300, dtype=torch.int64)
    for n, c in enumerate(cuts):
        ids[:, c:] = (n + 1) % 2  # ids come again: 0 1 0 1
    a["seq_idx"] = ids
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "edges %s" % cuts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("a_range,dt_range", [((1e-4, 1e-3), (1e-3, 1e-2)), ((16.0, 64.0), (0.5, 2.0)), ((1.0, 1.0), (5.0, 9.0))])
def test_slow_and_steep_decays(a_range, dt_range, dtype):
    a = make(1, 400, 4, 1, 64, dtype, seed=7, state=True, a_range=a_range, dt_range=dt_range)
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "decays")


def test_no_decay_and_vanishing_steps():
    a = make(1, 130, 2, 1, 64, "f32", seed=8, state=True)
    a["A"] = torch.zeros(2)
    a["dt_bias"] = torch.tensor([0.5, -120.0])  # a step of 0 in float32
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "no decay")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_columns_of_wider_tensors(dtype):
    a = make(2, 150, 4, 2, 64, dtype, seed=9)
    g = gpu(a)
    t = DT[dtype]
    xbc = torch.zeros(2, 150, 256 + 2 * 128 + 8, dtype=t, device="cuda")
    views = dict(x=xbc[..., :256].unflatten(-1, (4, 64)), B=xbc[..., 256:384].unflatten(-1, (2, 64)),
                 C=xbc[..., 384:512].unflatten(-1, (2, 64)))
    views["dt"] = torch.zeros(2, 150, 9, dtype=t, device="cuda")[..., 3:7]
    views["dy"] = torch.zeros(2, 150, 320, dtype=t, device="cuda")[..., 64:].unflatten(-1, (4, 64))
    for n, v in views.items():
        v.copy_(g[n])
        assert not v.is_contiguous()
    want, got = call(g), call(dict(g, **views))
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    check(a, got, "columns")


def test_against_differences_of_the_forward():
    """Along a random direction, the forward's difference is what the gradients say (float32: a difference of 2 h |g| has
    the forward's rounding, about 1e-6 of its outputs' size, and the third derivative's h^2)."""
    a = make(1, 300, 2, 1, 64, "f32", seed=10, state=True)
    g = gpu(a)
    grads = call(g)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for n in (*KEYS, "state"):
        d = torch.randn(g[n].shape, device="cuda", generator=gen) * g[n].abs().mean().clamp(min=0.1)
        h = 1e-2

        def loss(sign):
            args = dict(g)
            args[n] = g[n] + sign * h * d
            y, s = ms.ssd_fwd(*(args[k] for k in KEYS), args["state"])
            return float((y.double() * g["dy"].double()).sum() + (s.double() * g["dstate"].double()).sum())

        diff = (loss(1) - loss(-1)) / (2 * h)
        want = float((grads["d" + n].double() * d.double()).sum())
        scale = float(grads["d" + n].double().norm() * d.double().norm())
        assert abs(diff - want) <= 2e-3 * scale + 1e-2 * abs(want), (n, diff, want, scale)


def test_workspace_and_determinism():
    a = gpu(make(2, 600, 6, 1, 128, "bf16", seed=11, state=True, docs=100))
    need = ms.ssd_bwd_workspace_bytes(2, 600, 6, 64, 128, 1, torch.bfloat16)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = call(a, workspace=ws)
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(got[n], first[n]) for n in got)


def test_a_constant_seq_idx_changes_no_bit():
    a = gpu(make(1, 500, 4, 2, 64, "bf16", seed=12, state=True))
    want = call(a)
    got = call(dict(a, seq_idx=torch.full((1, 500), 7, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_stream_and_captured_graph():
    a = gpu(make(2, 300, 4, 1, 64, "bf16", seed=13, state=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(a)
    for i in range(3):
        a["x"].copy_(torch.randn(a["x"].shape, generator=torch.Generator().manual_seed(i)))
        want = call(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_two_calls_at_once():
    """Two streams, each with its own tensors and workspace."""
    sets = [gpu(make(1, 700, 4, 1, 128, "bf16", seed=20 + i, state=True)) for i in range(2)]
    want = [call(a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = call(sets[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(got[i][n], want[i][n]) for n in want[i])


@pytest.mark.parametrize("what", ["all nan", "all inf", "one x", "one B", "one dy", "one C", "dt"])
@pytest.mark.parametrize("N,G,dtype", [(64, 2, "f32"), (128, 1, "f32"), (64, 1, "bf16"), (128, 1, "bf16")])
def test_what_is_not_finite_stays_in_its_document(N, G, dtype, what):
    """Documents begin inside tiles, at a tile's and behind a chunk's edge; what the second and the fifth hold is not
    finite. The others' gradients are those of finite inputs, to the same bounds."""
    b, L, H = 2, 700, 4
    a = make(b, L, H, G, N, dtype, seed=11, state=True)
    ids = torch.zeros(b, L, dtype=torch.int32)
    for n, at in enumerate((37, 101, 192, 300, 517, 640)):
        ids[:, at:] = n + 1
    a["seq_idx"] = ids
    bad = (ids == 1) | (ids == 4)
    bad[0] = ids[0] == 1
    clean = ~bad.numpy()
    want, tol = oracle_ssd_bwd(**a), bounds(a)
    g = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    value = float("nan") if what == "all nan" else float("inf")
    for n in ("x", "dt", "B", "C", "dy"):
        if what.startswith("all"):
            g[n][bad] = value
        elif what == "dt" == n:
            g[n][bad] = float("nan")
        elif what == "one " + n:
            g[n][0, 60, 0, 5] = value
            g[n][1, 400, -1, -1] = -value
    say(what, N, G, dtype)
    got = call(gpu(g))
    torch.cuda.synchronize()
    for n in ("dx", "ddt", "dB", "dC"):
        rounded = dtype == "bf16"
        t = tol[n] + (BF * (np.abs(want[n]) + tol[n]) if rounded else 0) + 1e-37
        v = f64(got[n])
        assert np.isfinite(v[clean]).all(), n
        assert (np.abs(v - want[n]) <= t)[clean].all(), n
        if what.startswith("all"):
            assert not np.isfinite(v[~clean]).any(), n
    assert (np.abs(f64(got["dstate"]) - want["dstate"]) <= tol["dstate"] + 1e-37).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_finite_reaches_what_it_is_a_term_of(dtype):
    """Without documents: x and B of a token are terms of its own dx and dB and of dC from it on, C and dy of its own dC
    and of dx and dB up to it."""
    a = make(1, 330, 2, 1, 128, dtype, seed=12, state=True)
    want, tol = oracle_ssd_bwd(**a), bounds(a)
    for names, at in ((("x", "B"), 40), (("C", "dy"), 290), (("C", "dy"), 20)):
        g = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in a.items()}
        for n in names:
            g[n][0, at] = float("nan")
        say(names, at, dtype)
        got = call(gpu(g))
        torch.cuda.synchronize()
        t = np.arange(330)
        for n in ("dx", "dB", "dC"):
            if names[0] == "x":
                free = t < at if n == "dC" else t != at
            else:
                free = t != at if n == "dC" else t > at
            bound = tol[n] + (BF * (np.abs(want[n]) + tol[n]) if dtype == "bf16" else 0) + 1e-37
            v = f64(got[n])
            assert (np.abs(v - want[n]) <= bound)[0, free].all(), n
            assert not np.isfinite(v[0, at]).any(), n
