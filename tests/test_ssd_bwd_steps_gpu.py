"""Gradients of the Mamba-2 SSD scan where a step is so large that nothing is
left of what came before it (finite ones up to 10^25, and infinity), against
the fp64 oracle. What such a step does not meet is as right as ever; what the
oracle has not finite is not finite.

The bounds are those of tests/test_ssd_bwd_gpu.py, in three places closer to
the arithmetic. delta is within 12 U of itself from v = 0 on (it is v and more
there), so only a negative v's 2 |v| counts. The running sums that g may be
taken from start again at a document's begin and at a step of -104 or less,
behind which float32 keeps nothing: a token has the terms of its tile from the
latest of these up to the next one, and at such a step itself none."""
import numpy as np
import pytest
import torch

from oracle.linattn import f64
from oracle.ssd_bwd import oracle_ssd_bwd
from tests.test_ssd_bwd_gpu import BF, DT, U, call, gpu, make

pytestmark = pytest.mark.gpu


def bounds(a):
    """What each output may be off, but for the rounding to the io type; not finite where a term is not."""
    with np.errstate(all="ignore"):
        size = oracle_ssd_bwd(**a, magnitudes=True)
        b, L, H, _ = a["x"].shape
        G, N = a["B"].shape[2:]
        delta, A = size["delta"], np.abs(f64(a["A"]))
        chunks = -(-L // 256)
        of_delta = 2 * np.maximum(-size["v"], 0).max() + 12
        n = (64 + N) + 256 + chunks + 1 + H // G + (of_delta + 3) * (1 + 104.0) + 40
        wide = 128 if a["x"].dtype == torch.bfloat16 else 0
        gone = delta * A >= 104.0
        start = gone.copy()
        start[:, ::64] = True
        if a["seq_idx"] is not None:
            ids = f64(a["seq_idx"])
            start[:, 1:] |= (ids[:, 1:] != ids[:, :-1])[..., None]
        piece = np.cumsum(start, 1)
        tile = np.zeros_like(delta)
        for i, h in np.ndindex(b, H):
            for p in range(1, piece[i, -1, h] + 1):
                of = piece[i, :, h] == p
                tile[i, of, h] = size["inside"][i, of, h].sum()
        g = n * U * (size["g"] + np.where(gone, 0.0, tile))
        ddt = n * U * size["ddt"] + A * g * size["sig"]
        tol = {m: (n + wide) * U * size[m] for m in ("dx", "dB", "dC")}
        tol.update(ddt=ddt, dstate=n * U * size["dstate"], dD=(n + b * L) * U * size["dD"],
                   ddt_bias=ddt.sum((0, 1)) + (b * L + 8) * U * size["ddt_bias"],
                   dA=(g * delta).sum((0, 1)) + (n + b * L) * U * size["dA"])
    return tol


def check(a, got, what):
    with np.errstate(all="ignore"):
        want = oracle_ssd_bwd(**a)
    tol = bounds(a)
    for n in ("dx", "dB", "dC", "ddt", "dstate", "dD", "ddt_bias", "dA"):
        v, w = f64(got[n]), want[n]
        rounded = a["x"].dtype == torch.bfloat16 and n in ("dx", "ddt", "dB", "dC")
        finite = np.isfinite(w)
        with np.errstate(all="ignore"):
            t = np.where(finite, tol[n] + (BF * (np.abs(w) + tol[n]) if rounded else 0) + 1e-37, 0)
        assert np.isfinite(t).all(), what + " " + n  # (the bound itself says something)
        lost, made = ~finite & np.isfinite(v), finite & ~np.isfinite(v)
        assert not lost.any(), "%s %s: finite at %s" % (what, n, np.argwhere(lost)[:4])
        assert not made.any(), "%s %s: not finite at %s" % (what, n, np.argwhere(made)[:4])
        err = np.where(finite, np.abs(np.where(finite, v, 0) - np.where(finite, w, 0)), 0)
        at = np.unravel_index(np.argmax(err / np.where(finite, t, 1)), err.shape)
        assert (err <= t).all(), "%s %s: %g off at %s, %g allowed" % (what, n, err[at], at, t[at])


def put(a, tokens, value, heads=None):
    a["dt"] = a["dt"].clone()
    for t in tokens:
        a["dt"][0, t, slice(None) if heads is None else heads] = value
    return a


# tokens whose steps are large: at a sequence's, a tile's and a chunk's edges, next to one another, and the last one
PLACES = [(0,), (40,), (63, 64), (100, 101, 300), (255,), (256,), (20, 520), (599,)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [600.0, 1e5, 1e12, 1e25])
@pytest.mark.parametrize("tokens", PLACES, ids=str)
def test_large_steps(tokens, size, dtype):
    print(tokens, size, dtype, flush=True)
    a = put(make(1, 600, 4, 2, 64, dtype, seed=3, state=True), tokens, size)
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "large")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [None, 1])
@pytest.mark.parametrize("tokens", PLACES, ids=str)
def test_infinite_steps(tokens, heads, dtype):
    """An infinite step's own gradients, and all that its state reaches, are not finite; the tokens before it never meet
    it, but in sums over tokens and heads."""
    print(tokens, heads, dtype, flush=True)
    a = put(make(1, 600, 4, 2, 128, dtype, seed=4, state=True), tokens, float("inf"), heads)
    got = call(gpu(a))
    torch.cuda.synchronize()
    check(a, got, "infinite")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e12, float("inf")])
def test_in_packed_documents(size, dtype):
    """A document's large steps are none of another's, wherever these begin."""
    a = make(2, 700, 4, 1, 64, dtype, seed=5, state=True)
    ids = torch.zeros(2, 700, dtype=torch.int32)
    for n, at in enumerate((37, 101, 192, 300, 517, 640)):
        ids[:, at:] = n + 1
    a["seq_idx"] = ids
    for tokens in ((36,), (37,), (50, 60), (150, 310), (600,), (639, 640)):
        print(tokens, size, dtype, flush=True)
        bad = put(dict(a), tokens, size)
        got = call(gpu(bad))
        torch.cuda.synchronize()
        check(bad, got, "documents")


def test_steep_heads():
    """A so low that every step leaves nothing, -infinity among them."""
    a = make(1, 300, 3, 1, 64, "f32", seed=6, state=True)
    a["A"] = torch.tensor([-1e30, -float("inf"), -1.0])
    got = call(gpu(a))
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want = oracle_ssd_bwd(**a)
    for n in ("dx", "dB", "dC"):
        assert np.isfinite(f64(got[n])).all() and np.isfinite(want[n]).all()
        w = want[n] if n != "dx" else want[n][:, :, :2]
        v = f64(got[n]) if n != "dx" else f64(got[n])[:, :, :2]
        size = oracle_ssd_bwd(**dict(a, A=torch.tensor([-1e30, -1e30, -1.0])), magnitudes=True)[n]
        size = size if n != "dx" else size[:, :, :2]
        assert (np.abs(v - w) <= 12000 * U * size + 1e-37).all(), n
