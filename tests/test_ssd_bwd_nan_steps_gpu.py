"""Gradients of the Mamba-2 SSD scan where single steps are NaN, against the
fp64 oracle: what such a step is a term of is not finite, whatever tile, chunk
or document it stands in; what it is no term of (dx and dB of the tokens behind
it, dC of those before it, other documents, heads and rows) is what it is
without it, to the same bounds, which are those of the same inputs with a number
in its place: the terms that these outputs have are the same."""
import numpy as np
import pytest
import torch

from oracle.linattn import f64
from oracle.ssd_bwd import oracle_ssd_bwd
from tests.test_ssd_bwd_gpu import BF, call, gpu, make
from tests.test_ssd_bwd_steps_gpu import PLACES, bounds, put

pytestmark = pytest.mark.gpu
NAN = float("nan")


def check(a, got, tol, what, may_be_lost=()):
    with np.errstate(all="ignore"):
        want = oracle_ssd_bwd(**a)
    for n in ("dx", "dB", "dC", "ddt", "dstate", "dD", "ddt_bias", "dA"):
        v, w = f64(got[n]), want[n]
        rounded = a["x"].dtype == torch.bfloat16 and n in ("dx", "ddt", "dB", "dC")
        finite = np.isfinite(w)
        lost, made = ~finite & np.isfinite(v), finite & ~np.isfinite(v)
        assert not lost.any(), "%s %s: finite at %s" % (what, n, np.argwhere(lost)[:4])
        if n in may_be_lost:
            finite &= ~made
        else:
            assert not made.any(), "%s %s: not finite at %s" % (what, n, np.argwhere(made)[:4])
        t = tol[n] + 1e-37
        err = np.where(finite, np.abs(np.where(finite, v, 0) - np.where(finite, w, 0)), 0)
        t = t + (BF * (np.abs(np.where(finite, w, 0)) + tol[n]) if rounded else 0)
        at = np.unravel_index(np.argmax(err / t), err.shape)
        assert (err <= t).all(), "%s %s: %g off at %s, %g allowed" % (what, n, err[at], at, t[at])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [None, 1])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("tokens", PLACES, ids=str)
def test_without_documents(tokens, state, heads, dtype):
    print(tokens, state, heads, dtype, flush=True)
    a = make(1, 600, 4, 2, 64 if state else 128, dtype, seed=14, state=state)
    tol = bounds(a)
    bad = put(dict(a), tokens, NAN, heads)
    got = call(gpu(bad))
    torch.cuda.synchronize()
    if not state:
        got["dstate"] = torch.from_numpy(oracle_ssd_bwd(**bad)["dstate"])
    check(bad, got, tol, "nan")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("steep", [False, True])
def test_in_packed_documents(steep, dtype):
    """Also where every chunk's decay vanishes, and where a large step stands beside the NaN."""
    more = dict(a_range=(16.0, 32.0), dt_range=(0.1, 0.4)) if steep else {}
    a = make(2, 700, 4, 1, 64, dtype, seed=15, state=True, **more)
    ids = torch.zeros(2, 700, dtype=torch.int32)
    for n, at in enumerate((37, 101, 192, 300, 517, 640)):
        ids[:, at:] = n + 1
    a["seq_idx"] = ids
    for tokens in ((0,), (36,), (37,), (50, 60), (150, 310), (516,), (600,), (639, 640), (699,)):
        for large in ((), (45, 155, 305), (515,)):
            print(tokens, large, steep, dtype, flush=True)
            ok = put(dict(a), large, 1e6)
            tol = bounds(ok)
            bad = put(dict(ok), tokens, NAN, 2)
            got = call(gpu(bad))
            torch.cuda.synchronize()
            check(bad, got, tol, "documents %s %s" % (tokens, large))


@pytest.mark.parametrize("L,N,dtype", [(1, 64, "f32"), (2, 64, "bf16"), (65, 128, "f32"), (300, 64, "bf16")])
def test_every_step(L, N, dtype):
    a = make(2, L, 2, 1, N, dtype, seed=16, state=True)
    bad = dict(a, dt=torch.full_like(a["dt"], NAN))
    got = call(gpu(bad))
    torch.cuda.synchronize()
    check(bad, got, bounds(a), "all")


@pytest.mark.parametrize("name", ["A", "dt_bias"])
def test_a_head_whose_parameter_is_nan(name):
    """A head with A NaN has NaN steps only. (Its first token's dC and last token's dx and dB, which meet no decay, may be NaN.)"""
    a = make(1, 400, 4, 2, 64, "f32", seed=17, state=True)
    tol = bounds(a)
    bad = dict(a, **{name: a[name].clone()})
    bad[name][2] = NAN
    got = call(gpu(bad))
    torch.cuda.synchronize()
    check(bad, got, tol, name, may_be_lost=("dx", "dB", "dC", "ddt", "dstate"))
    for n in ("dx", "ddt", "dstate"):
        heads = 2 if n != "dstate" else 1
        keep = np.arange(4) != 2
        assert np.isfinite(np.compress(keep, f64(got[n]), axis=heads)).all(), n
    for n in ("dB", "dC"):
        assert np.isfinite(f64(got[n])[:, :, 0]).all(), n
