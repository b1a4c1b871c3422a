"""Gradients of the Mamba-2 SSD scan where what is not finite has to cross
chunks whose decay vanishes in float32: a decay is never 0 (a step's exponent is
finite), so the state behind such a chunk is not finite either, nor the gradient
before it, and no document's begin stands between. Against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle.linattn import f64
from oracle.ssd_bwd import oracle_ssd_bwd
from tests.test_ssd_bwd_gpu import BF, bounds, call, gpu, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("names,at", [(("x",), 10), (("B",), 300), (("dy",), 1100), (("C",), 700), (("state",), 0),
                                      (("dstate",), 0), (("x", "dy"), 600)], ids=str)
@pytest.mark.parametrize("docs", [False, True])
def test_not_finite_across_vanishing_decays(names, at, docs, dtype):
    """1200 tokens, five chunks, each of which decays to e^-300 and less."""
    a = make(1, 1200, 4, 2, 64, dtype, seed=31, state=True, a_range=(16.0, 32.0), dt_range=(0.1, 0.4))
    if docs:  # one that all of this is in, and one behind it that has none of it
        ids = torch.zeros(1, 1200, dtype=torch.int32)
        ids[:, 1150:] = 1
        a["seq_idx"] = ids
    tol = bounds(a)
    for n in names:
        a[n] = a[n].clone()
        if n.endswith("state"):
            a[n][0, 0] = float("nan")
        else:
            a[n][0, at] = float("nan")
    print(names, at, docs, dtype, flush=True)
    got = call(gpu(a))
    torch.cuda.synchronize()
    want = oracle_ssd_bwd(**a)
    for n in ("dx", "dB", "dC", "ddt", "dstate"):
        v, w = f64(got[n]), want[n]
        finite = np.isfinite(w)
        assert not np.isfinite(v[~finite]).any(), (n, np.argwhere(np.isfinite(v) & ~finite)[:4])
        if n == "ddt":  # (of its document it may be NaN anywhere)
            finite = finite & ((np.arange(1200) >= 1150) & docs)[None, :, None]
        t = tol[n] + (BF * (np.abs(w) + tol[n]) if dtype == "bf16" and n != "dstate" else 0) + 1e-37
        assert (np.abs(v - w) <= t)[finite].all(), n
