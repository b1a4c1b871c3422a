"""The oracle of the SSD scan's gradients against central differences of the
pinned forward oracle, and its packed form against each document on its own."""
import numpy as np
import pytest

from oracle import ssd
from oracle.ssd_bwd import oracle_ssd_bwd


def make(b, L, H, G, N, seed, docs=None):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    a = dict(x=n(b, L, H, 4), dt=0.5 * n(b, L, H), B=n(b, L, G, N), C=n(b, L, G, N), dt_bias=n(H), A=-np.exp(n(H)), D=n(H))
    return a, n(b, L, H, 4), n(b, H, 4, N), n(b, H, 4, N), docs


@pytest.mark.parametrize("docs", [None, [[0, 0, 1, 1, 1, 0, 0], [3, 3, 3, 3, 3, 3, 2]]])
def test_gradients_against_differences(docs):
    a, dy, s0, ds, docs = make(2, 7, 2, 1, 3, 1, docs)
    ids = None if docs is None else np.array(docs, dtype=np.int32)
    got = oracle_ssd_bwd(**a, dy=dy, state=s0, dstate=ds, seq_idx=ids)

    def loss(**over):
        y, s = ssd.oracle_ssd_fwd(**{**a, "state": s0, **over}, seq_idx=ids)
        return (y * dy).sum() + (s * ds).sum()

    for n, value in dict(a, state=s0).items():
        want = got["d" + n]
        for at in np.ndindex(value.shape):
            up, down = value.copy(), value.copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            assert abs((loss(**{n: up}) - loss(**{n: down})) / 2e-5 - want[at]) < 1e-7, (n, at)


def test_packed_is_each_document_alone():
    a, dy, s0, ds, _ = make(1, 9, 4, 2, 3, 2)
    ids = np.array([[0, 0, 0, 5, 5, 1, 1, 1, 1]], dtype=np.int32)
    got = oracle_ssd_bwd(**a, dy=dy, state=s0, dstate=ds, seq_idx=ids)
    whole = {n: 0.0 for n in ("ddt_bias", "dA", "dD")}
    for lo, hi in ((0, 3), (3, 5), (5, 9)):
        cut = {n: v[:, lo:hi] if n in ("x", "dt", "B", "C") else v for n, v in a.items()}
        one = oracle_ssd_bwd(**cut, dy=dy[:, lo:hi], state=s0 if lo == 0 else None, dstate=ds if hi == 9 else None)
        for n in ("dx", "ddt", "dB", "dC"):
            assert np.abs(one[n] - got[n][:, lo:hi]).max() < 1e-13
        for n in whole:
            whole[n] = whole[n] + one[n]
        if lo == 0:
            assert np.abs(one["dstate"]).max() > 0 and (got["dstate"] == one["dstate"]).all()
    for n in whole:
        assert np.abs(whole[n] - got[n]).max() < 1e-12


def test_magnitudes_bound_the_gradients():
    a, dy, s0, ds, _ = make(2, 6, 4, 2, 3, 3)
    got = oracle_ssd_bwd(**a, dy=dy, state=s0, dstate=ds)
    size = oracle_ssd_bwd(**a, dy=dy, state=s0, dstate=ds, magnitudes=True)
    for n in got:
        assert (np.abs(got[n]) <= size[n] * (1 + 1e-12)).all(), n
