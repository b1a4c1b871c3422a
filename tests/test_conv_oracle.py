"""The oracle of the short causal convolution against torch's own convolution,
step chains, and its gradients against central differences."""
import numpy as np
import pytest
import torch

from oracle import conv as oc


def make(b, L, c, k, seed, state=True, docs=0):
    g = np.random.default_rng(seed)
    ids = None
    if docs:
        ids = np.cumsum(g.random((b, L)) < 1.0 / docs, 1).astype(np.int32)
    return dict(x=g.standard_normal((b, L, c)), weight=g.uniform(-1, 1, (c, k)), bias=g.standard_normal(c),
                state=g.standard_normal((b, c, k - 1)) if state else None, seq_idx=ids)


@pytest.mark.parametrize("k", [2, 3, 4])
def test_against_torch_conv1d(k):
    a = make(2, 19, 5, k, k)
    line = np.concatenate([a["state"].transpose(0, 2, 1), a["x"]], 1)
    want = torch.nn.functional.conv1d(torch.from_numpy(line).transpose(1, 2), torch.from_numpy(a["weight"])[:, None],
                                      torch.from_numpy(a["bias"]), groups=5).transpose(1, 2)
    y, last = oc.oracle_fwd(a["x"], a["weight"], a["bias"], a["state"], activation="none")
    assert np.abs(y - want.numpy()).max() < 1e-14
    y, _ = oc.oracle_fwd(a["x"], a["weight"], a["bias"], a["state"])
    assert np.abs(y - torch.nn.functional.silu(want).numpy()).max() < 1e-14
    assert (last == line[:, -(k - 1):].transpose(0, 2, 1)).all()


def test_step_chain_and_documents():
    a = make(2, 23, 3, 4, 1, docs=5)
    y, last = oc.oracle_fwd(**a)
    for b in range(2):
        ids, s = a["seq_idx"][b], a["state"][b:b + 1]
        for t in range(23):
            if t and ids[t] != ids[t - 1]:
                s = np.zeros_like(s)
            one, s = oc.oracle_step(a["x"][b:b + 1, t], a["weight"], a["bias"], s)
            assert np.abs(one - y[b, t]).max() < 1e-15
        assert (s[0] == last[b]).all()


@pytest.mark.parametrize("L,docs,activation", [(1, 0, "silu"), (2, 0, "silu"), (9, 3, "silu"), (9, 0, "none")])
def test_gradients_against_differences(L, docs, activation):
    a = make(2, L, 3, 4, 7, docs=docs)
    g = np.random.default_rng(8)
    dy, ds = g.standard_normal((2, L, 3)), g.standard_normal((2, 3, 3))
    got = oc.oracle_bwd(dy=dy, dstate=ds, activation=activation, **a)

    def loss(**over):
        y, s = oc.oracle_fwd(**{**a, **over}, activation=activation)
        return (y * dy).sum() + (s * ds).sum()

    for n in ("x", "weight", "bias", "state"):
        for at in np.ndindex(a[n].shape):
            up, down = a[n].copy(), a[n].copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            diff = (loss(**{n: up}) - loss(**{n: down})) / 2e-5
            assert abs(diff - got["d" + n][at]) < 1e-8, (n, at)
