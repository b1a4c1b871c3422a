"""The fp64 oracle of linear attention against independent evaluations: the
quadratic form, the SSD oracle at a constant step, split and resume, packed
documents as separate calls, and its gradients against central differences and
autograd."""
import numpy as np
import pytest
import torch

from oracle import linattn as la
from oracle import ssd as ossd


def make(b=2, L=9, H=4, G=2, dk=3, dv=5, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((b, L, G, dk)), k=r.standard_normal((b, L, G, dk)), v=r.standard_normal((b, L, H, dv)),
                log_decay=-r.uniform(0.01, 1.0, H)), r.standard_normal((b, H, dv, dk)), r


def test_quadratic_form():
    i, s0, _ = make()
    y, s = la.oracle_fwd(**i, state=s0)
    b, L, H, dv = i["v"].shape
    q, k = np.repeat(i["q"], 2, 2), np.repeat(i["k"], 2, 2)
    for h in range(H):
        g = i["log_decay"][h]
        for t in range(L):
            want = np.exp((t + 1) * g) * np.einsum("bvk,bk->bv", s0[:, h], q[:, t, h])
            for u in range(t + 1):
                want += np.exp((t - u) * g) * (q[:, t, h] * k[:, u, h]).sum(-1)[:, None] * i["v"][:, u, h]
            np.testing.assert_allclose(y[:, t, h], want * 3 ** -0.5, rtol=1e-12, atol=1e-13)


def test_equals_ssd_with_a_constant_step():
    """softplus(dt + bias) = 1 and D = 0 leave the SSD scan with the decay exp(A) per head."""
    i, _, r = make(dk=64, dv=64, L=20)
    s0 = r.standard_normal((2, 4, 64, 64))
    y, s = la.oracle_fwd(**i, state=s0, scale=1.0)
    dt = np.full((2, 20, 4), np.log(np.expm1(1.0)))
    ys, ss = ossd.oracle_ssd_fwd(i["v"], dt, i["k"], i["q"], np.zeros(4), i["log_decay"], np.zeros(4), state=s0)
    np.testing.assert_allclose(y, ys, rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(s, ss, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("cut", [1, 4, 8])
def test_split_and_resume(cut):
    i, s0, _ = make()
    y, s = la.oracle_fwd(**i, state=s0)
    part = lambda a, b: dict(i, **{n: i[n][:, a:b] for n in "qkv"})  # noqa: E731
    y1, s1 = la.oracle_fwd(**part(0, cut), state=s0)
    y2, s2 = la.oracle_fwd(**part(cut, 9), state=s1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(s2, s, rtol=1e-12, atol=1e-13)


def test_packed_documents_are_separate_calls():
    i, s0, r = make(L=11)
    ids = np.array([[0] * 4 + [1] * 1 + [2] * 6, [5] * 11])
    y, s = la.oracle_fwd(**i, state=s0, seq_idx=ids)
    dy, ds = r.standard_normal(y.shape), r.standard_normal(s.shape)
    g = la.oracle_bwd(**i, dy=dy, state=s0, dstate=ds, seq_idx=ids)
    one = lambda b, lo, hi: dict(i, **{n: i[n][b:b + 1, lo:hi] for n in "qkv"})  # noqa: E731
    for b, lo, hi in ((0, 0, 4), (0, 4, 5), (0, 5, 11), (1, 0, 11)):
        st = s0[b:b + 1] if lo == 0 else None
        y1, s1 = la.oracle_fwd(**one(b, lo, hi), state=st)
        np.testing.assert_allclose(y[b:b + 1, lo:hi], y1, rtol=1e-12, atol=1e-13)
        end = hi == 11
        if end:
            np.testing.assert_allclose(s[b:b + 1], s1, rtol=1e-12, atol=1e-13)
        g1 = la.oracle_bwd(**one(b, lo, hi), dy=dy[b:b + 1, lo:hi], state=st, dstate=ds[b:b + 1] if end else None)
        for n in ("dq", "dk", "dv"):
            np.testing.assert_allclose(g[n][b:b + 1, lo:hi], g1[n], rtol=1e-11, atol=1e-12)
        if lo == 0:
            np.testing.assert_allclose(g["dstate"][b:b + 1], g1["dstate"], rtol=1e-11, atol=1e-12)


def test_gradients_against_differences_and_autograd():
    i, s0, r = make(L=6)
    ids = np.array([[0, 0, 0, 1, 1, 1], [0] * 6])
    y, s = la.oracle_fwd(**i, state=s0, seq_idx=ids)
    dy, ds = r.standard_normal(y.shape), r.standard_normal(s.shape)
    g = la.oracle_bwd(**i, dy=dy, state=s0, dstate=ds, seq_idx=ids)

    def loss(**over):
        a = dict(i, state=s0)
        a.update(over)
        y, s = la.oracle_fwd(**a, seq_idx=ids)
        return (y * dy).sum() + (s * ds).sum()

    for name in ("q", "k", "v", "state"):
        base = s0 if name == "state" else i[name]
        d = r.standard_normal(base.shape)
        e = 1e-5
        slope = (loss(**{name: base + e * d}) - loss(**{name: base - e * d})) / (2 * e)
        got = (g["d" + name] * d).sum()
        assert abs(slope - got) <= 1e-8 * (1 + abs(got)), name
    # autograd of the same recurrence in torch
    t = {n: torch.tensor(a, requires_grad=True) for n, a in dict(i, state=s0).items() if n != "log_decay"}
    lam = torch.exp(torch.tensor(i["log_decay"]))[None, :, None, None]
    S, ys = t["state"], []
    for u in range(6):
        keep = torch.ones(2) if u == 0 else torch.tensor(ids[:, u] == ids[:, u - 1]).double()
        k, q = t["k"][:, u].repeat_interleave(2, 1), t["q"][:, u].repeat_interleave(2, 1)
        S = lam * keep.view(2, 1, 1, 1) * S + t["v"][:, u, :, :, None] * k[:, :, None, :]
        ys.append(3 ** -0.5 * (S * q[:, :, None, :]).sum(-1))
    total = (torch.stack(ys, 1) * torch.tensor(dy)).sum() + (S * torch.tensor(ds)).sum()
    for name, want in zip(t, torch.autograd.grad(total, list(t.values()))):
        np.testing.assert_allclose(g["d" + name], want.numpy(), rtol=1e-11, atol=1e-12)
