"""The group norm and linear attention on the GPU at the limits of what their
headers allow: the most rows and heads, decays above 0, an eps of 0 over values
whose squares leave float32's normal range."""
import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import gnorm as gn
from oracle import linattn as la
from tests.test_gnorm_gpu import DT, U
from tests.test_linattn_gpu import BF, absolute, bwd_args, check_bwd, check_fwd, fwd_args, gpu, make, say, steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(48, 4), (130, 10), (1536, 1), (16384, 1)], ids=str)
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -66, 2.0 ** -70])
def test_tiny_values_without_eps(size, shape, dtype):
    """A sum of squares below 2^-126 is held in steps of 2^-149: each of gs squares and each partial sum is off by at
    most half a step, 2 gs 2^-150 of a sum of about gs size^2, and the reciprocal root by half of that share."""
    c, groups = shape
    g = torch.Generator().manual_seed(81)
    x = (torch.randn(7, c, generator=g) * size).to(DT[dtype])
    dy = torch.randn(7, c, generator=g).to(DT[dtype])
    say("tiny", size, shape, dtype)
    how = dict(eps=0.0, activation="none")
    y = ms.group_norm_fwd(x.cuda(), None, None, groups, **how)
    grads = ms.group_norm_bwd(x.cuda(), None, None, groups, dy.cuda(), **how)
    torch.cuda.synchronize()
    want = gn.oracle_fwd(x, None, None, groups, **how)
    r = 1 / np.sqrt((gn.f64(x) ** 2).reshape(7, groups, -1).mean(-1))
    low = 2.0 ** -149 * (r ** 2).max()  # of the sum of squares, and twice that allowed for the mean's own error
    tol = (c // groups + 80) * 4 * U + 2 * low + (BF if dtype == "bf16" else 0)
    assert low < 1.0 / 16
    err = np.abs(y.cpu().double().numpy() - want) / (1 + np.abs(want))
    assert np.isfinite(y.cpu().double().numpy()).all() and err.max() <= tol
    dx, wdx = grads["dx"].cpu().double().numpy(), gn.oracle_bwd(x, None, None, groups, dy, **how)["dx"]
    m = (1 + np.abs(want)) ** 2 * (1 + np.abs(gn.f64(dy)).max()) * r.max() * 2
    assert np.isfinite(dx).all() and (np.abs(dx - wdx) / m).max() <= 4 * tol


def test_the_most_rows_of_one_channel():
    """rows * groups of 2^31 - 1."""
    rows = (1 << 31) - 1
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[1::2] = -3.0
    def holds(t, even, odd):
        return bool((t[::2] == even).all()) and bool((t[1::2] == odd).all())

    how = dict(center=False, eps=0.0, activation="none")
    y = ms.group_norm_fwd(x, None, None, 1, **how)
    assert holds(y, 1.0, -1.0)
    y = ms.group_norm_fwd(x, None, None, 1, x, **how)
    assert holds(y, 1.0, 3.0)
    w = torch.full((1,), 2.0, device="cuda")
    g = ms.group_norm_bwd(x, w, None, 1, x, x, **how)
    torch.cuda.synchronize()
    # y = sign(x) w z: dz = dy sign(x) w; dw = the sum of dy z sign(x), 1 for even rows and -9 for odd ones; dx is
    # r d (1 - xh^2), d = dy z w, where xh = x r is 1 up to the 2 u of r and the u of the product
    assert holds(g["dz"], 2.0, 6.0)
    most = float(g["dx"].abs().max())
    assert most <= 18 * 8 * U
    exact = (rows + 1) // 2 - 9 * (rows // 2)
    assert abs(float(g["dweight"]) - exact) <= 2.0 ** -10 * 10 * rows


def test_the_most_heads():
    """batch * nheads of 2^20, the heads of a row on one group."""
    b, H, d = 1 << 18, 4, 8
    gen = torch.Generator("cuda").manual_seed(82)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    q, k, v, dy = rnd(b, 1, 1, d), rnd(b, 1, 1, d), rnd(b, 1, H, d), rnd(b, 1, H, d)
    s, ds = rnd(b, H, d, d), rnd(b, H, d, d)
    decay = -torch.tensor([0.5, 0.1, 0.02, 3.0], device="cuda")
    y, s1 = ms.lin_attn_fwd(q, k, v, decay, s)
    yt, st = ms.lin_attn_step(q[:, 0], k[:, 0], v[:, 0], decay, s)
    g = ms.lin_attn_bwd(q, k, v, decay, dy, s, ds)
    lam = decay.double().exp().view(1, H, 1, 1)
    Q, K, V, Y = q[:, 0].double(), k[:, 0].double(), v[:, 0].double(), dy[:, 0].double()
    S = lam * s.double() + V[..., None] * K[:, :, None]
    want_y = d ** -0.5 * (S * Q[:, :, None]).sum(-1)
    R = ds.double() + d ** -0.5 * Y[..., None] * Q[:, :, None]
    want = {"dq": d ** -0.5 * (S * Y[..., None]).sum((1, 2))[:, None], "dk": (R * V[..., None]).sum((1, 2))[:, None],
            "dv": (R * K[:, :, None]).sum(-1), "dstate": lam * R}
    # sums of at most 32 terms below 6^3 each, some 60 roundings
    tol = 60 * U * 32 * 216
    for got, w in [(y[:, 0], want_y), (yt, want_y), (s1, S), (st, S)] + [(g[n].view(want[n].shape), want[n]) for n in want]:
        assert float((got.double() - w).abs().max()) <= tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 300, 3, 3, 64, 64), (1, 1100, 1, 1, 40, 128)], ids=str)
def test_decays_above_zero(shape, dtype):
    """The state grows; the first head's by e^30 or so."""
    a = make(*shape, DT[dtype], seed=83, state=True, backward=True)
    a["log_decay"] = a["log_decay"].abs() * (30 / shape[1] / a["log_decay"].abs().max())
    d = gpu(a)
    got, grads = ms.lin_attn_fwd(*fwd_args(d)), ms.lin_attn_bwd(*bwd_args(d))
    torch.cuda.synchronize()
    check_fwd(a, got, "growing")
    check_bwd(a, grads, "growing")


@pytest.mark.parametrize("L,decay", [(128, 1.3), (8192, 0.5)])
def test_a_growing_head_that_starts_from_nothing(L, decay):
    """Keys of 0 up to the last tokens: the power of lam over all that (lam^8192 is far beyond float32) has nothing to
    multiply, in one segment and in several."""
    a = make(1, L, 1, 1, 32, 32, torch.float32, seed=84)
    a["k"][:, :-20] = 0
    a["log_decay"] = torch.tensor([decay])
    assert (ms.lin_attn_workspace_bytes(1, L, 1, 1, 32, 32, torch.float32) > 0) == (L > 1000)
    d = gpu(a)
    y, s = ms.lin_attn_fwd(*fwd_args(d))
    torch.cuda.synchronize()
    want, size = la.oracle_fwd(*fwd_args(a)), la.oracle_fwd(*fwd_args(absolute(a)))
    # as many roundings as a sequence of the last two chunks has
    tol = steps(dict(a, q=a["q"][:, -128:])) * U
    for got, w, m in zip((y, s), want, size):
        assert (np.abs(got.cpu().double().numpy() - w) <= tol * m + 1e-30).all()


@pytest.mark.parametrize("where", ["v", "state"])
@pytest.mark.parametrize("L", [300, 4200])
def test_an_infinity_lasts(L, where):
    """An infinite value or state is infinite at the end of a sequence, in one segment as in several, over which the
    power of lam is below float32; a head without memory has 0 times it, NaN, at the next token already."""
    a = make(1, L, 2, 2, 64, 64, torch.bfloat16, seed=85, state=True)
    assert (ms.lin_attn_workspace_bytes(1, L, 2, 2, 64, 64, torch.bfloat16) > 0) == (L > 1000)
    a["q"], a["k"] = a["q"].abs() + 0.5, a["k"].abs() + 0.5
    a["log_decay"] = torch.tensor([-0.5, -0.01])
    d = gpu(a)
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d))
    bad = -float("inf")
    if where == "v":
        d["v"] = d["v"].clone()
        d["v"][0, 5, :, 9] = bad
    else:
        d["state"] = d["state"].clone()
        d["state"][0, :, 9] = bad
    y, s = ms.lin_attn_fwd(*fwd_args(d))
    torch.cuda.synchronize()
    first = 5 if where == "v" else 0
    assert (y[0, first:, :, 9] == bad).all() and (s[0, :, 9] == bad).all()
    rest = torch.arange(64) != 9
    assert torch.equal(y[..., rest], y0[..., rest]) and torch.equal(s[:, :, rest], s0[:, :, rest])
    assert torch.equal(y[:, :first], y0[:, :first])
