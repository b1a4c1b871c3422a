"""Linear attention on the GPU with an infinite value in one place: what it is a
term of is not finite, and all else has the bits that it has without it, in both
io types, at head sizes that fill a tile and that do not, in one chunk, in several
and over segments, forwards and backwards.

All that the infinity meets is positive and far from 0, so that the recurrence has
an infinity of one sign everywhere. Where values meet it as several bfloat16 parts
of which one may be 0, NaN comes out; bfloat16 values and states do not: they meet
keys and queries, which are one part, and stay infinities of their sign."""
import pytest
import torch

import selective_state_space_07_amd as ms
from tests.test_linattn_gpu import DT, bwd_args, fwd_args, gpu, make, say

pytestmark = pytest.mark.gpu
INF = float("inf")
SHAPES = [(1, 70, 2, 2, 64, 64), (1, 200, 2, 1, 40, 72), (2, 130, 2, 2, 96, 24), (1, 150, 1, 1, 128, 128),
          (1, 2100, 2, 2, 64, 40), (1, 1500, 1, 1, 104, 64)]


def positive(shape, dtype, seed):
    a = make(*shape, DT[dtype], seed=seed, state=True, backward=True)
    for n in ("q", "k", "v", "dy", "state", "dstate"):
        a[n] = a[n].abs() + 0.25
    a["log_decay"] = a["log_decay"] * 0.02  # no weight leaves float32
    return a


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, sign):
    say("infinities", shape, dtype, sign)
    a = positive(shape, dtype, 101)
    b, L, H, G, dk, dv = shape
    d = gpu(a)
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d))
    bad = sign * INF
    for at in (0, 9, 66, L - 1):
        for n, e in (("v", dv - 1), ("k", dk - 1), ("q", dk // 2)):
            t = d[n].clone()
            t[0, at, -1, e] = bad
            y, s = ms.lin_attn_fwd(*fwd_args(dict(d, **{n: t})))
            w, _ = ms.lin_attn_fwd(*fwd_args(dict(d, **{n: t})), return_state=False)
            torch.cuda.synchronize()
            assert torch.equal(y.nan_to_num(3e4), w.nan_to_num(3e4))
            heads = torch.arange(H, device="cuda") // (H // G) == G - 1  # of the head, or of the group of q and k
            hit = torch.zeros(b, L, H, dv, dtype=torch.bool, device="cuda")
            sit = torch.zeros(b, H, dv, dk, dtype=torch.bool, device="cuda")
            if n == "v":
                hit[0, at:, -1, e] = True
                sit[0, -1, e] = True
            elif n == "k":
                hit[0, at:, heads] = True
                sit[0, heads, :, e] = True
            else:
                hit[0, at, heads] = True
            assert torch.equal(y[~hit], y0[~hit]) and torch.equal(s[~sit], s0[~sit]), (n, at)
            if n == "v" and dtype == "bf16":
                assert (y[hit] == bad).all() and (s[sit] == bad).all(), at
            assert not torch.isfinite(y[hit]).any() and not torch.isfinite(s[sit]).any(), (n, at)
    t = d["state"].clone()
    t[0, 0, dv // 2, dk - 1] = bad
    y, s = ms.lin_attn_fwd(*fwd_args(dict(d, state=t)))
    torch.cuda.synchronize()
    assert s[0, 0, dv // 2, dk - 1] == bad and not torch.isfinite(y[0, :, 0, dv // 2]).any()
    if dtype == "bf16":
        assert (y[0, :, 0, dv // 2] == bad).all()
    y[0, :, 0, dv // 2], s[0, 0, dv // 2, dk - 1] = y0[0, :, 0, dv // 2], s0[0, 0, dv // 2, dk - 1]
    assert torch.equal(y, y0) and torch.equal(s, s0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, dtype):
    """Of an infinite dy: dq of its token, dk and dv of the tokens up to it, and the state's gradient."""
    a = positive(shape, dtype, 102)
    b, L, H, G, dk, dv = shape
    d = gpu(a)
    g0 = ms.lin_attn_bwd(*bwd_args(d))
    for at in (0, 65, L - 1):
        t = d["dy"].clone()
        t[0, at, -1, dv - 1] = -INF
        g = ms.lin_attn_bwd(*bwd_args(dict(d, dy=t)))
        torch.cuda.synchronize()
        hit = {n: torch.zeros_like(x, dtype=torch.bool) for n, x in g.items()}
        hit["dq"][0, at, -1] = hit["dk"][0, :at + 1, -1] = True
        hit["dv"][0, :at + 1, -1, dv - 1] = True
        hit["dstate"][0, -1, dv - 1] = True
        for n in g:
            assert torch.equal(g[n][~hit[n]], g0[n][~hit[n]]), (n, at)
            assert not torch.isfinite(g[n][hit[n]]).any(), (n, at)
            if n in ("dv", "dstate") and dtype == "bf16":  # here dy is the value
                assert (g[n][hit[n]] == -INF).all(), (n, at)


def test_infinities_of_both_signs_and_zeros():
    """Infinities of two signs in one column, and infinity times a key of 0, are NaN there, and nothing elsewhere."""
    a = positive((1, 200, 1, 1, 72, 64), "bf16", 103)
    d = gpu(a)
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d))
    v, k = d["v"].clone(), d["k"].clone()
    v[0, 30, 0, 5], v[0, 120, 0, 5], v[0, 150, 0, 6], k[0, 150, 0, 70] = INF, -INF, INF, 0.0
    y, s = ms.lin_attn_fwd(d["q"], k, v, d["log_decay"], d["state"])
    y1, s1 = ms.lin_attn_fwd(d["q"], k, d["v"], d["log_decay"], d["state"])
    torch.cuda.synchronize()
    assert (y[0, 30:120, 0, 5] == INF).all() and torch.isnan(y[0, 120:, 0, 5]).all() and torch.isnan(s[0, 0, 5]).all()
    assert torch.isnan(s[0, 0, 6, 70]) and (s[0, 0, 6, :70] == INF).all()
    # the token itself sums its scores before the value comes to them, later ones read the state's NaN
    assert (y[0, 150:192, 0, 6] == INF).all() and torch.isnan(y[0, 192:, 0, 6]).all()
    y[..., 5:7], s[:, :, 5:7] = y1[..., 5:7], s1[:, :, 5:7]
    y[:, :30], y1[:, :30] = y0[:, :30], y0[:, :30]
    assert torch.equal(y, y1) and torch.equal(s, s1)
