"""Linear attention on the GPU at the ends of its types' ranges: finite values up
to the highest and lowest in each operand, with partners so small that what they
enter stays finite.

Bounds as in test_linattn_gpu.py. A float32 is three bfloat16 parts, of which the
first is cut, not rounded (rounding would take values beyond 3.38e38 to infinity):
the second is below 2^-7 of the value and the third at most 2^-16, so that they
hold it whole and the products that are left out are below 2 * 2^-23 + 2^-32 of
the product, 4 u; its six others are added one by one: 6 c + 5 instead of c."""
import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import linattn as la
from tests.test_linattn_gpu import BF, DT, U, absolute, bwd_args, fwd_args, gpu, make, say, steps

pytestmark = pytest.mark.gpu
SMALL = 2.0 ** -20  # on every other tensor: three factors and sums of hundreds of terms stay far below 1e38


def extremes(dtype):
    f = torch.finfo(dtype)
    ends = [f.max, f.min]
    if dtype == torch.float32:  # on either side of what rounds to infinity in bfloat16
        ends += [3.3895e38, -3.39e38, 3.4e38]
    return ends


def close(got, want, size, a, what, rounded):
    got = got.detach().cpu().double().numpy()
    bf16 = a["q"].dtype == torch.bfloat16
    tol = (6 * steps(a) + 5) * U * size + 1e-30
    if rounded and bf16:
        tol = tol + BF * np.abs(want) + BF * (1 + BF) * size
    assert np.isfinite(got).all(), "%s: %d not finite" % (what, (~np.isfinite(got)).sum())
    assert (np.abs(got - want) <= tol).all(), what


@pytest.mark.parametrize("docs", [0, 90], ids=["one", "packed"])
@pytest.mark.parametrize("which", ["q", "k", "v", "dy", "state", "dstate"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 200, 2, 1, 64, 72), (1, 1100, 1, 1, 128, 40)], ids=str)
def test_the_highest_and_lowest_values(shape, dtype, which, docs):
    say("extremes", shape, dtype, which, docs)
    a = make(*shape, DT[dtype], seed=61, state=True, docs=docs, backward=True)
    for n in ("q", "k", "v", "dy", "state", "dstate"):
        a[n] = a[n] * SMALL
    t = a[which]
    at = torch.randperm(t.numel(), generator=torch.Generator().manual_seed(62))
    for i, v in enumerate(extremes(t.dtype) * 4):
        t.view(-1)[at[i]] = v
    d = gpu(a)
    got = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    alone = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"], return_state=False)
    grads = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    kw = dict(seq_idx=a["seq_idx"])
    want, size = la.oracle_fwd(*fwd_args(a), **kw), la.oracle_fwd(*fwd_args(absolute(a)), **kw)
    close(got[0], want[0], size[0], a, "y", True)
    close(alone[0], want[0], size[0], a, "y without the state", True)
    close(got[1], want[1], size[1], a, "state", False)
    want, size = la.oracle_bwd(*bwd_args(a), **kw), la.oracle_bwd(*bwd_args(absolute(a)), **kw)
    for n in grads:
        close(grads[n], want[n], size[n], a, n, n != "dstate")


@pytest.mark.parametrize("which", ["q", "k", "v", "state"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token(dtype, which):
    a = make(5, 1, 4, 2, 64, 40, DT[dtype], seed=63, state=True)
    for n in ("q", "k", "v", "state"):
        a[n] = a[n] * SMALL
    t = a[which]
    for i, v in enumerate(extremes(t.dtype)):
        t.view(-1)[7 + 61 * i] = v
    d = gpu(a)
    y, s = ms.lin_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"])
    torch.cuda.synchronize()
    want, size = la.oracle_fwd(*fwd_args(a)), la.oracle_fwd(*fwd_args(absolute(a)))
    close(y, want[0][:, 0], size[0][:, 0], a, "y", True)
    close(s, want[1], size[1], a, "state", False)


def test_an_infinity_in_float32_is_not_finite_where_it_enters():
    """It may come out as NaN there (infinity times the parts of a value that are 0), but nowhere else."""
    a = make(1, 200, 2, 2, 64, 64, torch.float32, seed=64)
    d = gpu(a)
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d))
    for bad in (float("inf"), -float("inf")):
        v = d["v"].clone()
        v[0, 70, 1, 9] = bad
        y, s = ms.lin_attn_fwd(d["q"], d["k"], v, d["log_decay"])
        torch.cuda.synchronize()
        assert not torch.isfinite(y[0, 70:, 1, 9]).any() and not torch.isfinite(s[0, 1, 9]).any()
        y[0, 70:, 1, 9], s[0, 1, 9] = y0[0, 70:, 1, 9], s0[0, 1, 9]
        assert torch.isfinite(y).all() and torch.equal(s, s0)
        torch.testing.assert_close(y, y0, rtol=2e-5, atol=2e-5)
