"""Linear attention on the GPU with many heads on few groups and batch rows, and
how exact its outputs are in the mean. Bounds as in test_linattn_gpu.py."""
import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import linattn as la
from tests.test_linattn_gpu import DT, bwd_args, check_bwd, check_fwd, fwd_args, gpu, make, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("docs", [0, 60], ids=["one", "packed"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 256, 48, 1, 128, 128), (1, 1024, 32, 1, 32, 40), (3, 130, 24, 1, 64, 64),
                                   (1, 700, 14, 2, 64, 128), (1, 70, 9, 3, 8, 8), (7, 65, 5, 1, 24, 16)], ids=str)
def test_few_groups(shape, dtype, docs):
    """Fewer pairs of a batch row and a group than the card has XCDs."""
    say("few groups", shape, dtype, docs)
    a = make(*shape, DT[dtype], seed=sum(shape), state=True, docs=docs, backward=True)
    d = gpu(a)
    got = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    grads = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    check_fwd(a, got, str(shape))
    check_bwd(a, grads, str(shape))


@pytest.mark.parametrize("keep", [False, True], ids=["alone", "with_state"])
@pytest.mark.parametrize("shape", [(2, 600, 3, 3, 64, 64), (1, 1500, 2, 1, 128, 128), (1, 17, 12, 12, 64, 64)], ids=str)
def test_bfloat16_outputs_have_one_rounding_in_the_mean(shape, keep):
    """A value rounded to bfloat16 is off by 2^-8 / sqrt(3) / m of itself, m its significand in [1, 2): in the mean of
    squares, with m spread as numbers are (evenly in its logarithm), sqrt(0.75 / (2 ln 2)) of that, 1.66e-3. An output
    is rounded once, at its end; a score or a state that was rounded on its way into it, as they are factors of all
    its terms, would add as much again and make it sqrt(2) times that. The bound leaves a twentieth for the spread of
    1e4 values."""
    a = make(*shape, torch.bfloat16, seed=5, state=True, backward=True)
    d = gpu(a)
    y, _ = ms.lin_attn_fwd(*fwd_args(d), return_state=keep)
    g = ms.lin_attn_bwd(*bwd_args(d))
    torch.cuda.synchronize()
    one = 2.0 ** -8 / 3 ** 0.5 * (0.75 / (2 * np.log(2))) ** 0.5
    want = dict(la.oracle_bwd(*bwd_args(a)), y=la.oracle_fwd(*fwd_args(a))[0])
    for n, t in dict(dq=g["dq"], dk=g["dk"], dv=g["dv"], y=y).items():
        err = np.linalg.norm(t.cpu().double().numpy() - want[n]) / np.linalg.norm(want[n])
        say(n, "%.3g" % err)
        assert err <= 1.05 * one, n


@pytest.mark.parametrize("docs", [0, 60], ids=["one", "packed"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 333, 3, 1, 64, 64), (1, 1500, 2, 2, 128, 72)], ids=str)
def test_outputs_do_not_depend_on_which_are_wanted(shape, dtype, docs):
    """The same bits whether or not the state, or its gradient, is asked for."""
    a = make(*shape, DT[dtype], seed=6, state=True, docs=docs, backward=True)
    d = gpu(a)
    kw = dict(seq_idx=d["seq_idx"])
    y = [ms.lin_attn_fwd(*fwd_args(d), **kw, return_state=keep)[0] for keep in (True, False)]
    args = bwd_args(d)
    g = [ms.lin_attn_bwd(*args[:5], s, **kw) for s in (None, torch.zeros_like(d["state"]))]
    torch.cuda.synchronize()
    assert torch.equal(*y) and "dstate" not in g[0] and "dstate" in g[1]
    for n in g[0]:
        assert torch.equal(g[0][n], g[1][n]), n
