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
@pytest.mark.parametrize("shape", [(2, 600, 3, 3, 64, 64), (1, 1500, 2, 1, 128, 128)], ids=str)
def test_bfloat16_outputs_have_two_roundings_in_the_mean(shape, keep):
    """A value rounded to bfloat16 is off by 2^-8 / sqrt(3) / m of itself, m its significand in [1, 2): in the mean of
    squares, with m spread as numbers are (evenly in its logarithm), sqrt(0.75 / (2 ln 2)) of that, 1.66e-3. An output
    is rounded once. The scores and the state that it is made of, which are its terms' only factors that are not
    inputs, are rounded once each on their way into it: another 1.66e-3 of the root of the sum of the terms' squares,
    which is the output's size where signs are random. Together sqrt(2) times 1.66e-3 = 2.35e-3; a state rounded twice
    would make it up to sqrt(3) times. The bound leaves a twentieth for the spread of 1e5 values."""
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
        assert err <= 1.05 * 2 ** 0.5 * one, n
