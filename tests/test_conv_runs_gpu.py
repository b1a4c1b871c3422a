"""The short causal convolution where workgroups come round more than once: a
backward's wave with the runs of several short rows (its sums go on, all else
begins anew), a forward and a one-token call with more than a launch's
workgroups. Gradients against the fp64 oracle to the bounds of
tests/test_conv_gpu.py; what a row alone decides, bit for bit as in a call on
that row."""
import pytest
import torch

import selective_state_space_07_amd as ms
from tests.test_conv_gpu import DT, check_bwd, check_fwd, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("docs", [0, 2])
@pytest.mark.parametrize("b,L,c,k", [(4000, 3, 260, 4), (4000, 3, 67, 4), (6200, 1, 260, 3), (3100, 7, 65, 2), (1601, 9, 516, 4)])
def test_many_short_rows(b, L, c, k, docs, dtype):
    """Of 768 workgroups for each of the call's column groups, four rows at a time: every wave has two to five."""
    print(b, L, c, k, docs, dtype, flush=True)
    a, dy, ds = make(b, L, c, k, DT[dtype], seed=b + L, state=True, docs=docs)
    g = cuda(a)
    got = ms.conv_fwd(**g)
    grads = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), **g)
    torch.cuda.synchronize()
    check_fwd(a, got, "silu", "rows")
    check_bwd(a, dy, ds, grads, "silu", "rows")
    s = slice(b - 50, b)
    one = ms.conv_bwd(dy=dy.cuda()[s], dstate=cuda(ds)[s], **{n: t[s] if n in ("x", "state", "seq_idx") and t is not None else t
                                                              for n, t in g.items()})
    torch.cuda.synchronize()
    assert torch.equal(one["dx"], grads["dx"][s]) and torch.equal(one["dstate"], grads["dstate"][s])


def test_more_rows_than_workgroups():
    b, c = 1 << 24, 260
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(b, 1, c, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w, bias = torch.rand(c, 4, device="cuda", generator=gen) - 0.5, torch.randn(c, device="cuda", generator=gen)
    y, _ = ms.conv_fwd(x, w, bias, return_state=False)
    for lo in (0, (1 << 23) - 25, b - 50):
        one, _ = ms.conv_fwd(x[lo:lo + 50], w, bias, return_state=False)
        torch.cuda.synchronize()
        assert torch.equal(y[lo:lo + 50], one), lo


def test_more_tokens_than_threads():
    b, c = (1 << 20) + 9, 260
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(b, c, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    state = torch.empty(b, c, 3, device="cuda").normal_(generator=gen)
    w, bias = torch.rand(c, 4, device="cuda", generator=gen) - 0.5, torch.randn(c, device="cuda", generator=gen)
    y, new = ms.conv_step(x, w, bias, state)
    for lo in (0, (1 << 28) // c - 25, b - 50):
        one, last = ms.conv_step(x[lo:lo + 50], w, bias, state[lo:lo + 50])
        torch.cuda.synchronize()
        assert torch.equal(y[lo:lo + 50], one) and torch.equal(new[lo:lo + 50], last), lo
