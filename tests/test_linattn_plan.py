"""The split of a sequence into segments, read off the workspace that it needs
(CPU): whole segments of at least four chunks of 64 tokens, none of them empty,
and none where there is enough to do without."""
import itertools

import pytest
import torch

from selective_state_space_07_amd import linattn as L


def segments(batch, seqlen, nheads, ngroups, d_k, d_v, dtype, backward):
    """(number of segments, bytes left over behind their states and flags)."""
    n = L.lin_attn_workspace_bytes(batch, seqlen, nheads, ngroups, d_k, d_v, dtype, backward=backward) // 4
    roles = 3 if backward else 1
    kd, vd = (max(d_k, d_v),) * 2 if backward else (d_k, d_v)
    if backward and nheads != ngroups:
        n -= 2 * batch * seqlen * nheads * d_k  # dq and dk of every head
    state = roles * batch * nheads * -(-vd // 64) * 64 * (64 if kd <= 64 else 128)
    nseg = n // state
    flags = (roles * batch * nseg + 63) // 64 * 64
    return nseg, n - nseg * state - (flags if nseg else 0)


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_segments_are_whole_and_long_enough(backward):
    sizes = itertools.product([1, 2, 7, 64], [1, 64, 65, 255, 256, 300, 512, 513, 1501, 4133, 65536, 1 << 20],
                              [(1, 1), (12, 3), (24, 24)], [(8, 8), (64, 96), (128, 128)])
    for batch, seqlen, (nheads, ngroups), (d_k, d_v) in sizes:
        nseg, rest = segments(batch, seqlen, nheads, ngroups, d_k, d_v, torch.bfloat16, backward)
        what = (batch, seqlen, nheads, ngroups, d_k, d_v)
        assert rest == 0, what
        chunks = -(-seqlen // 64)
        assert nseg <= min(256, chunks // 4), what
        assert nseg != 1, what  # a single one needs no workspace
        if nseg:
            assert -(-chunks // -(-chunks // nseg)) == nseg, what
        if batch * nheads >= 256:
            assert nseg == 0, what


def test_refused_sizes_need_nothing():
    assert L.lin_attn_workspace_bytes(1, 1 << 20, 4, 3, 64, 64, torch.float32) == 0
    assert L.lin_attn_workspace_bytes(1, 1 << 20, 4, 4, 60, 64, torch.float32) == 0
