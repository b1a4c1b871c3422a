"""The RMS norm with the residual's addition where x and the residual are
columns of wider tensors: rows any multiple of 16 bytes apart, each tensor's by
its own type, so a float32 residual's may be 4 elements off those of bfloat16
x. Every output is held to the oracle, to the bounds of tests/test_rmsnorm_gpu.py,
and the memory that outputs come from holds something else before each call.
"""
import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import rmsnorm as orn
from tests.test_rmsnorm_gpu import TYPES, U, check_bwd, check_fwd, cuda, half, hold, make, stands_for

pytestmark = pytest.mark.gpu


def columns(t, more):
    """t on the GPU as the first columns of a tensor that is `more` wider."""
    wide = torch.full((t.shape[0], t.shape[1] + more), 7.0, dtype=t.dtype, device="cuda")
    view = wide[:, :t.shape[1]]
    view.copy_(t)
    return view, wide


def dirty(*shapes):
    """Memory of these sizes goes back to the allocator filled with 0x55."""
    keep = [torch.full((int(np.prod(s)) * 4,), 0x55, dtype=torch.uint8, device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del keep


def check8(x, r, w, q, scales, h, block, what):
    wy, wh = orn.oracle_fwd(x, r, w)
    ws, each = orn.oracle_scales(wy, block)
    hold(scales, ws, 36 * U * ws, what + " scales")
    hold(stands_for(q, scales, block), wy, (2.0 ** -4 + 40 * U) * np.abs(wy) + 2.0 ** -10 * (1 + 40 * U) * each, what + " y")
    hold(h, wh, (U + half(r.dtype) * (1 + U)) * np.abs(wh), what + " h")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("more_x,more_r", [(0, 4), (8, 0), (8, 4), (8, 12), (16, 8)])
@pytest.mark.parametrize("rows,c", [(1, 16), (37, 48), (9, 144), (20, 768), (50, 2048), (3, 4112), (2, 16384)])
def test_rows_of_each_type_apart(rows, c, more_x, more_r, types):
    x, r, w, dy, dh = make(rows, c, *types, seed=rows + c)
    if types[1] == "bf16":
        more_r *= 2  # 16 bytes
    print(rows, c, more_x, more_r, types, flush=True)
    gx, wide_x = columns(x, more_x)
    gr, wide_r = columns(r, more_r)
    gw = cuda(w)
    for block in (None, 128):
        dirty((rows, c), (rows, -(-c // 128)))
        q, scales, h = ms.add_rms_norm_fp8(gx, gr, gw, block=block)
        torch.cuda.synchronize()
        check8(x, r, w, q, scales, h, block, "8 bits")
    dirty((rows, c))
    y, h = ms.add_rms_norm_fwd(gx, gr, gw)
    torch.cuda.synchronize()
    check_fwd(x, r, w, y, h, "forward")
    gdy, _ = columns(dy, more_x)
    gdh, _ = columns(dh, more_r)
    dirty((rows, c), (c,))
    grads = ms.add_rms_norm_bwd(gr, gw, gdy, gdh)
    torch.cuda.synchronize()
    check_bwd(r, w, dy, dh, grads, "gradients")
    # (what lies beside the columns is as it was)
    assert (wide_x[:, c:] == 7).all() and (wide_r[:, c:] == 7).all()


@pytest.mark.parametrize("block", [None, 128])
def test_rows_at_the_front_ends_own_strides(block):
    """A residual that starts inside a wider tensor's row, 16-byte aligned, and one that does not (which is copied)."""
    rows, c = 70, 768
    x, r, w, _, _ = make(rows, c, "bf16", "f32", seed=5)
    for at in (4, 1):
        wide = torch.zeros(rows, c + 20, device="cuda")
        view = wide[:, at:at + c]
        view.copy_(r)
        dirty((rows, c), (rows, 6))
        q, scales, h = ms.add_rms_norm_fp8(cuda(x), view, cuda(w), block=block)
        torch.cuda.synchronize()
        check8(x, r, w, q, scales, h, block, "at %d" % at)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("block", [None, 128])
def test_in_place_beside_columns(block, types):
    """x as columns, h over the (contiguous) residual."""
    for rows, c in ((40, 144), (9, 2048)):
        x, r, w, _, _ = make(rows, c, *types, seed=c)
        gx, _ = columns(x, 8)
        gr = cuda(r)
        dirty((rows, c), (rows, 16))
        q, scales, h = ms.add_rms_norm_fp8(gx, gr, cuda(w), block=block, inplace=True)
        torch.cuda.synchronize()
        assert h is gr
        check8(x, r, w, q, scales, h, block, "in place")
