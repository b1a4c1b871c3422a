"""Tensors with a dimension of zero: linear attention and the group norm refuse
them as the library refuses any other size, before anything is launched."""
import pytest
import torch

import selective_state_space_07_amd as ms

pytestmark = pytest.mark.gpu


def refused(f, *args, **kw):
    with pytest.raises(ms.MambaScanError) as e:
        f(*args, **kw)
    assert e.value.status == 2, str(e.value)


@pytest.mark.parametrize("scale", [None, 1.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [(0, 5, 4, 2, 8, 8), (2, 0, 4, 2, 8, 8), (2, 5, 0, 2, 8, 8), (2, 5, 4, 0, 8, 8),
                                  (2, 5, 4, 2, 0, 8), (2, 5, 4, 2, 8, 0), (0, 0, 0, 0, 0, 0)], ids=str)
def test_linear_attention(size, dtype, scale):
    b, L, H, G, dk, dv = size
    new = lambda *s, dtype=dtype: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    q, v, g = new(b, L, G, dk), new(b, L, H, dv), new(H, dtype=torch.float32)
    s = new(b, H, dv, dk, dtype=torch.float32)
    for state in (None, s):
        refused(ms.lin_attn_fwd, q, q, v, g, state, scale=scale)
        refused(ms.lin_attn_bwd, q, q, v, g, v, state, scale=scale)
    refused(ms.lin_attn_fwd, q, q, v, g, scale=scale, seq_idx=new(b, L, dtype=torch.int32))
    if L:
        for inplace in (False, True):
            refused(ms.lin_attn_step, q[:, 0], q[:, 0], v[:, 0], g, s, scale=scale, inplace=inplace)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(0, 16), (3, 0), (0, 5, 16), (0,), (0, 0)], ids=str)
def test_group_norm(shape, dtype):
    x = torch.zeros(*shape, device="cuda", dtype=dtype)
    w = torch.ones(shape[-1], device="cuda")
    for groups in (0, 1, 4):
        for z in (None, x):
            refused(ms.group_norm_fwd, x, w, w, groups, z)
            refused(ms.group_norm_bwd, x, w, w, groups, x, z)
