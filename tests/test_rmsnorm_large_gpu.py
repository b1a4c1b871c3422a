"""The RMS norm at row counts whose workgroups, one a row, would have 2^32
threads and more: every row is as in a call on it alone."""
import pytest
import torch

import selective_state_space_07_amd as ms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [(1 << 22) - 1, 1 << 22])
def test_a_row_for_each_of_the_largest_workgroups(rows):
    c = 3841  # single elements, four a lane: 1024 threads a row
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        torch.cuda.empty_cache()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, c, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(c, device="cuda", generator=g)
    print(rows, c, flush=True)
    y, _ = ms.add_rms_norm_fwd(x, None, w)
    torch.cuda.synchronize()
    for lo in (0, (1 << 20) - 3, (1 << 21) - 3, rows - 77):
        one, _ = ms.add_rms_norm_fwd(x[lo:lo + 77], None, w)
        torch.cuda.synchronize()
        assert torch.equal(y[lo:lo + 77], one), lo
    del x, y
    torch.cuda.empty_cache()
