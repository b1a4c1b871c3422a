"""Gradients of the Mamba-2 SSD scan at counts of workgroups whose threads pass
2^32: the largest batch, one token a row, and so many groups of heads. Every
row is as in a call on it alone."""
import pytest
import torch

import selective_state_space_07_amd as ms

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_than_two_to_the_32_threads(dtype):
    b, H, N = 65535, 33, 64
    need = ms.ssd_bwd_workspace_bytes(b, 1, H, 64, N, H, dtype)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip("needs %d GB of device memory" % ((need + (16 << 30)) >> 30))
    print(b, H, N, dtype, need, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dtype)  # noqa: E731
    x, dy, B, C, dt = rnd(b, 1, H, 64), rnd(b, 1, H, 64), rnd(b, 1, H, N), rnd(b, 1, H, N), rnd(b, 1, H)
    par = [torch.randn(H, device="cuda", generator=g), -torch.rand(H, device="cuda", generator=g),
           torch.randn(H, device="cuda", generator=g)]
    got = ms.ssd_bwd(x, dt, B, C, *par, dy)
    torch.cuda.synchronize()
    for lo in (0, 31774, 63548, b - 40):  # (31775 rows of 33 groups are the first 2^22 workgroups)
        s = slice(lo, lo + 40)
        one = ms.ssd_bwd(x[s], dt[s], B[s], C[s], *par, dy[s])
        torch.cuda.synchronize()
        for n in ("dx", "ddt", "dB", "dC"):
            assert torch.equal(got[n][s], one[n]), (lo, n)
    terms = (x.double() * dy.double())
    want, size = terms.sum((0, 1, 3)), terms.abs().sum((0, 1, 3))
    assert ((got["dD"].double() - want).abs() <= (64 + b + 40) * U * size).all()
    del x, dy, B, C, dt, got, terms
    torch.cuda.empty_cache()
