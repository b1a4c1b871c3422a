"""The SSD scan's gradients without a GPU: workspace sizes and every refusal of
the C ABI before any HIP call."""
import pytest
import torch

import selective_state_space_07_amd as ms
from selective_state_space_07_amd import _binding as _b

P = 0x7F0000000000  # fake addresses, never dereferenced
G = 0x10000000
IN = ("x", "dt", "B", "C")
OUT = ("dx", "ddt", "dB", "dC", "ddt_bias", "dA", "dD", "dsi", "ws")
AT = {n: P + i * G for i, n in enumerate((*IN, "ids", "dt_bias", "A", "D", "si", "dy", "dso", *OUT))}


def call(**over):
    a = dict(AT, b=2, L=16, H=4, P=64, N=64, G=2, io=0, xs=256, dts=4, Bs=128, Cs=128, dys=256, wb=1 << 30)
    a.update(over)
    args = [a[n] for n in ("b", "L", "H", "P", "N", "G", "io")]
    for n in IN:
        args += [a[n], a[n + "s"]]
    args += [a[n] for n in ("ids", "dt_bias", "A", "D", "si", "dy", "dys", "dso", *OUT, "wb")]
    return _b.mamba2_ssd_bwd(*args, 0, check=False)


@pytest.mark.parametrize("over,status", [
    (dict(b=0), 2), (dict(L=0), 2), (dict(H=0), 2), (dict(G=0), 2), (dict(G=3), 2), (dict(P=32), 2), (dict(N=96), 2),
    (dict(b=65536), 2), (dict(H=65536 * 2, G=2), 2), (dict(L=1 << 24), 2), (dict(io=2), 3),
    *[({n: 0}, 1) for n in (*IN, "dy", "dt_bias", "A", "D", "dx", "ddt", "dB", "dC", "ddt_bias", "dA", "dD")],
    (dict(xs=255), 2), (dict(dts=3), 2), (dict(Bs=127), 2), (dict(Cs=0), 2), (dict(dys=(1 << 24) + 4), 2),
    (dict(xs=257), 4), (dict(Bs=130), 4), (dict(io=1, Cs=132), 4), (dict(x=AT["x"] + 8), 4), (dict(dt=AT["dt"] + 2), 4),
    (dict(dy=AT["dy"] + 4), 4), (dict(ids=AT["ids"] + 2), 4), (dict(si=AT["si"] + 4), 4), (dict(dso=AT["dso"] + 8), 4),
    (dict(dx=AT["dx"] + 4), 4), (dict(ddt=AT["ddt"] + 2), 4), (dict(dB=AT["dB"] + 8), 4), (dict(dA=AT["dA"] + 2), 4),
    (dict(dsi=AT["dsi"] + 4), 4), (dict(A=AT["A"] + 1), 4),
    (dict(dx=AT["x"]), 5), (dict(dx=AT["dy"] + 16), 5), (dict(dB=AT["C"]), 5), (dict(dC=AT["dB"]), 5), (dict(dsi=AT["si"]), 5),
    (dict(dsi=AT["dso"]), 5), (dict(dA=AT["dD"]), 5), (dict(ddt_bias=AT["dt_bias"]), 5), (dict(ws=AT["x"]), 5),
    (dict(ws=AT["dx"]), 5), (dict(ddt=AT["ids"]), 5),
    (dict(ws=0), 6), (dict(wb=1024), 6), (dict(ws=AT["ws"] + 16), 4),
])
def test_validation(over, status):
    assert call(**over) == status, ms.mamba_scan_last_error()
    assert ms.mamba_scan_status_str(status) in ms.mamba_scan_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("over", [{}, dict(ids=0, si=0, dso=0, dsi=0), dict(io=1, dt=AT["dt"] + 2, dts=5), dict(xs=512, dys=1024),
                                  dict(B=AT["x"], Bs=512, xs=512), dict(N=128, Bs=256, Cs=256)])
def test_valid_calls_reach_the_device_check(over):
    assert call(**over) == 7, ms.mamba_scan_last_error()


def test_workspaces():
    bf = torch.bfloat16
    one = ms.ssd_bwd_workspace_bytes(8, 2048, 24, 64, 128, 1, bf)
    states = 2 * 8 * 8 * 24 * 64 * 128 * 4
    assert states < one < 2 * states
    for bad in ((0, 2048, 24, 64, 128, 1), (8, 2048, 24, 32, 128, 1), (8, 2048, 24, 64, 100, 1), (8, 2048, 24, 64, 128, 5)):
        assert ms.ssd_bwd_workspace_bytes(*bad, bf) == 0


def test_front_end_refusals():
    x, dt, B = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2), torch.zeros(1, 4, 1, 64)
    p = torch.zeros(2)
    with pytest.raises(_b.MambaScanError) as e:
        ms.ssd_bwd(x, dt, B, B, p, p, p, x)
    assert e.value.status == 7
    with pytest.raises(TypeError):
        ms.ssd_bwd(x.double(), dt, B, B, p, p, p, x)
