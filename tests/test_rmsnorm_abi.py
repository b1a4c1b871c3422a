"""The RMS norm with the residual's addition without a GPU: the header's
functions are exported and bound, workspace sizes, and every refusal of the C
ABI before any HIP call."""
import os
import re

import pytest
import torch

import selective_state_space_07_amd as ms
from selective_state_space_07_amd import _binding as _b
from selective_state_space_07_amd import rmsnorm

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mamba_rmsnorm.h")
P = 0x7F0000000000  # fake addresses, never dereferenced
G = 0x10000000


@pytest.fixture(scope="module")
def lib():
    return rmsnorm.load()


def test_header_and_exports_match(lib):
    declared = set(re.findall(r"^\s*(?:int|size_t)\s+(mamba_rmsnorm_\w+)\s*\(", open(HEADER).read(), re.M))
    assert declared == set(rmsnorm.EXPORTS)
    for name in declared:
        assert hasattr(lib, name)


def call(lib, what, **over):
    a = dict(rows=4, c=64, io=0, res=0, eps=1e-5, block=0, x=P, xs=64, r=P + G, rs=64, w=P + 2 * G, y=P + 3 * G, h=P + 4 * G,
             sc=P + 5 * G, dy=P + 6 * G, dys=64, dh=P + 7 * G, dhs=64, dx=P + 8 * G, dr=P + 9 * G, dw=P + 10 * G, ws=P + 11 * G,
             wb=1 << 20)
    a.update(over)
    head = [a[n] for n in ("rows", "c", "io", "res", "eps")]
    if what == "fwd":
        return lib.mamba_rmsnorm_fwd(*head, *[a[n] for n in ("x", "xs", "r", "rs", "w", "y", "h")], 0)
    if what == "fp8":
        return lib.mamba_rmsnorm_fp8(*head, *[a[n] for n in ("block", "x", "xs", "r", "rs", "w", "y", "sc", "h")], 0)
    return lib.mamba_rmsnorm_bwd(*head, *[a[n] for n in ("x", "xs", "w", "dy", "dys", "dh", "dhs", "dx", "dr", "dw", "ws", "wb")], 0)


ALL = [
    (dict(rows=0), 2), (dict(rows=-1), 2), (dict(c=0), 2), (dict(c=16385, xs=20000, rs=20000, dys=20000, dhs=20000), 2),
    (dict(rows=1 << 31), 2), (dict(io=2), 3), (dict(io=-1), 3), (dict(res=2), 3), (dict(res=1), 3), (dict(eps=-1.0), 2),
    (dict(eps=float("nan")), 2), (dict(x=0), 1), (dict(xs=63), 2), (dict(xs=(1 << 24) + 1), 2), (dict(x=P + 2), 4),
    (dict(w=P + 2 * G + 2), 4),
]
FWD = [
    (dict(rs=63), 2), (dict(r=P + G + 2), 4), (dict(y=0), 1), (dict(y=P + 3 * G + 1), 4), (dict(h=P + 4 * G + 2), 4),
    (dict(y=P), 5), (dict(y=P + 240), 5), (dict(y=P + G), 5), (dict(y=P + 2 * G), 5), (dict(h=P), 5), (dict(h=P + G + 16), 5),
    (dict(h=P + 3 * G), 5), (dict(rs=80, h=P + G), 5),
]


@pytest.mark.parametrize("what,over,status", [(w, o, s) for w in ("fwd", "fp8", "bwd") for o, s in ALL] +
                         [(w, o, s) for w in ("fwd", "fp8") for o, s in FWD] + [
    ("fp8", dict(block=64), 2), ("fp8", dict(block=-128), 2), ("fp8", dict(c=56), 2), ("fp8", dict(sc=0), 1),
    ("fp8", dict(sc=P + 5 * G + 2), 4), ("fp8", dict(xs=65), 4), ("fp8", dict(x=P + 4), 4), ("fp8", dict(r=P + G + 8), 4),
    ("fp8", dict(y=P + 3 * G + 8), 4), ("fp8", dict(sc=P + 4 * G + 1020), 5),
    ("bwd", dict(dy=0), 1), ("bwd", dict(dys=8), 2), ("bwd", dict(dhs=8), 2), ("bwd", dict(dx=0, dr=0), 1),
    ("bwd", dict(dx=P + 8 * G + 2), 4), ("bwd", dict(dr=P + 9 * G + 2), 4), ("bwd", dict(dw=P + 10 * G + 2), 4),
    ("bwd", dict(dx=P), 5), ("bwd", dict(dx=P + 6 * G), 5), ("bwd", dict(dx=P + 7 * G), 5), ("bwd", dict(dr=P + 8 * G), 5),
    ("bwd", dict(dw=P + 2 * G), 5), ("bwd", dict(ws=P + 9 * G), 5), ("bwd", dict(ws=0), 6), ("bwd", dict(wb=16), 6),
    ("bwd", dict(ws=P + 11 * G + 16), 4),
])
def test_validation(lib, what, over, status):
    assert call(lib, what, **over) == status, ms.mamba_scan_last_error()
    assert ms.mamba_scan_status_str(status) in ms.mamba_scan_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("what,over", [
    ("fwd", {}), ("fp8", {}), ("bwd", {}), ("fwd", dict(h=P + G)), ("fwd", dict(r=0, rs=0, h=0, w=0)), ("fp8", dict(block=128, h=P + G)),
    ("fwd", dict(io=1, res=1, x=P + 2, xs=65)), ("fwd", dict(io=1, res=0)), ("bwd", dict(dr=P + 7 * G)), ("bwd", dict(dx=0)),
    ("bwd", dict(dr=0)), ("bwd", dict(dh=0, dhs=0, w=0, dw=0, ws=0, wb=0)), ("fwd", dict(eps=0.0, c=1, xs=1, rs=1)),
])
def test_valid_calls_reach_the_device_check(lib, what, over):
    assert call(lib, what, **over) == 7, ms.mamba_scan_last_error()


def test_workspaces(lib):
    need = ms.add_rms_norm_workspace_bytes(16384, 768, torch.bfloat16)
    assert 0 < need < 16384 * 768 * 2
    assert ms.add_rms_norm_workspace_bytes(0, 768, torch.bfloat16) == 0
    assert lib.mamba_rmsnorm_bwd_workspace_bytes(16384, 768, 1, 0, 0) == 0


def test_front_end_refusals():
    x = torch.zeros(4, 16)
    for f, status in ((lambda: ms.add_rms_norm_fwd(x, x, None), 7), (lambda: ms.add_rms_norm_fp8(x, x, None, block=64), 2),
                      (lambda: ms.add_rms_norm_fwd(x, None, None, inplace=True), 7)):
        with pytest.raises(_b.MambaScanError) as e:
            f()
        assert e.value.status == status
    with pytest.raises(TypeError):
        ms.add_rms_norm_fwd(x.double(), None, None)
    with pytest.raises(TypeError):
        ms.add_rms_norm_bwd(x, None, [1.0])
