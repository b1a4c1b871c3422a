"""The group norm without a GPU: the header's functions are exported and bound,
workspace sizes, and every refusal of the C ABI before any HIP call."""
import os
import re

import pytest
import torch

import selective_state_space_07_amd as ms
from selective_state_space_07_amd import _binding as _b
from selective_state_space_07_amd import gnorm

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mamba_gnorm.h")
P = 0x7F0000000000  # fake addresses, never dereferenced
G = 0x10000000


@pytest.fixture(scope="module")
def lib():
    return gnorm.load()


def test_header_and_exports_match(lib):
    declared = set(re.findall(r"^\s*(?:int|size_t)\s+(mamba_gnorm_\w+)\s*\(", open(HEADER).read(), re.M))
    assert declared == set(gnorm.EXPORTS)
    for name in declared:
        assert hasattr(lib, name)


def call(lib, what, **over):
    a = dict(rows=4, c=64, groups=4, io=0, act=1, gate=1, center=1, eps=1e-5, x=P, xs=64, z=P + G, zs=64, w=P + 2 * G,
             b=P + 3 * G, dy=P + 4 * G, dys=64, y=P + 5 * G, dz=P + 6 * G, dw=P + 7 * G, db=P + 8 * G, ws=P + 9 * G,
             wb=1 << 20)
    a.update(over)
    head = [a[n] for n in ("rows", "c", "groups", "io", "act", "gate", "center", "eps", "x", "xs", "z", "zs", "w", "b")]
    if what == "fwd":
        return lib.mamba_gnorm_fwd(*head, a["y"], 0)
    return lib.mamba_gnorm_bwd(*head, *[a[n] for n in ("dy", "dys", "y", "dz", "dw", "db", "ws", "wb")], 0)


BOTH = [
    (dict(rows=0), 2), (dict(rows=-5), 2), (dict(c=0), 2), (dict(groups=0), 2), (dict(groups=3), 2),
    (dict(c=16385, groups=1, xs=16385, zs=16385, dys=16385), 2), (dict(c=(1 << 20) + 64, groups=1 << 14), 2),
    (dict(rows=1 << 29), 2), (dict(rows=1 << 40), 2), (dict(io=2), 3), (dict(act=3), 2), (dict(act=-1), 2),
    (dict(gate=3), 2), (dict(gate=-1), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(x=0), 1), (dict(z=0), 1), (dict(y=0), 1), (dict(gate=0), 2),
    (dict(xs=63), 2), (dict(zs=0), 2), (dict(xs=(1 << 24) + 1), 2),
    (dict(x=P + 2), 4), (dict(io=1, z=P + G + 1), 4), (dict(w=P + 2 * G + 2), 4), (dict(b=P + 3 * G + 1), 4),
    (dict(y=P + 5 * G + 2), 4),
    (dict(y=P), 5), (dict(y=P + 4), 5), (dict(xs=1000, y=P + 4 * 3010), 5), (dict(y=P + G + 1020), 5),
    (dict(y=P + 2 * G), 5), (dict(y=P + 3 * G + 252), 5),
]


@pytest.mark.parametrize("what,over,status", [(w, o, s) for w in ("fwd", "bwd") for o, s in BOTH] + [
    ("bwd", dict(dy=0), 1), ("bwd", dict(dz=0), 1), ("bwd", dict(gate=0, z=0), 2), ("bwd", dict(dys=10), 2),
    ("bwd", dict(dz=P + 6 * G + 2), 4), ("bwd", dict(dw=P + 7 * G + 2), 4), ("bwd", dict(db=P + 8 * G + 2), 4),
    ("bwd", dict(dz=P + 5 * G), 5), ("bwd", dict(dw=P + 8 * G), 5), ("bwd", dict(y=P + 4 * G), 5),
    ("bwd", dict(ws=P + 5 * G), 5), ("bwd", dict(ws=0), 6), ("bwd", dict(wb=64), 6), ("bwd", dict(ws=P + 9 * G + 16), 4),
])
def test_validation(lib, what, over, status):
    assert call(lib, what, **over) == status, ms.mamba_scan_last_error()
    assert ms.mamba_scan_status_str(status) in ms.mamba_scan_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("what,over", [
    ("fwd", {}), ("bwd", {}), ("fwd", dict(w=0, b=0, gate=2)), ("fwd", dict(gate=0, z=0, act=0)),
    ("bwd", dict(gate=0, z=0, dz=0)), ("bwd", dict(w=0, b=0, dw=0, db=0, ws=0, wb=0)), ("fwd", dict(z=P, zs=128, xs=128)),
    ("fwd", dict(io=1, x=P + 2, y=P + 5 * G + 2, xs=65)), ("fwd", dict(eps=0.0)),
])
def test_valid_calls_reach_the_device_check(lib, what, over):
    assert call(lib, what, **over) == 7, ms.mamba_scan_last_error()


def test_workspaces(lib):
    bf = torch.bfloat16
    one = ms.group_norm_workspace_bytes(16384, 1536, 1, bf, bias=False)
    assert 0 < one and ms.group_norm_workspace_bytes(16384, 1536, 1, bf) == 2 * one
    assert ms.group_norm_workspace_bytes(16384, 1536, 1, bf, weight=False, bias=False) == 0
    assert ms.group_norm_workspace_bytes(0, 1536, 1, bf) == 0
    assert ms.group_norm_workspace_bytes(10, 1536, 7, bf) == 0


def test_front_end_refusals():
    x = torch.zeros(4, 8)
    for bad, status in ((dict(activation="gelu"), 2), (dict(gate_first=True), 1), (dict(), 7)):
        with pytest.raises(_b.MambaScanError) as e:
            ms.group_norm_fwd(x, None, None, 2, **bad)
        assert e.value.status == status
    with pytest.raises(TypeError):
        ms.group_norm_fwd(x.double(), None, None, 2)
    with pytest.raises(TypeError):
        ms.group_norm_fwd([1.0], None, None, 2)
