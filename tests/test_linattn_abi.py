"""Linear attention without a GPU: the header's functions are exported and
bound, sizes of the workspaces, every refusal of the C ABI before any HIP call,
and the front end's reading of row strides."""
import os
import re

import pytest
import torch

import selective_state_space_07_amd as ms
from selective_state_space_07_amd import _binding as _b
from selective_state_space_07_amd import linattn

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mamba_linattn.h")
# Fake, never-dereferenced device addresses: validation must reject every call
# below before any HIP call.
P = 0x7F0000000000
G = 0x10000000


@pytest.fixture(scope="module")
def lib():
    return linattn.load()


def test_header_and_exports_match(lib):
    declared = set(re.findall(r"^\s*(?:int|size_t)\s+(mamba_linattn_\w+)\s*\(", open(HEADER).read(), re.M))
    assert declared == set(linattn.EXPORTS)
    for name in declared:
        assert hasattr(lib, name)


def call(lib, what, **over):
    a = dict(batch=2, seqlen=8, nheads=4, ngroups=2, d_k=64, d_v=32, io=0, scale=1.0, q=P, qs=128, k=P + G, ks=128,
             v=P + 2 * G, vs=128, ids=0, g=P + 3 * G, s=0, dy=P + 4 * G, dys=128, dso=0, y=P + 5 * G, so=P + 6 * G,
             dq=P + 7 * G, dk=P + 8 * G, dv=P + 9 * G, dsi=0, ws=P + 10 * G, wb=1 << 24)
    if what == "step":
        a.update(s=P + 11 * G)
    a.update(over)
    io = [a[n] for n in ("q", "qs", "k", "ks", "v", "vs")]
    dims = [a[n] for n in ("batch", "seqlen", "nheads", "ngroups", "d_k", "d_v", "io")]
    if what == "fwd":
        return lib.mamba_linattn_fwd(*dims, a["scale"], *io, a["ids"], a["g"], a["s"], a["y"], a["so"], a["ws"], a["wb"], 0)
    if what == "bwd":
        return lib.mamba_linattn_bwd(*dims, a["scale"], *io, a["ids"], a["g"], a["s"], a["dy"], a["dys"], a["dso"],
                                     a["dq"], a["dk"], a["dv"], a["dsi"], a["ws"], a["wb"], 0)
    del dims[1]
    return lib.mamba_linattn_step(*dims, a["scale"], *io, a["g"], a["s"], a["y"], a["so"], 0)


DIMS = [
    (dict(batch=0), 2), (dict(nheads=0), 2), (dict(ngroups=0), 2), (dict(nheads=-4), 2), (dict(ngroups=3), 2),
    (dict(d_k=0), 2), (dict(d_k=12), 2), (dict(d_k=136), 2), (dict(d_v=4), 2), (dict(d_v=130), 2), (dict(d_v=-8), 2),
    (dict(nheads=4098, vs=4098 * 32), 2), (dict(batch=1 << 19), 2), (dict(io=2), 3), (dict(io=-1), 3),
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(g=0), 1),
    (dict(qs=127), 2), (dict(ks=0), 2), (dict(vs=-128), 2), (dict(qs=(1 << 24) + 4), 2), (dict(g=P + 3 * G + 2), 4),
]


@pytest.mark.parametrize("what,over,status", [(w, o, s) for w in ("fwd", "bwd", "step") for o, s in DIMS] + [
    ("fwd", dict(seqlen=0), 2), ("bwd", dict(seqlen=-1), 2), ("fwd", dict(seqlen=(1 << 30) + 1), 2),
    ("fwd", dict(batch=4, seqlen=1 << 29), 2),
    ("fwd", dict(q=P + 8), 4), ("fwd", dict(io=1, vs=132), 4), ("fwd", dict(y=P + 5 * G + 4), 4),
    ("fwd", dict(s=P + 11 * G + 4), 4), ("fwd", dict(so=P + 6 * G + 8), 4), ("fwd", dict(ids=P + 11 * G + 2), 4),
    ("fwd", dict(y=0), 1), ("bwd", dict(dy=0), 1), ("bwd", dict(dq=0), 1), ("bwd", dict(dk=0), 1), ("bwd", dict(dv=0), 1),
    ("bwd", dict(dys=127), 2), ("bwd", dict(dq=P + 7 * G + 8), 4), ("bwd", dict(dsi=P + 11 * G + 4), 4),
    ("bwd", dict(dso=P + 11 * G + 4), 4),
    ("fwd", dict(y=P), 5), ("fwd", dict(y=P + 4 * (15 * 128)), 5), ("fwd", dict(so=P + 5 * G + 16), 5),
    # y inside q's last row at a row stride of 1024
    ("fwd", dict(qs=1024, y=P + 4 * (15 * 1024 + 64)), 5),
    ("fwd", dict(s=P + 6 * G + 16), 5), ("fwd", dict(ids=P + 5 * G), 5), ("fwd", dict(y=P + 3 * G), 5),
    ("bwd", dict(dq=P + 4 * G), 5), ("bwd", dict(dq=P + 8 * G), 5), ("bwd", dict(s=P + 11 * G, dsi=P + 11 * G), 5),
    ("bwd", dict(dso=P + 11 * G, dsi=P + 11 * G), 5), ("bwd", dict(ws=P + 7 * G), 5),
    ("bwd", dict(ws=0), 6), ("bwd", dict(wb=16), 6), ("bwd", dict(ws=P + 10 * G + 64), 4),
    ("fwd", dict(seqlen=4096, wb=16), 6), ("fwd", dict(seqlen=4096, ws=0), 6),
    ("fwd", dict(seqlen=4096, ws=P + 5 * G, wb=1 << 30), 5),
    ("step", dict(s=0), 1), ("step", dict(so=0), 1), ("step", dict(y=0), 1), ("step", dict(s=P + 6 * G + 16), 5),
    ("step", dict(y=P + 64), 5), ("step", dict(io=1, q=P + 1), 4), ("step", dict(q=P + 2), 4),
])
def test_validation(lib, what, over, status):
    assert call(lib, what, **over) == status, ms.mamba_scan_last_error()
    assert ms.mamba_scan_status_str(status) in ms.mamba_scan_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("what,over", [
    ("fwd", {}), ("bwd", {}), ("step", {}), ("fwd", dict(so=0, ws=0, wb=0)), ("fwd", dict(s=P + 6 * G)),
    ("step", dict(s=P + 6 * G)), ("fwd", dict(q=P, k=P + 512, v=P + 1024, qs=512, ks=512, vs=512)),
    ("bwd", dict(ngroups=4, qs=256, ks=256, ws=0, wb=0)),
    ("step", dict(io=1, q=P + 2, k=P + G + 2, v=P + 2 * G + 2, y=P + 5 * G + 2, qs=129, ks=131, vs=129)),
])
def test_valid_calls_reach_the_device_check(lib, what, over):
    assert call(lib, what, **over) == 7, ms.mamba_scan_last_error()


def test_workspaces(lib):
    bf = torch.bfloat16
    assert ms.lin_attn_workspace_bytes(1, 64, 4, 4, 64, 64, bf) == 0       # one chunk
    assert ms.lin_attn_workspace_bytes(1, 65536, 4, 4, 64, 64, bf) > 0     # split into segments
    assert ms.lin_attn_workspace_bytes(64, 65536, 16, 16, 64, 64, bf) == 0  # enough heads to go unsplit
    for bad in ((0, 64, 4, 4, 64, 64), (1, 0, 4, 4, 64, 64), (1, 64, 4, 3, 64, 64), (1, 64, 4, 4, 60, 64)):
        assert ms.lin_attn_workspace_bytes(*bad, bf) == 0
        assert ms.lin_attn_workspace_bytes(*bad, bf, backward=True) == 0
    # dq and dk of every head in float32, where heads share them
    assert ms.lin_attn_workspace_bytes(2, 64, 4, 1, 64, 64, bf, backward=True) >= 2 * 2 * 64 * 4 * 64 * 4
    # the segments' states stay bounded however long the sequence
    assert ms.lin_attn_workspace_bytes(1, 1 << 30, 1, 1, 128, 128, bf) < 1 << 27


@pytest.mark.parametrize("shape,strides,nrow,want", [
    ((2, 5, 4, 8), (160, 32, 8, 1), 2, 32),
    ((2, 5, 4, 8), (500, 100, 8, 1), 2, 100),    # columns of rows of 100
    ((2, 5, 4, 8), (400, 100, 8, 1), 2, 0),      # batch rows closer than their tokens
    ((2, 5, 4, 8), (1000, 100, 8, 1), 2, 0),     # a part of a longer sequence
    ((1, 5, 4, 8), (7, 100, 8, 1), 2, 100),      # one batch row: its stride says nothing
    ((2, 1, 4, 8), (100, 3, 8, 1), 2, 100),      # one token: the batch rows' stride
    ((2, 5, 4, 8), (160, 32, 1, 4), 2, 0),       # heads and their elements exchanged
    ((2, 5, 4, 8), (0, 0, 8, 1), 2, 0),          # one row repeated
    ((2, 5, 4, 8), (80, 16, 8, 1), 2, 0),        # rows that overlap
    ((2, 5, 1, 8), (80, 16, 3, 1), 2, 16),       # one head: its stride says nothing
    ((3, 4, 8), (64, 8, 1), 1, 64),
    ((1, 1, 4, 8), (9, 9, 8, 1), 2, 32),
    ((2, 2, 1, 8), (1 << 26, 1 << 25, 8, 1), 2, 0),  # past the largest row stride
])
def test_row_stride(shape, strides, nrow, want):
    assert linattn.row_stride(shape, strides, nrow) == want


def test_front_end_refusals():
    cpu = torch.zeros(1, 4, 2, 8)
    with pytest.raises(_b.MambaScanError) as e:
        ms.lin_attn_fwd(cpu, cpu, cpu, torch.zeros(2))
    assert e.value.status == 7
    with pytest.raises(TypeError):
        ms.lin_attn_fwd(cpu.double(), cpu, cpu, torch.zeros(2))
    with pytest.raises(TypeError):
        ms.lin_attn_step([1.0], cpu, cpu, torch.zeros(2), cpu)
