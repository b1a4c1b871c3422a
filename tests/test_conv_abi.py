"""The short causal convolution without a GPU: the header's functions are
exported and bound, workspace sizes, and every refusal of the C ABI before any
HIP call."""
import ctypes
import os
import re

import pytest
import torch

import selective_state_space_07_amd as ms
from selective_state_space_07_amd import _binding as _b
from selective_state_space_07_amd import conv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mamba_conv.h")
P = 0x7F0000000000  # fake addresses, never dereferenced
G = 0x10000000


@pytest.fixture(scope="module")
def lib():
    return conv.load()


def test_header_and_exports_match(lib):
    text = open(HEADER).read()
    declared = set(re.findall(r"^\s*(?:int|size_t)\s+(mamba_conv_\w+)\s*\(", text, re.M))
    assert declared == set(conv.EXPORTS)
    for name in declared:
        assert hasattr(lib, name)
    assert int(re.search(r"#define MAMBA_CONV_MAX_PARTS (\d+)", text).group(1)) == conv.MAX_PARTS


def call(lib, what, **over):
    a = dict(b=2, L=16, c=64, k=4, io=0, act=1, x=P, xs=64, ids=P + G, w=P + 2 * G, bias=P + 3 * G, s=P + 4 * G, n=2,
             sizes=(48, 16), parts=(P + 5 * G, P + 6 * G), strides=(48, 16), so=P + 7 * G, dso=P + 8 * G, dx=P + 9 * G,
             dw=P + 10 * G, db=P + 11 * G, dsi=P + 12 * G, ws=P + 13 * G, wb=1 << 24)
    a.update(over)
    sizes = (ctypes.c_int32 * 8)(*a["sizes"]) if a["sizes"] else None
    parts = (ctypes.c_void_p * 8)(*a["parts"]) if a["parts"] else None
    strides = (ctypes.c_int64 * 8)(*a["strides"]) if a["strides"] else None
    if what == "step":
        return lib.mamba_conv_step(a["b"], a["c"], a["k"], a["io"], a["act"], a["x"], a["xs"], a["w"], a["bias"], a["s"], a["n"],
                                   sizes, parts, a["so"], 0)
    head = [a[n] for n in ("b", "L", "c", "k", "io", "act", "x", "xs", "ids", "w", "bias", "s", "n")] + [sizes, parts]
    if what == "fwd":
        return lib.mamba_conv_fwd(*head, a["so"], 0)
    return lib.mamba_conv_bwd(*head, strides, *[a[n] for n in ("dso", "dx", "dw", "db", "dsi", "ws", "wb")], 0)


ALL = [
    (dict(b=0), 2), (dict(c=0), 2), (dict(c=-3), 2), (dict(k=1), 2), (dict(k=5), 2), (dict(c=(1 << 20) + 1), 2),
    (dict(b=(1 << 24) + 1), 2), (dict(io=2), 3), (dict(act=2), 2), (dict(act=-1), 2), (dict(x=0), 1), (dict(w=0), 1),
    (dict(xs=63), 2), (dict(xs=(1 << 24) + 1), 2), (dict(x=P + 2), 4), (dict(w=P + 2 * G + 2), 4), (dict(bias=P + 3 * G + 1), 4),
    (dict(s=P + 4 * G + 2), 4), (dict(n=0), 2), (dict(n=5), 2), (dict(sizes=None), 1), (dict(parts=None), 1),
    (dict(parts=(P + 5 * G, 0)), 1), (dict(parts=(P + 5 * G + 2, P + 6 * G)), 4), (dict(sizes=(48, 15)), 2),
    (dict(sizes=(64, 0)), 2), (dict(sizes=(48, 17), strides=(48, 17)), 2), (dict(n=1), 2),
]
OUT = [  # y of a forward call or of a step
    (dict(parts=(P, P + 6 * G)), 5), (dict(parts=(P + 5 * G, P + 5 * G + 4)), 5), (dict(parts=(P + 5 * G, P + 2 * G)), 5),
    (dict(parts=(P + 5 * G, P + 7 * G)), 5), (dict(so=P + 4 * G + 4), 5), (dict(so=P + 7 * G + 2), 4), (dict(so=P), 5),
]


@pytest.mark.parametrize("what,over,status", [(w, o, s) for w in ("fwd", "bwd", "step") for o, s in ALL] +
                         [(w, o, s) for w in ("fwd", "step") for o, s in OUT] + [
    ("fwd", dict(L=0), 2), ("fwd", dict(b=1 << 12, L=1 << 19), 2), ("fwd", dict(ids=P + G + 2), 4), ("fwd", dict(so=P + 4 * G), 5),
    ("fwd", dict(parts=(P + G, P + 6 * G)), 5), ("bwd", dict(L=-1), 2), ("bwd", dict(strides=None), 1),
    ("bwd", dict(strides=(47, 16)), 2), ("bwd", dict(dx=0), 1), ("bwd", dict(dw=0), 1), ("bwd", dict(dx=P + 9 * G + 2), 4),
    ("bwd", dict(dw=P + 10 * G + 1), 4), ("bwd", dict(dso=P + 8 * G + 2), 4), ("bwd", dict(dsi=P + 12 * G + 2), 4),
    ("bwd", dict(dx=P), 5), ("bwd", dict(dx=P + 5 * G), 5), ("bwd", dict(dw=P + 2 * G), 5), ("bwd", dict(dsi=P + 4 * G), 5),
    ("bwd", dict(dsi=P + 8 * G), 5), ("bwd", dict(db=P + 10 * G), 5), ("bwd", dict(ws=P + 9 * G), 5), ("bwd", dict(ws=0), 6),
    ("bwd", dict(wb=64), 6), ("bwd", dict(ws=P + 13 * G + 16), 4), ("step", dict(s=0), 1), ("step", dict(so=0), 1),
])
def test_validation(lib, what, over, status):
    assert call(lib, what, **over) == status, ms.mamba_scan_last_error()
    assert ms.mamba_scan_status_str(status) in ms.mamba_scan_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake addresses")
@pytest.mark.parametrize("what,over", [
    ("fwd", {}), ("bwd", {}), ("step", {}), ("step", dict(so=P + 4 * G)), ("fwd", dict(ids=0, bias=0, s=0, so=0)),
    ("bwd", dict(ids=0, bias=0, s=0, dso=0, db=0, dsi=0)), ("fwd", dict(n=1, sizes=(64,))), ("fwd", dict(xs=1000)),
    ("fwd", dict(io=1, x=P + 2, parts=(P + 5 * G + 2, P + 6 * G + 2), xs=65)), ("bwd", dict(strides=(64, 100), act=0, k=2)),
    ("fwd", dict(c=1, xs=1, n=1, sizes=(1,), b=1, L=1)),
])
def test_valid_calls_reach_the_device_check(lib, what, over):
    assert call(lib, what, **over) == 7, ms.mamba_scan_last_error()


def test_workspaces():
    need = ms.conv_workspace_bytes(8, 2048, 1792, 4, torch.bfloat16)
    assert 0 < need < 8 * 2048 * 1792 * 2
    assert ms.conv_workspace_bytes(8, 0, 1792, 4, torch.bfloat16) == 0
    assert ms.conv_workspace_bytes(8, 2048, 1792, 5, torch.bfloat16) == 0


def test_front_end_refusals():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for bad, status in ((dict(activation="gelu"), 2), (dict(), 7)):
        with pytest.raises(_b.MambaScanError) as e:
            ms.conv_fwd(x, w, **bad)
        assert e.value.status == status
    with pytest.raises(_b.MambaScanError):
        ms.conv_step(x[:, 0], w, None, None)
    with pytest.raises(_b.MambaScanError):
        ms.conv_fwd(x[0], w)
    with pytest.raises(TypeError):
        ms.conv_fwd(x.double(), w)
    for split in ((4, 5), (8, 0), (1, 1, 1, 1, 4), ()):
        with pytest.raises(_b.MambaScanError):
            conv._sizes(split, 8)


def test_as_many_tokens_as_numbers_hold(lib):
    """A run's end and the tokens read ahead of it are int32 numbers."""
    for what in ("fwd", "bwd"):
        assert call(lib, what, b=1, L=1 << 30) == 2 and "2^30" in ms.mamba_scan_last_error()
        assert call(lib, what, b=1, L=(1 << 30) - 1, ids=0) != 2 or "2^30" not in ms.mamba_scan_last_error()
    assert ms.conv_workspace_bytes(1, 1 << 30, 8, 4, torch.float32) == 0
    assert ms.conv_workspace_bytes(1, (1 << 30) - 1, 8, 4, torch.float32) > 0
