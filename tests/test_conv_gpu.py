"""The short causal convolution on the GPU against the fp64 oracle: outputs,
states and gradients at every number of taps and io type, lengths from one
token on, runs that end inside a row, packed documents, carried states, split
and strided tensors, odd channels, infinities and NaN in other documents,
offsets past 2^31 elements, streams and captured graphs.

The bounds are counted, not fitted. With U = 2^-24, u has k + 1 roundings of
its terms' magnitudes; silu(u) = u / (1 + e^-u) moves by at most 1.1 times
that, and by (2 |u| + 6) U of itself (the exponent's rounding stands |u| log2 e
from 0, the two instructions and three products have one or two each). Its
derivative moves by at most 0.5 times u's error and (2 |u| + 8) U of 1.1. Sums
over tokens add a rounding for each term, and an output in bfloat16 half a
step, 2^-8 of itself."""
import sys

import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import conv as oc
from oracle.linattn import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(b, L, c, k, dtype, seed=0, state=False, docs=0, bias=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(b, L, c + wide, generator=g).to(dtype)[..., wide // 2:wide // 2 + c]
    a = dict(x=x, weight=torch.rand(c, k, generator=g) - 0.5, bias=0.1 * torch.randn(c, generator=g) if bias else None,
             state=torch.randn(b, c, k - 1, generator=g) if state else None, seq_idx=None)
    if docs:
        a["seq_idx"] = torch.cumsum(torch.rand(b, L, generator=g) < 1.0 / docs, 1).to(torch.int32)
    dy = torch.randn(b, L, c, generator=g).to(dtype)
    ds = torch.randn(b, c, k - 1, generator=g) if state else None
    return a, dy, ds


def cuda(a):
    """On the GPU, strides kept."""
    if isinstance(a, dict):
        return {n: cuda(t) for n, t in a.items()}
    if a is None:
        return None
    base = torch.empty_strided(a.shape, a.stride(), dtype=a.dtype, device="cuda")
    return base.copy_(a)


def magnitude(a):
    """(u, the sum of its terms' magnitudes) of every token"""
    plain = dict(a, activation="none")
    u, _ = oc.oracle_fwd(**plain)
    size, _ = oc.oracle_fwd(**{n: None if t is None else np.abs(f64(t)) if n != "seq_idx" else t for n, t in a.items()},
                            activation="none")
    return u, size


def hold(got, want, tol, what, dtype=torch.float32):
    got = f64(got)
    tol = tol + (BF * np.abs(want) + BF * tol if dtype == torch.bfloat16 else 0) + 1e-37
    assert got.shape == want.shape and np.isfinite(got).all(), what
    err = np.abs(got - want)
    at = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), "%s: %g off at %s, %g allowed" % (what, err[at], at, tol[at])


def check_fwd(a, got, activation, what):
    y, last = got
    y = torch.cat(y, -1) if isinstance(y, tuple) else y
    want, state = oc.oracle_fwd(**a, activation=activation)
    u, size = magnitude(a)
    k = a["weight"].shape[1]
    tol = (k + 2) * U * size
    if activation == "silu":
        tol = 1.1 * tol + (2 * np.abs(u) + 6) * U * np.abs(want)
    hold(y, want, tol, what + " y", a["x"].dtype)
    if last is not None:
        assert (f64(last) == state).all(), what + " state"


def check_bwd(a, dy, ds, got, activation, what):
    want = oc.oracle_bwd(dy=dy, dstate=ds, activation=activation, **a)
    u, size = magnitude(a)
    b, L, c = a["x"].shape
    k = a["weight"].shape[1]
    err = (k + 2) * U * size * 0.5 + (2 * np.abs(u) + 8) * 1.1 * U if activation == "silu" else np.zeros_like(u)
    du = np.abs(f64(dy)) * 1.1
    err = np.abs(f64(dy)) * err + U * du
    ab = {n: None if t is None else np.abs(f64(t)) for n, t in a.items() if n != "seq_idx"}

    def through(e, s):
        return oc.oracle_bwd(dy=e, dstate=s, activation="none", seq_idx=a["seq_idx"], **ab)

    off, mag = through(err, None), through(du, None if ds is None else np.abs(f64(ds)))
    n = {"dx": k + 2, "dstate": k + 2, "dweight": b * L + 8, "dbias": b * L + 8}
    names = {"dx", "dweight"} | ({"dbias"} if a["bias"] is not None else set()) | ({"dstate"} if a["state"] is not None else set())
    assert set(got) == names
    for name in got:
        hold(got[name], want[name], off[name] + n[name] * U * mag[name], what + " " + name,
             a["x"].dtype if name == "dx" else torch.float32)


SHAPES = [
    # batch, seqlen, channels
    (1, 1, 8), (3, 1, 16), (2, 2, 64), (1, 3, 264), (2, 15, 40), (1, 16, 512), (2, 17, 24), (1, 33, 1792), (3, 64, 8),
    (1, 127, 256), (2, 129, 96), (1, 513, 72), (40, 7, 32), (1, 2050, 264), (9, 300, 520),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward_and_gradients(i, dtype):
    b, L, c = SHAPES[i]
    k = 2 + i % 3 if i % 2 else 4
    act = "none" if i % 4 == 2 else "silu"
    a, dy, ds = make(b, L, c, k, DT[dtype], seed=i, state=i % 3 != 0, bias=i % 5 != 1)
    print(SHAPES[i], k, act, dtype, flush=True)
    g = cuda(a)
    got = ms.conv_fwd(**g, activation=act)
    torch.cuda.synchronize()
    check_fwd(a, got, act, "conv")
    grads = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), activation=act, **g)
    torch.cuda.synchronize()
    check_bwd(a, dy, ds, grads, act, "conv")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,L,c,k,docs", [(2, 200, 48, 4, 3), (1, 65, 24, 3, 1), (3, 700, 264, 4, 40), (2, 100, 21, 2, 2),
                                          (2, 3, 16, 4, 2), (2, 333, 17, 4, 9)])
def test_packed_documents(b, L, c, k, docs, dtype):
    a, dy, ds = make(b, L, c, k, DT[dtype], seed=L, state=True, docs=docs)
    g = cuda(a)
    got = ms.conv_fwd(**g)
    grads = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), **g)
    torch.cuda.synchronize()
    check_fwd(a, got, "silu", "packed")
    check_bwd(a, dy, ds, grads, "silu", "packed")


def test_same_id_again_is_a_new_document():
    """Ids are compared with the one before alone: 5 5 7 7 5 5 are three documents."""
    a, dy, ds = make(1, 6, 8, 4, torch.float32, state=True)
    a["seq_idx"] = torch.tensor([[5, 5, 7, 7, 5, 5]])
    g = cuda(a)
    got, grads = ms.conv_fwd(**g), ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), **g)
    torch.cuda.synchronize()
    check_fwd(a, got, "silu", "ids")
    check_bwd(a, dy, ds, grads, "silu", "ids")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c,split,wide", [(1792, (1536, 128, 128), 1560), (72, (8, 64), 16), (30, (7, 3, 15, 5), 3), (24, (24,), 0),
                                          (40, (36, 4), 8), (21, None, 5)])
def test_split_and_strided(c, split, wide, dtype):
    a, dy, _ = make(2, 70, c, 4, DT[dtype], seed=c, wide=wide)
    g = cuda(a)
    assert wide == 0 or not g["x"].is_contiguous()
    got = ms.conv_fwd(**g, split=split)
    assert split is None or [y.shape[-1] for y in got[0]] == list(split) and all(y.is_contiguous() for y in got[0])
    check_fwd(a, got, "silu", "split")
    dys = dy.cuda()
    parts = dys.split(split, -1) if split else dys  # columns of one tensor, read in place
    grads = ms.conv_bwd(dy=parts, **g)
    torch.cuda.synchronize()
    check_bwd(a, dy, None, grads, "silu", "split")


def test_vector_and_element_paths_agree_bitwise():
    """A tensor that starts off a 16-byte boundary is read element by element, with the same sums for each channel."""
    a, dy, _ = make(2, 150, 64, 4, torch.bfloat16, seed=3, docs=20)
    g = cuda(a)
    off = torch.empty(2 * 150 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 150, 64).copy_(g["x"])
    one, two = ms.conv_fwd(**g), ms.conv_fwd(**dict(g, x=off))
    d1, d2 = ms.conv_bwd(dy=dy.cuda(), **g), ms.conv_bwd(dy=dy.cuda(), **dict(g, x=off))
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1]) and torch.equal(d1["dx"], d2["dx"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,c,k,split", [(1, 8, 4, None), (5, 33, 3, (30, 3)), (256, 1792, 4, (1536, 128, 128)), (3, 64, 2, None)])
def test_step(b, c, k, split, dtype):
    a, _, _ = make(b, 6, c, k, DT[dtype], seed=b, state=True, wide=8)
    g = cuda(a)
    state, ys = g["state"].clone(), []
    for t in range(6):
        y, new = ms.conv_step(g["x"][:, t], g["weight"], g["bias"], state, split=split, inplace=t % 2 == 1)
        assert (new is state) == (t % 2 == 1)
        state = new
        ys.append(torch.cat(y, -1) if split else y)
    torch.cuda.synchronize()
    check_fwd(a, (torch.stack(ys, 1), state), "silu", "step")


def test_prompt_then_tokens_bitwise():
    a, _, _ = make(3, 40, 72, 4, torch.bfloat16, seed=9)
    g = cuda(a)
    whole, last = ms.conv_fwd(**g)
    y, s = ms.conv_fwd(g["x"][:, :33], g["weight"], g["bias"])
    parts = [y]
    for t in range(33, 40):
        y, s = ms.conv_step(g["x"][:, t], g["weight"], g["bias"], s)
        parts.append(y[:, None])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, last)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_documents_and_earlier_tokens_keep_their_bits(bad):
    a, dy, ds = make(1, 90, 16, 4, torch.bfloat16, seed=4, state=True)
    a["seq_idx"] = torch.zeros(1, 90, dtype=torch.int32)
    a["seq_idx"][:, 31:60], a["seq_idx"][:, 60:] = 1, 2
    g, d = cuda(a), dy.cuda()
    want, wd = ms.conv_fwd(**g), ms.conv_bwd(dy=d, dstate=cuda(ds), **g)
    x, d2 = g["x"].clone(), d.clone()
    x[:, 31:60] = bad
    d2[:, 31:60] = bad
    got, gd = ms.conv_fwd(**dict(g, x=x)), ms.conv_bwd(dy=d2, dstate=cuda(ds), **dict(g, x=x))
    torch.cuda.synchronize()
    out = torch.ones(90, dtype=torch.bool)
    out[31:60] = False
    out = out.cuda()
    assert torch.equal(got[0][:, out], want[0][:, out]) and torch.equal(got[1], want[1])
    assert torch.equal(gd["dx"][:, out], wd["dx"][:, out]) and torch.equal(gd["dstate"], wd["dstate"])
    x = g["x"].clone()
    x[:, 20] = bad
    got = ms.conv_fwd(**dict(g, x=x))
    torch.cuda.synchronize()
    assert torch.equal(got[0][:, :20], want[0][:, :20]) and torch.equal(got[0][:, 24:], want[0][:, 24:])


def test_silu_closes_at_the_lowest_values():
    x = torch.tensor([-float("inf"), -3e38, -1e4, -200.0, 0.0, 200.0, 3e38, float("inf")]).repeat(1, 1, 1).cuda()
    w = torch.zeros(8, 2)
    w[:, 1] = 1
    y, _ = ms.conv_fwd(x, w.cuda())
    dx = ms.conv_bwd(x, w.cuda(), torch.ones_like(x))["dx"]
    torch.cuda.synchronize()
    want = [0.0, 0.0, 0.0, 0.0, 0.0, 200.0, 3e38, float("inf")]
    assert torch.equal(y.cpu()[0, 0].abs(), torch.tensor(want))
    assert torch.allclose(dx.cpu()[0, 0], torch.tensor([0, 0, 0, 0, 0.5, 1, 1, 1.0]), atol=1e-6)


def test_given_outputs_and_workspace_and_determinism():
    a, dy, ds = make(2, 300, 136, 4, torch.float32, seed=11, state=True, docs=30)
    g = cuda(a)
    ys = [torch.full((2, 300, n), 7.0, device="cuda") for n in (128, 8)]
    st = torch.full((2, 136, 3), 7.0, device="cuda")
    got = ms.conv_fwd(**g, split=(128, 8), out=ys, state_out=st)
    assert got[0][0] is ys[0] and got[1] is st
    check_fwd(a, got, "silu", "given")
    need = ms.conv_workspace_bytes(2, 300, 136, 4, torch.float32)
    first = None
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        grads = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), workspace=ws, **g)
        torch.cuda.synchronize()
        first = first or grads
        assert all(torch.equal(grads[n], first[n]) for n in grads)
    check_bwd(a, dy, ds, first, "silu", "workspace")
    assert ms.conv_fwd(**g, return_state=False)[1] is None


def test_stream_and_captured_graph():
    a, dy, ds = make(2, 257, 64, 4, torch.bfloat16, seed=12, state=True)
    g, d, s = cuda(a), dy.cuda(), cuda(ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ms.conv_fwd(**g)
        ms.conv_bwd(dy=d, dstate=s, **g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = ms.conv_fwd(**g)
        grads = ms.conv_bwd(dy=d, dstate=s, **g)
    for i in range(3):
        g["x"].copy_(torch.randn(g["x"].shape, generator=torch.Generator().manual_seed(i)))
        want, wl = ms.conv_fwd(**g)
        wg = ms.conv_bwd(dy=d, dstate=s, **g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(last, wl)
        assert all(torch.equal(grads[n], wg[n]) for n in wg)


def test_past_two_to_the_31_elements():
    """The last tokens of a row whose elements pass 2^31 are those of a call on them alone, from the state before them."""
    L, c, n = (1 << 31) // 1032 + 4096, 1032, 50
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, L, c, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    w, bias = torch.rand(c, 4, device="cuda", generator=g) - 0.5, torch.randn(c, device="cuda", generator=g)
    y, last = ms.conv_fwd(x, w, bias)
    before = x[:, L - n - 3:L - n].float().transpose(1, 2).contiguous()
    y2, last2 = ms.conv_fwd(x[:, L - n:], w, bias, before)
    torch.cuda.synchronize()
    assert torch.equal(y[:, L - n:], y2) and torch.equal(last, last2)
    grads = ms.conv_bwd(x, w, y, bias)
    tail = ms.conv_bwd(x[:, L - n:], w, y2, bias, before)
    torch.cuda.synchronize()
    assert torch.equal(grads["dx"][:, L - n:], tail["dx"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("docs", [0, 7])
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("c", [260, 67])
def test_every_kernel(c, k, docs, act, dtype):
    """Taps, documents, activations, types, and channels by four and one by one: a kernel for each."""
    for L in (1, 2, 3, 5, 38, 1027):
        a, dy, ds = make(2, L, c, k, DT[dtype], seed=L + k, state=True, docs=docs)
        g = cuda(a)
        print(c, k, docs, act, dtype, L, flush=True)
        got = ms.conv_fwd(**g, activation=act)
        grads = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), activation=act, **g)
        torch.cuda.synchronize()
        check_fwd(a, got, act, "every")
        check_bwd(a, dy, ds, grads, act, "every")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_another_documents_values_reach_none(value, dtype):
    """x and dy of the second document, which begins and ends inside runs, hold nothing finite."""
    a, dy, ds = make(2, 150, 72, 4, DT[dtype], seed=5, state=True)
    ids = torch.zeros(2, 150, dtype=torch.int32)
    ids[:, 21:] = 1
    ids[:, 90:] = 2
    a["seq_idx"] = ids
    clean = (ids != 1).numpy()
    y0, s0 = ms.conv_fwd(**cuda(a))
    d0 = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), **cuda(a))
    a["x"][:, 21:90] = value
    dy[:, 21:90] = value
    y1, s1 = ms.conv_fwd(**cuda(a))
    d1 = ms.conv_bwd(dy=dy.cuda(), dstate=cuda(ds), **cuda(a))
    torch.cuda.synchronize()
    for u, v in ((y0, y1), (d0["dx"], d1["dx"])):
        assert torch.equal(u.cpu()[clean], v.cpu()[clean])
    assert torch.equal(s0, s1) and torch.equal(d0["dstate"], d1["dstate"])
