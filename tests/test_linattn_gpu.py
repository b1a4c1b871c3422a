"""Linear attention with a decay for each head on the GPU against the fp64
oracle: every output, every direction and io type, at head sizes that fill a
tile and that do not, lengths around the chunk and segment edges, shared
heads, carried states, packed documents, strided rows, infinities and NaN in
masked places, offsets past 2^31 elements, streams and captured graphs.

The bounds are counted, not fitted. With u = 2^-24, float32 arithmetic leaves
each output within c u of the sum of its terms' magnitudes, c the number of
roundings a term goes through: the d of its dot product, one for each of the L
terms of a sum, 3 |n g| + 4 in a weight exp2(n g log2 e) (three roundings of
the exponent, which stands n g from 0, and the instruction's own). For bfloat16
io the decayed scores and the state are rounded once on their way into y's
products (half a step: 2^-8 of each term), and the output once more. The
magnitudes come from the oracle on the absolute values of its inputs."""
import sys

import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import linattn as la

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make(b, L, H, G, dk, dv, dtype, seed=0, state=False, docs=0, backward=False, steep=False):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = dict(q=rnd(b, L, G, dk).to(dtype), k=rnd(b, L, G, dk).to(dtype), v=rnd(b, L, H, dv).to(dtype),
             log_decay=-torch.exp2(-1.0 - 7.0 * torch.arange(H) / max(1, H - 1)) * (8 if steep else 1),
             state=2 * rnd(b, H, dv, dk) if state else None, seq_idx=None)
    if docs:
        a["seq_idx"] = torch.cumsum(torch.rand(b, L, generator=g) < 1.0 / docs, 1).to(torch.int32)
    if backward:
        a["dy"] = rnd(b, L, H, dv).to(dtype)
        a["dstate"] = rnd(b, H, dv, dk) if state else None
    return a


def gpu(a):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in a.items()}


def steps(a):
    L, d = a["q"].shape[1], max(a["q"].shape[3], a["v"].shape[3])
    rep = a["v"].shape[2] // a["q"].shape[2]
    return d + L + 4 * L * float(a["log_decay"].abs().max()) + rep + 40


def absolute(a):
    return {n: t.double().abs() if isinstance(t, torch.Tensor) and n not in ("log_decay", "seq_idx") else t
            for n, t in a.items()}


def close(got, want, size, a, what, rounded=True):
    """Every element within the counted bound; `rounded`: an io output (else float32 for either io type)."""
    got = got.detach().cpu().double().numpy()
    tol = steps(a) * U * size + 1e-30
    if rounded and a["q"].dtype == torch.bfloat16:
        tol = tol + BF * np.abs(want) + BF * (1 + BF) * size
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    at = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), "%s: %g off at %s, %g allowed" % (what, err[at], at, tol[at])


def fwd_args(a):
    return [a[n] for n in ("q", "k", "v", "log_decay", "state")]


def check_fwd(a, got, what):
    kw = dict(seq_idx=a["seq_idx"])
    want, size = la.oracle_fwd(*fwd_args(a), **kw), la.oracle_fwd(*fwd_args(absolute(a)), **kw)
    close(got[0], want[0], size[0], a, what + " y")
    if got[1] is not None:
        close(got[1], want[1], size[1], a, what + " state", rounded=False)


def bwd_args(a):
    return [a[n] for n in ("q", "k", "v", "log_decay", "dy", "state", "dstate")]


def check_bwd(a, got, what):
    kw = dict(seq_idx=a["seq_idx"])
    want, size = la.oracle_bwd(*bwd_args(a), **kw), la.oracle_bwd(*bwd_args(absolute(a)), **kw)
    assert set(got) == ({"dq", "dk", "dv", "dstate"} if a["state"] is not None else {"dq", "dk", "dv"})
    for n in got:
        close(got[n], want[n], size[n], a, "%s %s" % (what, n), rounded=n != "dstate")


SHAPES = [
    # batch, seqlen, heads, groups, d_k, d_v
    (1, 1, 1, 1, 8, 8),
    (2, 2, 2, 1, 64, 64),
    (1, 63, 3, 3, 128, 64),
    (2, 64, 2, 2, 64, 128),
    (1, 65, 4, 2, 128, 128),
    (3, 127, 2, 2, 40, 96),
    (1, 129, 6, 2, 72, 24),
    (2, 200, 3, 1, 16, 120),
    (1, 513, 2, 2, 128, 8),
    (1, 1100, 1, 1, 64, 64),   # split into segments
]


@pytest.mark.parametrize("docs", [0, 40], ids=["one", "packed"])
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_fwd(shape, dtype, state, docs):
    say("lin_attn fwd", shape, dtype, state, docs)
    a = make(*shape, DT[dtype], seed=sum(shape), state=state, docs=docs)
    d = gpu(a)
    got = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    check_fwd(a, got, str(shape))


@pytest.mark.parametrize("docs", [0, 40], ids=["one", "packed"])
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bwd(shape, dtype, state, docs):
    say("lin_attn bwd", shape, dtype, state, docs)
    a = make(*shape, DT[dtype], seed=sum(shape) + 1, state=state, docs=docs, backward=True)
    d = gpu(a)
    got = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    check_bwd(a, got, str(shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 4, 2, 128, 64), (5, 3, 3, 24, 40), (2, 6, 2, 64, 128),
                                   (7, 2, 2, 32, 16), (33, 12, 12, 128, 128)], ids=str)
def test_step(shape, dtype):
    b, H, G, dk, dv = shape
    say("lin_attn step", shape, dtype)
    a = make(b, 1, H, G, dk, dv, DT[dtype], seed=sum(shape), state=True)
    d = gpu(a)
    y, s = ms.lin_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"])
    st = d["state"].clone()
    y2, s2 = ms.lin_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], st, inplace=True)
    torch.cuda.synchronize()
    assert s2 is st and torch.equal(s2, s) and torch.equal(y2, y)
    want, size = la.oracle_fwd(*fwd_args(a)), la.oracle_fwd(*fwd_args(absolute(a)))
    # the step multiplies in float32 throughout: one rounding of the output
    tol = steps(a) * U * size[0] + (BF * np.abs(want[0]) if dtype == "bf16" else 0)
    assert (np.abs(y.cpu().double().numpy() - want[0][:, 0]) <= tol[:, 0]).all()
    close(s, want[1], size[1], a, "state", rounded=False)


def test_fwd_then_steps_then_fwd():
    """A prompt, tokens one by one on its state in place, and a second turn, against the whole sequence at once."""
    a = make(2, 150, 4, 2, 64, 96, torch.float32, seed=9)
    d = gpu(a)
    part = lambda lo, hi: [d[n][:, lo:hi] for n in "qkv"] + [d["log_decay"]]  # noqa: E731
    y1, s = ms.lin_attn_fwd(*part(0, 70))
    ys = [y1]
    for t in range(70, 80):
        y, s = ms.lin_attn_step(*[d[n][:, t] for n in "qkv"], d["log_decay"], s, inplace=True)
        ys.append(y[:, None])
    y2, s2 = ms.lin_attn_fwd(*part(80, 150), s, state_out=s)
    torch.cuda.synchronize()
    assert s2 is s
    check_fwd(a, (torch.cat(ys + [y2], 1), s), "turns")


def test_in_place_state_of_a_split_sequence():
    """The last segment writes the state that the first one starts from."""
    a = make(1, 1500, 2, 2, 64, 64, torch.bfloat16, seed=10, state=True)
    d = gpu(a)
    assert ms.lin_attn_workspace_bytes(1, 1500, 2, 2, 64, 64, torch.bfloat16) > 0
    want = ms.lin_attn_fwd(*fwd_args(d))
    for _ in range(5):
        st = d["state"].clone()
        y, s = ms.lin_attn_fwd(*fwd_args(dict(d, state=st)), state_out=st)
        torch.cuda.synchronize()
        assert s is st and torch.equal(s, want[1]) and torch.equal(y, want[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_columns_of_one_projection_are_read_in_place(dtype):
    b, L, H, dk, dv = 2, 130, 3, 64, 40
    wide = torch.randn(b, L, H * (2 * dk + 2 * dv) + 8, generator=torch.Generator().manual_seed(4)).to(DT[dtype]).cuda()
    cols = torch.split(wide[..., :-8], [H * dk, H * dk, H * dv, H * dv], -1)
    q, k, v, dy = (t.unflatten(-1, (H, -1)) for t in cols)
    g = -torch.tensor([0.5, 0.1, 0.02], device="cuda")
    y, s = ms.lin_attn_fwd(q, k, v, g)
    y2, s2 = ms.lin_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g)
    grads = ms.lin_attn_bwd(q, k, v, g, dy)
    grads2 = ms.lin_attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, dy.contiguous())
    yt, st = ms.lin_attn_step(q[:, 5], k[:, 5], v[:, 5], g, s)
    yt2, st2 = ms.lin_attn_step(q[:, 5].contiguous(), k[:, 5].contiguous(), v[:, 5].contiguous(), g, s)
    # rows whose layout no stride describes are copied
    y3, _ = ms.lin_attn_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, g)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(yt, yt2) and torch.equal(st, st2)
    assert torch.equal(y, y3)
    for n in grads:
        assert torch.equal(grads[n], grads2[n]), n


def test_no_memory_and_steep_decays():
    """log_decay -inf leaves each token its own product (a weight of 0^0 is 1); steep decays underflow to 0."""
    a = make(1, 100, 3, 3, 32, 32, torch.float32, seed=12, state=True)
    a["log_decay"] = torch.tensor([-float("inf"), -80.0, -1.0])
    d = gpu(a)
    y, s = ms.lin_attn_fwd(*fwd_args(d))
    yt, st = ms.lin_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"])
    torch.cuda.synchronize()
    b = dict(a, log_decay=torch.tensor([-1e4, -80.0, -1.0]))
    want, size = la.oracle_fwd(*fwd_args(b)), la.oracle_fwd(*fwd_args(absolute(b)))
    c = dict(a, log_decay=torch.ones(3))  # the count of roundings: terms of weight e^-x are off by x u e^-x < u
    close(y, want[0], size[0], c, "y")
    close(s, want[1], size[1], c, "state")
    assert torch.allclose(yt, y[:, 0], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_tokens_that_are_masked_leave_no_trace(which, bad, dtype):
    """An infinity or NaN in one token reaches only that document's tokens from there on: the others come out bit
    for bit as with an ordinary token in its place."""
    a = make(1, 300, 2, 2, 64, 64, DT[dtype], seed=13, state=True)
    ids = torch.zeros(1, 300, dtype=torch.int32)
    ids[:, 90:] = 1
    ids[:, 205:] = 2
    a["seq_idx"] = ids
    at = 140  # in document 1, between tokens of its own chunk and of others
    d = gpu(a)
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    d[which] = d[which].clone()
    d[which][0, at, 1, 3] = bad
    y1, s1 = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    assert not torch.isfinite(y1[0, at, 1]).all()
    keep = torch.ones(300, dtype=torch.bool)
    keep[at:205] = False
    tol = dict(rtol=1e-5, atol=1e-5) if dtype == "f32" else dict(rtol=0.02, atol=0.02)
    torch.testing.assert_close(y1[:, keep.cuda()], y0[:, keep.cuda()], **tol)
    assert torch.equal(y1[:, :, 0], y0[:, :, 0]), "another head"
    assert torch.equal(s1, s0), "the state follows the last document"


@pytest.mark.parametrize("which", ["q", "k", "v", "dy"])
def test_gradients_of_masked_tokens(which):
    """The same for the gradients: a NaN in one document stays out of the others'."""
    a = make(1, 200, 2, 1, 32, 64, torch.float32, seed=14, state=True, backward=True)
    ids = torch.zeros(1, 200, dtype=torch.int32)
    ids[:, 70:] = 1
    ids[:, 150:] = 2
    a["seq_idx"] = ids
    d = gpu(a)
    g0 = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    d[which] = d[which].clone()
    d[which][0, 100, 0, 3] = float("nan")
    g1 = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv"):
        for lo, hi in ((0, 70), (150, 200)):
            torch.testing.assert_close(g1[n][:, lo:hi], g0[n][:, lo:hi], rtol=1e-5, atol=1e-5)
    assert torch.equal(g1["dstate"], g0["dstate"])


def test_infinite_state_and_value_stay_infinite():
    """An infinite value gives an infinite state element, not NaN, where the key is finite and not 0."""
    a = make(1, 70, 1, 1, 32, 32, torch.bfloat16, seed=15)
    a["k"] = a["k"].abs() + 1
    a["v"][0, 10, 0, 2] = float("inf")
    d = gpu(a)
    _, s = ms.lin_attn_fwd(*fwd_args(d))
    torch.cuda.synchronize()
    assert torch.isinf(s[0, 0, 2]).all() and torch.isfinite(s[0, 0, [0, 1, 3]]).all()


def test_gradients_against_differences():
    """d loss / d(step along a direction) of the GPU's own forward against its gradients."""
    a = make(1, 150, 2, 1, 64, 64, torch.float32, seed=16, state=True, backward=True, docs=60)
    d = gpu(a)
    g = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])

    def loss(**over):
        e = dict(d, **over)
        y, s = ms.lin_attn_fwd(*fwd_args(e), seq_idx=d["seq_idx"])
        return float((y.double() * d["dy"].double()).sum() + (s.double() * d["dstate"].double()).sum())

    size = la.oracle_fwd(*fwd_args(absolute(a)), seq_idx=a["seq_idx"])
    scale = float((size[0] * np.abs(a["dy"].numpy())).sum() + (size[1] * np.abs(a["dstate"].numpy())).sum())
    for n in ("q", "k", "v", "state"):
        w = torch.randn(d[n].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        slope = (loss(**{n: d[n] + w}) - loss(**{n: d[n] - w})) / 2  # the loss is linear in each
        got = float((g["d" + n].double() * w.double()).sum())
        assert abs(slope - got) <= 8 * steps(a) * U * scale, n


def test_is_deterministic_and_ignores_the_workspace():
    a = make(2, 700, 4, 2, 128, 64, torch.bfloat16, seed=17, state=True, backward=True, docs=100)
    d = gpu(a)
    ref = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"])
    gref = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"])
    size = [ms.lin_attn_workspace_bytes(2, 700, 4, 2, 128, 64, torch.bfloat16, backward=b) for b in (False, True)]
    assert size[1] > 0
    ws = [torch.full((max(s, 256),), 0x7F, dtype=torch.uint8, device="cuda") for s in size]
    y, s = ms.lin_attn_fwd(*fwd_args(d), seq_idx=d["seq_idx"], workspace=ws[0])
    g = ms.lin_attn_bwd(*bwd_args(d), seq_idx=d["seq_idx"], workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(s, ref[1])
    for n in gref:
        assert torch.equal(g[n], gref[n]), n


def test_streams_and_captured_graphs():
    """Two graphs with workspaces of their own, replayed by turns and beside eager calls on another stream."""
    a = make(1, 1300, 2, 2, 64, 64, torch.bfloat16, seed=18, state=True, backward=True)
    d = gpu(a)
    ref, gref = ms.lin_attn_fwd(*fwd_args(d)), ms.lin_attn_bwd(*bwd_args(d))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((ms.lin_attn_fwd(*fwd_args(d)), ms.lin_attn_bwd(*bwd_args(d)),
                         ms.lin_attn_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["log_decay"], d["state"])))
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        for (y, s), gr, _ in outs:
            y.zero_(), s.zero_(), [t.zero_() for t in gr.values()]
        graphs[i % 2].replay()
        with torch.cuda.stream(side):
            ye, se = ms.lin_attn_fwd(*fwd_args(d))
        graphs[(i + 1) % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(ye, ref[0]) and torch.equal(se, ref[1])
        for (y, s), gr, (yt, st) in outs:
            assert torch.equal(y, ref[0]) and torch.equal(s, ref[1])
            assert all(torch.equal(gr[n], gref[n]) for n in gref)


def test_rows_past_2_31_elements():
    """Rows 2^24 elements apart: the last tokens lie more than 2^31 elements from the first (read in place)."""
    L, H, d = 190, 1, 64
    wide = torch.empty(1, L, 1 << 24, dtype=torch.bfloat16, device="cuda")
    a = make(1, L, H, H, d, d, torch.bfloat16, seed=19, backward=True)
    v = {}
    for i, n in enumerate(("q", "k", "v", "dy")):
        v[n] = wide[..., i * d:(i + 1) * d].view(1, L, 1, d)
        v[n].copy_(a[n])
    g = a["log_decay"].cuda()
    got = ms.lin_attn_fwd(v["q"], v["k"], v["v"], g)
    grads = ms.lin_attn_bwd(v["q"], v["k"], v["v"], g, v["dy"])
    torch.cuda.synchronize()
    assert (L - 1) << 24 > 1 << 31
    check_fwd(a, got, "wide rows")
    check_bwd(a, grads, "wide rows")


def test_many_rows_at_once():
    """More workgroups than one dispatch holds at a time, most of them of one token."""
    b, H = 5000, 16
    a = make(b, 1, H, 4, 16, 16, torch.bfloat16, seed=20, state=True, backward=True)
    d = gpu(a)
    got = ms.lin_attn_fwd(*fwd_args(d))
    grads = ms.lin_attn_bwd(*bwd_args(d))
    torch.cuda.synchronize()
    check_fwd(a, got, "many rows")
    check_bwd(a, grads, "many rows")
